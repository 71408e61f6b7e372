"""Host side of the expert layer's calls that needs no GPU: limits, workspace sizes, and every kind of refusal.
A refused call returns before it touches the handle or a device, so a zeroed block serves as one."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 1 << 20  # made-up device addresses, never read


@pytest.fixture(scope="module")
def pmx():
    from preconditioned_optimizer_matrix_amd import pmx
    return pmx


@pytest.fixture(scope="module")
def fake():
    return ctypes.create_string_buffer(4096)


def _at(i):
    return BASE + (i << 24)


def _size(pmx, name, *args):
    sz = ctypes.c_size_t(1 << 60)
    code = getattr(pmx.lib, name)(*args, ctypes.byref(sz))
    return code, sz.value


def _refusals(call, good, bad, codes):
    """Each change of `good` is refused with its code."""
    for change, code in zip(bad, codes):
        args = dict(good)
        args.update(change)
        assert call(**args) == code, change


def test_constants_and_struct_match_the_header(pmx):
    src = open(os.path.join(ROOT, "include", "pmx.h")).read()
    for name in ("MAX_NORM_COLS", "MAX_ROUTE_TOP", "MAX_ROUTE_ROWS"):
        assert int(re.search(r"#define PMX_%s (\d+)" % name, src).group(1)) == getattr(pmx, name)
    body = src[:src.index("} pmx_route_problem;")]
    body = re.sub(r"/\*.*?\*/", "", body[body.rindex("typedef struct {") + 16:], flags=re.S)
    assert re.findall(r"(\w+)\s*[,;]", body) == [f[0] for f in pmx.RouteProblem._fields_]


def test_workspace_sizes(pmx):
    f = "pmx_layer_norm_grad_workspace_size"
    assert _size(pmx, f, 0, 100, pmx.F32) == (pmx.OK, 0)
    for rows, cols in ((1, 1), (100, 1000), (1 << 20, 16384)):
        for dt in (pmx.F32, pmx.BF16):
            code, n = _size(pmx, f, rows, cols, dt)
            assert code == pmx.OK and n > 0 and n % (8 * cols) == 0 and n <= 512 * 8 * cols
    for bad in ((-1, 8, 0), (8, 0, 0), (8, pmx.MAX_NORM_COLS + 1, 0), (8, 8, 2)):
        assert _size(pmx, f, *bad)[0] == pmx.ERR_INVALID_VALUE
    assert pmx.lib.pmx_layer_norm_grad_workspace_size(8, 8, 0, None) == pmx.ERR_INVALID_VALUE

    def route(**kw):
        q = pmx.RouteProblem(1, pmx.F32, 100, 32, 4, _at(0), 32, None, 0.1, 0.1, 1, 0)
        for k, v in kw.items():
            setattr(q, k, v)
        return _size(pmx, "pmx_route_workspace_size", ctypes.byref(q))

    assert route(rows=64) == (pmx.OK, 0) and route(rows=0) == (pmx.OK, 0)
    # a chunk's sums and byte counts, 64 tokens a chunk up to 256 experts
    assert route()[1] >= 2 * (32 * 4 + 32) and route(rows=32768, experts=64, top=4)[1] >= 512 * (64 * 4 + 64)
    # with many chunks the counts before each as well
    assert route(rows=1 << 20)[1] >= (1 << 14) * (32 * 8 + 32)
    for kw in (dict(rows=-1), dict(rows=pmx.MAX_ROUTE_ROWS + 1), dict(experts=0), dict(experts=pmx.MAX_GROUPS + 1), dict(top=0),
               dict(top=33), dict(experts=64, top=pmx.MAX_ROUTE_TOP + 1), dict(dtype=3), dict(struct_version=2), dict(reserved=1)):
        assert route(**kw)[0] == pmx.ERR_INVALID_VALUE, kw


def test_layer_norm_refusals(pmx, fake):
    I, A = pmx.ERR_INVALID_VALUE, pmx.ERR_ALIAS

    def call(h=fake, x=_at(0), dt=0, rows=8, cols=100, ldx=100, w=_at(1), b=_at(2), pt=0, eps=1e-5, y=_at(3), ldy=100, stats=_at(4)):
        return pmx.lib.pmx_layer_norm(h, x, dt, rows, cols, ldx, w, b, pt, eps, y, ldy, stats, None)

    bad = [dict(h=None), dict(x=None), dict(x=_at(0) + 2), dict(dt=2), dict(rows=-1), dict(cols=0), dict(cols=16385, ldx=16385, ldy=16385),
           dict(ldx=99), dict(ldy=99), dict(w=_at(1) + 1), dict(b=_at(2) + 2), dict(pt=5), dict(eps=-1.0), dict(eps=float("inf")),
           dict(eps=float("nan")), dict(y=None), dict(stats=_at(4) + 2)]
    _refusals(call, {}, bad, [I] * len(bad))
    for kw in (dict(y=_at(0)), dict(y=_at(0) + 3196), dict(stats=_at(0) + 64), dict(y=_at(1)), dict(stats=_at(3) + 400), dict(b=_at(4) + 60)):
        assert call(**kw) == A, kw
    assert call(rows=0, x=None, y=None, stats=None) == pmx.OK

    def grad(h=fake, dy=_at(0), dt=0, rows=8, cols=100, lddy=100, x=_at(1), ldx=100, stats=_at(2), w=_at(3), pt=0, dx=_at(4), lddx=100,
             dw=_at(5), db=_at(6), acc=0, ws=_at(7), n=1 << 20):
        return pmx.lib.pmx_layer_norm_grad(h, dy, dt, rows, cols, lddy, x, ldx, stats, w, pt, dx, lddx, dw, db, acc, ws, n, None)

    bad = [dict(h=None), dict(dy=None), dict(dt=2), dict(cols=0), dict(lddy=99), dict(x=None), dict(ldx=99), dict(stats=None),
           dict(stats=_at(2) + 2), dict(w=_at(3) + 2), dict(pt=-1), dict(lddx=99), dict(dx=_at(4) + 1), dict(dw=_at(5) + 2), dict(db=_at(6) + 1),
           dict(acc=2)]
    _refusals(grad, {}, bad, [I] * len(bad))
    for kw in (dict(dx=_at(1)), dict(dx=_at(0) + 4), dict(dx=_at(0), lddx=101), dict(dw=_at(4)), dict(dw=_at(6)), dict(db=_at(1)), dict(ws=_at(4)),
               dict(ws=_at(2)), dict(dw=_at(3))):
        assert grad(**kw) == A, kw
    for kw in (dict(ws=None), dict(n=8), dict(ws=_at(7) + 4)):
        assert grad(**kw) == pmx.ERR_WORKSPACE, kw
    assert grad(dx=None, dw=None, db=None, ws=None, n=0) == pmx.OK  # nothing is wanted


def test_route_refusals(pmx, fake):
    I, A = pmx.ERR_INVALID_VALUE, pmx.ERR_ALIAS

    def problem(kw):
        q = pmx.RouteProblem(1, pmx.F32, 100, 32, 4, _at(0), 32, _at(1), 0.1, 0.1, 1, 0)
        for k in [f[0] for f in pmx.RouteProblem._fields_]:
            if k in kw:
                setattr(q, k, kw.pop(k))
        return q

    def call(**kw):
        q = problem(kw)
        a = dict(h=fake, ids=_at(2), gates=_at(3), counts=_at(4), offsets=_at(5), slots=_at(6), tokens=_at(7), loss=_at(8), ws=_at(9), n=1 << 20)
        a.update(kw)
        return pmx.lib.pmx_route(a["h"], ctypes.byref(q), a["ids"], a["gates"], a["counts"], a["offsets"], a["slots"], a["tokens"], a["loss"],
                                 a["ws"], a["n"], None)

    bad = [dict(h=None), dict(z=None), dict(z=_at(0) + 2), dict(ldz=31), dict(balance=float("inf")), dict(zloss=float("nan")), dict(normalize=2),
           dict(top=0), dict(top=33), dict(ids=None), dict(gates=None), dict(counts=None), dict(offsets=None), dict(loss=None), dict(slots=None),
           dict(tokens=None), dict(ids=_at(2) + 2), dict(tokens=_at(7) + 1)]
    for kw in bad:
        assert call(**kw) == I, kw
    for kw in (dict(ids=_at(0) + 128), dict(gates=_at(2)), dict(tokens=_at(6) + 1596), dict(counts=_at(5)), dict(loss=_at(4) + 128), dict(slots=_at(1)),
               dict(ws=_at(3)), dict(ws=_at(0))):
        assert call(**kw) == A, kw
    for kw in (dict(ws=None), dict(n=64), dict(ws=_at(9) + 128)):
        assert call(**kw) == pmx.ERR_WORKSPACE, kw

    def grad(**kw):
        q = problem(kw)
        a = dict(h=fake, ids=_at(2), gates=_at(3), counts=_at(4), dg=_at(5), up=_at(6), dz=_at(7), ld=32)
        a.update(kw)
        return pmx.lib.pmx_route_grad(a["h"], ctypes.byref(q), a["ids"], a["gates"], a["counts"], a["dg"], a["up"], a["dz"], a["ld"], None)

    for kw in (dict(h=None), dict(z=None), dict(counts=None), dict(ids=None), dict(gates=None), dict(dz=None), dict(ld=31), dict(dg=_at(5) + 2),
               dict(up=_at(6) + 1), dict(struct_version=0)):
        assert grad(**kw) == I, kw
    for kw in (dict(dz=_at(0) + 4), dict(dz=_at(0), ld=33), dict(dz=_at(5)), dict(dz=_at(4)), dict(dz=_at(1)), dict(dz=_at(6))):
        assert grad(**kw) == A, kw


def test_8bit_refusals(pmx, fake):
    I, A, L = pmx.ERR_INVALID_VALUE, pmx.ERR_ALIAS, pmx.lib

    def store(h=fake, x=_at(0), dt=1, rows=8, cols=200, ldx=200, v=_at(1), ldv=256, s=_at(2), lds=2):
        return L.pmx_fp8_store(h, x, dt, rows, cols, ldx, v, ldv, s, lds, None)

    common = [dict(h=None), dict(dt=2), dict(rows=-1), dict(cols=0), dict(cols=(1 << 20) + 1), dict(v=None), dict(v=_at(1) + 8), dict(ldv=264),
              dict(ldv=240), dict(s=None), dict(lds=1)]
    for kw in common + [dict(x=None), dict(x=_at(0) + 1), dict(ldx=199)]:
        assert store(**kw) == I, kw
    for kw in (dict(v=_at(0)), dict(s=_at(0) + 5), dict(s=_at(1) + 300)):
        assert store(**kw) == A, kw
    assert store(rows=0, x=None, v=None, s=None) == pmx.OK

    def load(h=fake, v=_at(0), ldv=256, s=_at(1), lds=2, rows=8, cols=200, y=_at(2), dt=1, ldy=200):
        return L.pmx_fp8_load(h, v, ldv, s, lds, rows, cols, y, dt, ldy, None)

    for kw in common + [dict(y=None), dict(ldy=199), dict(y=_at(2) + 1)]:
        kw = {k: (v if k != "v" or v is None else _at(0) + 8) for k, v in kw.items()}
        assert load(**kw) == I, kw
    assert load(y=_at(0)) == A and load(y=_at(1)) == A

    def weight(h=fake, w=_at(0), dt=1, groups=2, n=200, k=300, ldw=300, sw=60000, tr=0, v=_at(1), ldv=384, sv=76800, s=_at(2), lds=3, ss=6):
        return L.pmx_fp8_store_weight(h, w, dt, groups, n, k, ldw, sw, tr, v, ldv, sv, s, lds, ss, None)

    for kw in (dict(h=None), dict(w=None), dict(dt=3), dict(groups=0), dict(groups=1001), dict(n=0), dict(k=0), dict(ldw=299), dict(sw=59999),
               dict(sw=-1), dict(tr=2), dict(v=_at(1) + 4), dict(ldv=368), dict(ldv=392), dict(sv=76784), dict(sv=76808), dict(lds=2), dict(ss=5),
               dict(tr=1), dict(tr=1, ldv=256, sv=300 * 256, lds=2, ss=5)):
        assert weight(**kw) == I, kw
    assert weight(v=_at(0)) == A and weight(s=_at(1) + 76800) == A
    assert weight(groups=1000, n=1 << 20, k=1 << 20, ldw=1 << 20, sw=1 << 40, ldv=1 << 20, sv=1 << 40, lds=1 << 13, ss=1 << 26) == pmx.ERR_NOT_SUPPORTED

    def silu(h=fake, x=_at(0), dt=1, rows=8, cols=200, ldh=400, gated=1, a=_at(1), lda=200, v=_at(2), ldv=512, s=_at(3), lds=4):
        return L.pmx_silu_checkpoint(h, x, dt, rows, cols, ldh, gated, a, lda, v, ldv, s, lds, None)

    for kw in (dict(h=None), dict(x=None), dict(dt=9), dict(gated=2), dict(ldh=399), dict(lda=199), dict(a=None), dict(ldv=496), dict(lds=3),
               dict(v=None), dict(cols=0)):
        assert silu(**kw) == I, kw
    assert silu(a=_at(0)) == A and silu(v=_at(0)) == A and silu(s=_at(2) + 512) == A

    def sgrad(h=fake, da=_at(0), dt=1, rows=8, cols=200, ldda=200, v=_at(1), ldv=512, s=_at(2), lds=4, gated=1, dh=_at(3), lddh=400, a=_at(4),
              lda=200):
        return L.pmx_silu_checkpoint_grad(h, da, dt, rows, cols, ldda, v, ldv, s, lds, gated, dh, lddh, a, lda, None)

    for kw in (dict(h=None), dict(da=None), dict(dt=9), dict(gated=-1), dict(ldda=199), dict(lddh=399), dict(lda=199), dict(a=_at(4) + 1),
               dict(dh=None), dict(ldv=384), dict(lds=2)):
        assert sgrad(**kw) == I, kw
    assert sgrad(dh=_at(0)) == A and sgrad(a=_at(3)) == A and sgrad(a=_at(1)) == A


def test_fp8_product_refusals(pmx, fake):
    I, A = pmx.ERR_INVALID_VALUE, pmx.ERR_ALIAS

    def call(h=fake, a=_at(0), rows=8, k=200, lda=256, sa=_at(1), ldas=2, b=_at(2), n=100, ldb=256, sb=25600, bs=_at(3), ldbs=2, sbs=2, off=_at(4),
             it=0, groups=3, c=_at(5), ot=1, ldc=100):
        return pmx.lib.pmx_fp8_product(h, a, rows, k, lda, sa, ldas, b, n, ldb, sb, bs, ldbs, sbs, off, it, groups, c, ot, ldc, None)

    for kw in (dict(h=None), dict(a=None), dict(rows=-1), dict(k=(1 << 20) + 1), dict(a=_at(0) + 8), dict(lda=240), dict(lda=264), dict(sa=None), dict(ldas=1), dict(b=None), dict(ldb=240),
               dict(sb=25584), dict(sb=25601), dict(sb=-16), dict(bs=None), dict(ldbs=1), dict(sbs=1), dict(off=None), dict(off=_at(4) + 2), dict(it=2),
               dict(groups=0), dict(groups=1001), dict(c=None), dict(ot=2), dict(ldc=99), dict(c=_at(5) + 1), dict(k=0), dict(n=0)):
        assert call(**kw) == I, kw
    for kw in (dict(c=_at(0)), dict(c=_at(2) + 51200), dict(c=_at(4) - 2), dict(c=_at(3)), dict(c=_at(1) - 4)):
        assert call(**kw) == A, kw
    for kw in (dict(lda=(1 << 22) + 16), dict(ldb=(1 << 22) + 16, sb=1 << 31), dict(rows=1 << 30, n=1 << 20, ldc=1 << 20, sb=1 << 28, sbs=1 << 15, c=1 << 60)):
        assert call(**kw) == pmx.ERR_NOT_SUPPORTED, kw
    assert call(rows=0, a=None, sa=None, c=None) == pmx.OK


@pytest.mark.skipif("SAN_CHILD" in os.environ, reason="this is the child")
def test_clean_under_host_sanitizers():
    from preconditioned_optimizer_matrix_amd import build
    src = os.path.join(build.CSRC, "pmx_layer_api.hip")
    if not os.path.exists(build.SAN_LIB) or os.path.getmtime(build.SAN_LIB) < os.path.getmtime(src):
        build.build_sanitized(verbose=False)
    env = dict(os.environ, PMX_LIBRARY=build.SAN_LIB, LD_PRELOAD=build.asan_runtime(), SAN_CHILD="1",
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and " passed" in out, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
