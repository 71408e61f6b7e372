"""Values in 8 bits, byte for byte against the definition, and silu from them.

The stored bytes have one right value each (scaling by a power of two is exact,
ties go to even).  silu's tolerance (u = 2^-24): exp(-x) is off by (|x| + 3) u
relative (its argument's rounding, and 2 u of the instruction), 1 / (1 + e) by
that times at most 1, and 3 u; a product each adds u; results round by half a
step of their type.  1 + x (1 - s) can cancel, so its error is taken of 1 + |x|."""
import math

import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    from preconditioned_optimizer_matrix_amd import pmx
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    return torch, pmx


def _power(torch, k):
    """2^k in fp64, exactly, for whole k of -150 .. 150."""
    return torch.tensor([2.0 ** i for i in range(-150, 151)], dtype=torch.float64)[k.long() + 150]


def _code(amax):
    """k + 127 of the least k >= -126 with amax <= 448 2^k."""
    if amax == 0:
        return 127
    k = -126
    while amax > math.ldexp(448.0, k):
        k += 1
    return k + 127


def _e4m3(torch, u):
    """The e4m3 byte nearest to each |u| <= 448 (fp64), ties to even; NaN: 0x7f."""
    table = torch.tensor(
        [math.ldexp((m if e == 0 else 8 + m), (1 if e == 0 else e) - 10) for e in range(16) for m in range(8)][:127],
        dtype=torch.float64)
    a = u.abs()
    hi = torch.searchsorted(table, a.nan_to_num(0.0)).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up = table[hi] - a
    down = a - table[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)) | (table[hi] == a), hi, lo)
    pick = torch.where(a.isnan(), torch.full_like(pick, 0x7F), pick)
    return (pick | (torch.signbit(u) & ~u.isnan()).long() << 7).to(torch.uint8)


def _stored(torch, x):
    """(bytes, codes) of the rows of x."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x.double(), (0, -cols % 128))
    b = x.view(rows, -1, 128)
    fin = torch.where(b.isfinite(), b.abs(), torch.zeros_like(b))
    codes = torch.tensor([[_code(float(v)) for v in r] for r in fin.amax(2)], dtype=torch.uint8).view(rows, -1)
    u = b * _power(torch, 127 - codes.long())[:, :, None]
    return _e4m3(torch, torch.where(b.isfinite(), u, torch.full_like(u, math.nan))).view(rows, -1), codes


def _value(torch, q, codes, cols=None):
    v = q.cpu().view(torch.float8_e4m3fn).float().double().view(q.shape[0], -1, 128) * _power(torch, codes.cpu().long() - 127)[:, :, None]
    v = v.view(q.shape[0], -1)
    return v if cols is None else v[:, :cols]


def _same(torch, q, want):
    q = q.view(torch.uint8).cpu()
    nan = (want & 0x7F) == 0x7F  # a NaN's sign is free
    return bool(((q == want) | (nan & ((q & 0x7F) == 0x7F))).all())


def _wild(torch, rows, cols, dt, seed):
    """Values over many sizes, ties and the borders of a block's power among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-40, 40, (rows, 1), generator=g).float())
    x = x * torch.exp2(torch.randint(-12, 2, (rows, cols), generator=g).float())
    x[rows // 2] = (torch.randint(-448, 449, (cols,), generator=g)).float() * 0.5  # halves: ties
    x[rows // 3] = 0.0
    if rows > 3:
        x[1] = torch.finfo(dt).tiny * torch.randn(cols, generator=g)
        x[2] = torch.finfo(dt).max * torch.rand(cols, generator=g)
    x = x.to(dt)
    x[0, 0] = 448.0 if rows > 1 else x[0, 0]
    return x


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 128), (9, 127), (11, 129), (40, 515), (6, 1000), (5, 2048), (3, 4100), (300, 40)])
def test_store_and_load(env, rows, cols, dt):
    torch, pmx = env
    print("fp8 store", rows, cols, dt, flush=True)
    x = _wild(torch, rows, cols, getattr(torch, dt), rows * 3 + cols)
    q, s = pmx.fp8_store(x.cuda())
    wq, ws = _stored(torch, x)
    assert q.dtype == torch.float8_e4m3fn and q.shape == wq.shape and torch.equal(s.cpu(), ws) and _same(torch, q, wq)
    for out in (torch.bfloat16, torch.float32):
        y = pmx.fp8_load(q, s, cols, dtype=out)
        # four significant bits: exact, but for what lies below bf16's normal numbers, and 256 * 2^120 = 2^128, to
        # which magnitudes from 248 * 2^120 = 0.97 * 2^128 on are rounded and which is infinity in both types
        want = _value(torch, q.view(torch.uint8), s, cols).to(out)
        near = (y.double().cpu() - want.double()).abs() <= 2.0 ** -133 * (1 if out == torch.bfloat16 else 0)
        assert bool((near | (y.cpu() == want)).all())


def test_borders_and_special_values(env):
    torch, pmx = env
    rows = []
    for e in (-100, -8, 0, 5, 90):
        for f in (1.0, 1.5, 1.75, math.nextafter(1.75, 2), 1.9999):
            r = torch.zeros(128, dtype=torch.float64)
            r[3] = math.ldexp(f, e)
            r[4:20] = math.ldexp(f, e) * 2.0 ** -torch.arange(1, 17).double()
            rows.append(r)
    x = torch.stack(rows).float()
    x[0, 100:104] = torch.tensor([math.inf, -math.inf, math.nan, -0.0])
    x[1] = math.nan
    x[2] = torch.finfo(torch.float32).tiny / 8  # subnormal
    q, s = pmx.fp8_store(x.cuda())
    wq, ws = _stored(torch, x)
    assert torch.equal(s.cpu(), ws) and _same(torch, q, wq)
    y = pmx.fp8_load(q, s, dtype=torch.float32).cpu()
    assert bool(y[0, 100:103].isnan().all()) and float(y[0, 3]) == float(x[0, 3]) and bool(y[1].isnan().all())


def test_every_byte_reads_back(env):
    torch, pmx = env
    q = torch.arange(256, dtype=torch.uint8).view(2, 128).repeat(5, 1).contiguous()
    s = torch.tensor([127, 127, 1, 1, 100, 100, 200, 200, 247, 247], dtype=torch.uint8).view(10, 1)
    want = _value(torch, q, s)
    for dt in (torch.float32, torch.bfloat16):
        y = pmx.fp8_load(q.view(torch.float8_e4m3fn).cuda(), s.cuda(), dtype=dt).cpu()
        w = want.to(dt)
        assert bool(((y == w) | (y.isnan() & w.isnan())).all())
    z = pmx.fp8_load(q.view(torch.float8_e4m3fn).cuda(), torch.full((10, 1), 255, dtype=torch.uint8, device="cuda"))
    assert bool(z.isnan().all())


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("groups,n,k", [(1, 1, 1), (1, 128, 128), (2, 130, 127), (3, 40, 300), (2, 257, 515), (5, 64, 1024)])
def test_store_weight(env, groups, n, k, transposed):
    torch, pmx = env
    for dt in (torch.bfloat16, torch.float32):
        w = torch.stack([_wild(torch, n, k, dt, 11 * e + n) for e in range(groups)])
        w[0, 0, 0] = float("nan") if n > 1 else 1.0
        v, s = pmx.fp8_store_weight(w.cuda(), transposed=transposed)
        m = w.transpose(1, 2) if transposed else w
        r, c = m.shape[1:]
        p = torch.nn.functional.pad(m.double(), (0, -c % 128, 0, -r % 128))
        t = p.view(groups, p.shape[1] // 128, 128, p.shape[2] // 128, 128)
        fin = torch.where(t.isfinite(), t.abs(), torch.zeros_like(t)).amax(4).amax(2)
        codes = torch.tensor([_code(float(a)) for a in fin.flatten()], dtype=torch.uint8).view(fin.shape)
        u = t * _power(torch, 127 - codes.long())[:, :, None, :, None]
        want = _e4m3(torch, torch.where(t.isfinite(), u, torch.full_like(u, math.nan))).reshape(p.shape)[:, :r]
        assert torch.equal(s.cpu(), codes) and v.shape == want.shape and _same(torch, v, want)


def _silu(torch, h):
    h = h.double()
    s = 1 / (1 + torch.exp(-h))
    return s, h * s, s * (1 + h * (1 - s))


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 128), (17, 127), (33, 300), (8, 515), (4, 2050), (6, 4096), (400, 24)])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_silu_and_its_gradient(env, rows, cols, gated, dt):
    torch, pmx = env
    print("silu", rows, cols, gated, dt, flush=True)
    dt = getattr(torch, dt)
    half = torch.finfo(dt).eps / 2
    g = torch.Generator().manual_seed(rows + cols)
    h = (torch.randn(rows, (2 if gated else 1) * cols, generator=g) * 4).to(dt)
    h[0, 0] = -80.0
    da = torch.randn(rows, cols, generator=g).to(dt)
    a, q, s = pmx.silu_checkpoint(h.cuda(), gated=gated)
    parts = [h[:, :cols], h[:, cols:]][: 2 if gated else 1]
    wide = -(-cols // 128) * 128
    kept = []
    for i, part in enumerate(parts):
        wq, ws = _stored(torch, part)
        qi, si = q[:, i * wide:(i + 1) * wide], s[:, i * wide // 128:(i + 1) * wide // 128]
        assert torch.equal(si.cpu(), ws) and _same(torch, qi, wq)
        kept.append(_value(torch, wq, ws, cols))
    x = parts[0].double()
    _, y, _ = _silu(torch, x)
    want = y * parts[1].double() if gated else y
    assert bool(((a.double().cpu() - want).abs() <= (half + (x.abs() + 10) * U) * want.abs() + 1e-37).all())
    dh, again = pmx.silu_checkpoint_grad(da.cuda(), q, s, gated=gated)
    sg, y, slope = _silu(torch, kept[0])
    d = da.double()
    up = kept[1] if gated else torch.ones_like(y)
    e = (2 * kept[0].abs() + 20) * U
    tol = d.abs() * up.abs() * sg * (1 + kept[0].abs()) * e + half * (d * up * slope).abs() + 1e-37
    assert bool(((dh[:, :cols].double().cpu() - d * up * slope).abs() <= tol).all())
    if gated:
        assert bool(((dh[:, cols:].double().cpu() - d * y).abs() <= (half + e) * (d * y).abs() + 1e-37).all())
    assert bool(((again.double().cpu() - y * up).abs() <= (half + e) * (y * up).abs() + 1e-37).all())
    only, none = pmx.silu_checkpoint_grad(da.cuda(), q, s, gated=gated, again=False)
    assert none is None and torch.equal(only, dh)


def test_differences(env):
    """dH against central differences of the fp64 formula at the stored values."""
    torch, pmx = env
    g = torch.Generator().manual_seed(2)
    h = torch.randn(9, 2 * 50, generator=g)
    _, q, s = pmx.silu_checkpoint(h.cuda(), gated=True)
    b = torch.cat([_value(torch, q.view(torch.uint8)[:, :128], s[:, :1], 50), _value(torch, q.view(torch.uint8)[:, 128:], s[:, 1:], 50)], 1)
    da = torch.randn(9, 50, generator=g)
    dh, _ = pmx.silu_checkpoint_grad(da.cuda(), q, s, gated=True)
    v = torch.randn(9, 100, generator=g, dtype=torch.float64)

    def value(t):
        x = b + t * v
        return (da.double() * _silu(torch, x[:, :50])[1] * x[:, 50:]).sum()

    want = (value(1e-4) - value(-1e-4)) / 2e-4
    assert abs(float((dh.double().cpu() * v).sum() - want)) <= 1e-6 * float(dh.norm() * v.norm())


def test_strides_and_what_lies_beside(env):
    torch, pmx = env
    for dt in (torch.bfloat16, torch.float32):
        big = torch.randn(30, 900, device="cuda").to(dt)
        x = big[2:25, 7:410]
        v = torch.full((23, 600), 3, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, 16:528]
        sc = torch.full((23, 9), 9, dtype=torch.uint8, device="cuda")[:, 2:6]
        q, s = pmx.fp8_store(x, values=v[:, :512], scales=sc) if v.stride(0) % 16 == 0 else pmx.fp8_store(x)
        wq, ws = pmx.fp8_store(x.contiguous())
        assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s, ws)
        out = torch.full((23, 450), 5.0, device="cuda", dtype=dt)
        y = pmx.fp8_load(q, s, 403, out=out[:, 3:406])
        assert torch.equal(y, pmx.fp8_load(wq, ws, 403, dtype=dt)) and bool((out[:, :3] == 5).all()) and bool((out[:, 406:] == 5).all())
        a, q, s = pmx.silu_checkpoint(x[:, :400], gated=True, out=out[:, 1:201])
        b, q2, s2 = pmx.silu_checkpoint(x[:, :400].contiguous(), gated=True)
        assert torch.equal(a, b) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and bool((out[:, 0] == 5).all())
        da = big[4:27, 1:201]
        g1 = pmx.silu_checkpoint_grad(da, q, s, gated=True)
        g2 = pmx.silu_checkpoint_grad(da.contiguous(), q, s, gated=True)
        assert all(torch.equal(p, r) for p, r in zip(g1, g2))


def test_no_rows(env):
    torch, pmx = env
    x = torch.empty(0, 200, device="cuda")
    q, s = pmx.fp8_store(x)
    assert q.shape == (0, 256) and s.shape == (0, 2) and pmx.fp8_load(q, s, 200).shape == (0, 200)
    a, q, s = pmx.silu_checkpoint(x, gated=True)
    dh, again = pmx.silu_checkpoint_grad(a, q, s, gated=True)
    assert dh.shape == (0, 200) and again.shape == (0, 100)


def test_refusals(env):
    torch, pmx = env
    x = torch.randn(4, 256, device="cuda")
    q, s = pmx.fp8_store(x)

    def refused(f, kind=(ValueError, TypeError)):
        with pytest.raises(kind):
            f()

    refused(lambda: pmx.fp8_store(x.half()))
    refused(lambda: pmx.fp8_store(x.t()))
    refused(lambda: pmx.fp8_store(x, values=q[:, :128]))
    refused(lambda: pmx.fp8_store(x, scales=s[:3]))
    wide = torch.empty(4, 300, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    refused(lambda: pmx.fp8_store(x, values=wide[:, 1:257]), pmx.PmxError)      # not 16-byte aligned
    odd = torch.empty(4, 264, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    refused(lambda: pmx.fp8_store(x, values=odd[:, :256]), pmx.PmxError)        # row distance 264
    refused(lambda: pmx.fp8_load(q, s, 100))
    refused(lambda: pmx.fp8_load(q.view(torch.uint8), s))
    refused(lambda: pmx.fp8_load(q, s.int()))
    refused(lambda: pmx.fp8_load(q, s, 256, dtype=torch.float16))
    refused(lambda: pmx.fp8_load(q, s, 256, out=torch.empty(4, 255, device="cuda")))
    refused(lambda: pmx.silu_checkpoint(x[:, :255], gated=True))
    refused(lambda: pmx.silu_checkpoint(x, out=x), pmx.PmxError)
    refused(lambda: pmx.silu_checkpoint_grad(x, q, s, gated=True))
    refused(lambda: pmx.silu_checkpoint_grad(x[:, :100], q, s))
    refused(lambda: pmx.silu_checkpoint_grad(x, q, s, again=False, act=x))
    refused(lambda: pmx.silu_checkpoint_grad(x, q, s, out=x), pmx.PmxError)
    refused(lambda: pmx.fp8_store_weight(x.half()))
    refused(lambda: pmx.fp8_store_weight(x, values=torch.empty(1, 4, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)))
