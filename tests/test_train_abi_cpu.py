"""Host side of the training-step calls that needs no GPU: limits, workspace
sizes, and refusals that come before anything touches a device."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pmx():
    from preconditioned_optimizer_matrix_amd import pmx
    return pmx


def _size(pmx, name, *args):
    sz = ctypes.c_size_t(1 << 60)
    code = getattr(pmx.lib, name)(*args, ctypes.byref(sz))
    return code, sz.value


def test_constants_and_struct_match_the_header(pmx):
    src = open(os.path.join(ROOT, "include", "pmx.h")).read()
    for name in ("MAX_GROUPS", "MAX_TOP", "MAX_VOCAB", "MAX_TOKENS"):
        assert int(re.search(r"#define PMX_%s (\d+)" % name, src).group(1)) == getattr(pmx, name)
    body = src[:src.index("} pmx_distill_problem;")]
    body = re.sub(r"/\*.*?\*/", "", body[body.rindex("typedef struct {") + 16:], flags=re.S)
    names = re.findall(r"(\w+)\s*[,;]", body)
    assert names == [f[0] for f in pmx.DistillProblem._fields_]


def test_grouped_workspace_sizes(pmx):
    f = "pmx_grouped_product_workspace_size"
    assert _size(pmx, f, 0, 64, 64, 4, pmx.F32) == (pmx.OK, 0)
    assert _size(pmx, f, 32768, 1024, 4096, 32, pmx.BF16) == (pmx.OK, 0)  # tiles enough: nothing is split
    code, n = _size(pmx, f, 32, 8192, 128, 1, pmx.BF16)  # one tile: split
    assert code == pmx.OK and n > 0 and n % (32 * 128 * 4) == 0
    for bad in ((-1, 64, 64, 4), (8, 0, 64, 4), (8, 64, 0, 4), (8, 64, 64, 0), (8, 64, 64, pmx.MAX_GROUPS + 1),
                (8, (1 << 20) + 1, 64, 4), (8, 64, (1 << 20) + 1, 4)):
        for g in (f, "pmx_grouped_outer_workspace_size"):
            assert _size(pmx, g, *bad, pmx.F32)[0] == pmx.ERR_INVALID_VALUE, bad
    assert _size(pmx, f, 8, 64, 64, 4, 7)[0] == pmx.ERR_INVALID_VALUE
    assert pmx.lib.pmx_grouped_product_workspace_size(8, 64, 64, 4, pmx.F32, None) == pmx.ERR_INVALID_VALUE
    code, n = _size(pmx, "pmx_grouped_outer_workspace_size", 20000, 64, 64, 1, pmx.BF16)
    assert code == pmx.OK and n > 0 and n % (64 * 64 * 4) == 0
    assert _size(pmx, "pmx_grouped_outer_workspace_size", 32768, 4096, 1024, 32, pmx.BF16) == (pmx.OK, 0)


def test_large_tiles_are_never_split(pmx):
    """The bf16 256 x 256 tiles are taken from 256 of them on; their kernels write whole results, so no workspace."""
    f = "pmx_grouped_outer_workspace_size"
    for rows, m, n, groups in ((1024, 4096, 4096, 1), (16384, 1024, 1024, 16), (8192, 2048, 1024, 8), (4096, 2048, 2048, 4),
                               (65536, 4096, 4096, 1), (5000, 4096, 4352, 1), (5000, 257, 256, 128), (65536, 256, 256, 257)):
        assert _size(pmx, f, rows, m, n, groups, pmx.BF16) == (pmx.OK, 0), (rows, m, n, groups)
    # 255 of them: smaller tiles
    assert _size(pmx, f, 65536, 256, 256, 255, pmx.BF16)[0] == pmx.OK
    # products: (rows / 256) * columns of tiles from 256 on
    for rows, k, n, groups in ((65536, 4096, 256, 1), (16384, 1 << 20, 1024, 4), (65536, 4096, 256, 256)):
        assert _size(pmx, "pmx_grouped_product_workspace_size", rows, k, n, groups, pmx.BF16) == (pmx.OK, 0)


def test_embedding_workspace_sizes(pmx):
    f = "pmx_embedding_grad_workspace_size"
    few, many = _size(pmx, f, 200, 1000, 64), _size(pmx, f, 20000, 1000, 64)
    assert few == (pmx.OK, 256)
    # (key, position) pairs twice, two partial rows a chunk of at most 32 tokens
    assert many[0] == pmx.OK and many[1] >= 2 * 20000 * 8 + 2 * (20000 // 32) * 64 * 4
    assert _size(pmx, f, 0, 1, 1)[0] == pmx.OK
    for bad in ((-1, 10, 8), (pmx.MAX_TOKENS + 1, 10, 8), (5, 0, 8), (5, pmx.MAX_VOCAB + 1, 8), (5, 10, 0)):
        assert _size(pmx, f, *bad)[0] == pmx.ERR_INVALID_VALUE, bad


def test_distill_problem_is_checked(pmx):
    def size(**kw):
        q = pmx.DistillProblem(1, pmx.BF16, 8, 1000, 4, 4096, 1000, 8192, 4, 16384, 4, None, None, pmx.I32, 0, pmx.BF16,
                               1.0, 1.0, 0)
        for k, v in kw.items():
            setattr(q, k, v)
        sz = ctypes.c_size_t()
        return pmx.lib.pmx_distill_workspace_size(ctypes.byref(q), ctypes.byref(sz))

    assert size() == pmx.OK
    assert size(struct_version=2) == pmx.ERR_INVALID_VALUE
    assert size(reserved=1) == pmx.ERR_INVALID_VALUE
    assert size(rows=-1) == pmx.ERR_INVALID_VALUE
    assert size(vocab=0) == pmx.ERR_INVALID_VALUE
    assert size(vocab=pmx.MAX_VOCAB + 1) == pmx.ERR_INVALID_VALUE
    assert size(top=pmx.MAX_TOP + 1) == pmx.ERR_INVALID_VALUE
    assert pmx.lib.pmx_distill_workspace_size(None, None) == pmx.ERR_INVALID_VALUE


def test_distill_rows_cut_over_blocks(pmx):
    """Only few long rows are: their partial sums, the listed logits; one counter for long rows otherwise."""
    def size(rows, vocab, dtype, top=20):
        q = pmx.DistillProblem(1, dtype, rows, vocab, top, 4096, vocab, 8192, top, 16384, top, None, None, pmx.I32, 0, pmx.F32,
                               1.0, 1.0, 0)
        sz = ctypes.c_size_t()
        assert pmx.lib.pmx_distill_workspace_size(ctypes.byref(q), ctypes.byref(sz)) == pmx.OK
        return sz.value

    for rows in (1, 8, 32):
        for vocab, dtype in ((128000, pmx.BF16), (66000, pmx.BF16), (50000, pmx.F32), (262144, pmx.F32)):
            n = size(rows, vocab, dtype)
            assert n >= rows * (2 * 3 + 21) * 4 and n % (rows * 4) == 0, (rows, vocab, dtype)
        assert size(rows, 32000, pmx.BF16) == size(rows, 65536, pmx.BF16) == size(rows, 32000, pmx.F32) == 0
    assert size(64, 32000, pmx.BF16) == size(128, 17000, pmx.BF16) == size(64, 200000, pmx.BF16) == 0
    assert size(64, 128000, pmx.BF16) == size(33, 50000, pmx.F32) == 4


def test_no_handle_no_call(pmx):
    L, i = pmx.lib, pmx.ERR_INVALID_VALUE
    assert L.pmx_grouped_product(None, 256, pmx.F32, 8, 8, 8, 512, 8, 8, 64, 0, 256, pmx.I32, 1, 4096, pmx.F32, 8, None, 0, None) == i
    assert L.pmx_grouped_outer(None, 256, pmx.F32, 8, 8, 8, 512, 8, 8, 256, pmx.I32, 1, 4096, pmx.F32, 8, 64, 0, None, 0, None) == i
    assert L.pmx_embedding(None, 256, pmx.F32, 8, 8, 8, 512, pmx.I32, 4, 1.0, 4096, 8, None) == i
    assert L.pmx_embedding_grad(None, 256, pmx.F32, 8, 8, 8, 512, pmx.I32, 9, 1.0, -1, 4096, pmx.F32, 8, 0, None, 0, None) == i
    q = pmx.DistillProblem()
    assert L.pmx_distill_loss(None, ctypes.byref(q), 256, 512, 1024, None, 0, None, 0, None) == i
    assert L.pmx_distill_grad(None, ctypes.byref(q), 256, None, 512, 8, None) == i


@pytest.mark.skipif("SAN_CHILD" in os.environ, reason="torch is not for the sanitized child")
def test_workspace_of_another_device_or_layout(pmx):
    import torch
    w = torch.empty(1024, dtype=torch.uint8)
    assert pmx._ws_for(1000, w, w.device) == (w.data_ptr(), 1024)
    assert pmx._ws_for(0, None, w.device) == (None, 0)
    for bad, dev in ((w, torch.device("cuda:0")), (w[:1].expand(1024), w.device), (w[::2], w.device)):
        for need in (0, 500):
            with pytest.raises(ValueError):
                pmx._ws_for(need, bad, dev)


@pytest.mark.skipif("SAN_CHILD" in os.environ, reason="this is the child")
def test_clean_under_host_sanitizers():
    from preconditioned_optimizer_matrix_amd import build
    if not os.path.exists(build.SAN_LIB):
        build.build_sanitized(verbose=False)
    env = dict(os.environ, PMX_LIBRARY=build.SAN_LIB, LD_PRELOAD=build.asan_runtime(), SAN_CHILD="1",
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", os.path.abspath(__file__)],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and " passed" in out, out[-4000:]
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
