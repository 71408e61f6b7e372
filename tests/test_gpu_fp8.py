"""Products of 8-bit values, grouped by expert, against fp64 of the stored values.

Tolerances.  fp32 results: the values are exact in bf16, whose matrix instructions
add exact products in fp32: a sum over 128 values of k passes through at most 64
additions, its scaling by a power of two is exact, and the k / 128 sums through as
many: (66 + k / 128) 2^-24 of the sum of the products' magnitudes.  bf16 results:
the 8-bit instructions keep fewer bits below a group's largest product; 2^-14 of
the sum of magnitudes is asked for, a sixteenth of what one value's rounding to 8
bits (2^-4 of it) leaves even after 4096 of them have averaged out, and half a
step of the result's rounding, 2^-8."""
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


def _rows_value(torch, q, s):
    v = q.float().double().view(q.shape[0], -1, 128)
    return (v * torch.pow(2.0, s.double() - 127)[:, :, None]).view(q.shape)


def _weight_value(torch, q, s):
    n, k = q.shape
    f = torch.pow(2.0, s.double() - 127).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    return q.float().double() * f


def _check(env, x, w, offsets, out_dtype, itype=None, transposed=False):
    """x rows x k, w groups x n x k (transposed: groups x k x n, contracted over its rows)."""
    torch, pmx = env
    rows = x.shape[0]
    xq, xs = pmx.fp8_store(x)
    wq, ws = pmx.fp8_store_weight(w, transposed=transposed)
    off = None if offsets is None else torch.tensor(offsets, dtype=itype or torch.int32, device="cuda")
    y = pmx.fp8_product(xq, xs, wq, ws, off, out_dtype=out_dtype)
    bounds = [min(max(o, 0), rows) for o in (offsets or [0, rows])]
    for i in range(1, len(bounds)):
        bounds[i] = max(bounds[i], bounds[i - 1])
    n = wq.shape[1]
    want = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(want)
    a = _rows_value(torch, xq, xs)
    for e in range(w.shape[0]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            b = _weight_value(torch, wq[e], ws[e])
            want[lo:hi] = a[lo:hi] @ b.t().contiguous()
            size[lo:hi] = a[lo:hi].abs() @ b.abs().t().contiguous()
    k = xq.shape[1]
    tol = (66 + k / 128) * U * size + U * want.abs() if out_dtype == torch.float32 else 2.0 ** -14 * size + 2.0 ** -8 * want.abs()
    bad = ~((y.double() - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float((y.double() - want).abs().max()), float(want.abs().max()))
    assert torch.equal(y, pmx.fp8_product(xq, xs, wq, ws, off, out_dtype=out_dtype))
    return y


def _offsets(torch, rows, groups, seed):
    g = torch.Generator().manual_seed(seed)
    cuts = torch.sort(torch.randint(0, rows + 1, (groups - 1,), generator=g))[0].tolist() if groups > 1 else []
    return [0] + cuts + [rows]


CASES = [(1, 1, 1, 1), (1, 128, 64, 1), (3, 130, 17, 2), (16, 1024, 512, 8), (17, 500, 1001, 3), (40, 300, 65, 40), (63, 129, 63, 1),
         (130, 257, 129, 2), (200, 1111, 300, 3), (513, 640, 515, 4), (1000, 384, 1024, 2), (1025, 256, 257, 5), (37, 4096, 256, 6),
         (700, 128, 2003, 1), (3000, 515, 260, 7), (5000, 200, 130, 64), (16, 2048, 100, 300), (4500, 300, 1280, 3), (9000, 128, 4096, 2)]


@pytest.mark.parametrize("rows,k,n,groups", CASES)
@pytest.mark.parametrize("out", ["bfloat16", "float32"])
def test_against_fp64(env, rows, k, n, groups, out):
    torch, pmx = env
    print("fp8 product", rows, k, n, groups, out, flush=True)
    g = torch.Generator().manual_seed(rows + k + n)
    # rows and tiles of very different sizes, so that every scale counts
    x = torch.randn(rows, k, generator=g) * torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g).float())
    w = torch.randn(groups, n, k, generator=g) * torch.exp2(torch.randint(-9, 9, (groups, 1, 1), generator=g).float())
    x[:, : k // 2] *= 16.0
    w[:, n // 2:, k // 3:] *= 0.01
    dt = getattr(torch, out)
    _check(env, x.to(dt).cuda(), w.to(dt).cuda(), _offsets(torch, rows, groups, rows) if groups > 1 else None, dt)


@pytest.mark.parametrize("out", ["bfloat16", "float32"])
def test_large_groups(env, out):
    torch, pmx = env
    print("fp8 product large", out, flush=True)
    dt = getattr(torch, out)
    for rows, k, n, cuts in ((6000, 1024, 2048, [0, 100, 100, 2900, 2901, 6000]), (20000, 384, 1536, [0, 7001, 13000, 20000])):
        x = torch.randn(rows, k, device="cuda").to(dt)
        w = torch.randn(len(cuts) - 1, n, k, device="cuda").to(dt)
        _check(env, x, w, cuts, dt)


LARGE = [(8300, 520, 2100, [0, 100, 100, 4500, 4501, 8300], 0), (9000, 1000, 2304, [0, 8999, 9000], 0),
         (9000, 1000, 2304, [0, 8999, 9000], 8), (9000, 600, 2304, [30, 5000, 8000], 3), (66000, 512, 256, None, 0),
         (17000, 1152, 1111, [0, 0, 17000], 0), (30000, 768, 1024, [0] + [300 * i + 7 for i in range(1, 100)] + [30000], 0)]


@pytest.mark.parametrize("case", range(len(LARGE)))
def test_large_tiles(env, case):
    """256 x 256 tiles: contractions of 4 to 9 blocks, uneven and empty groups, columns past the last whole tile, results
    at odd row distances, more than 64 groups."""
    torch, pmx = env
    rows, k, n, cuts, pad = LARGE[case]
    print("fp8 large tiles", LARGE[case][:3], flush=True)
    g = torch.Generator(device="cuda").manual_seed(case)
    x = torch.randn(rows, k, generator=g, device="cuda").bfloat16()
    x *= torch.exp2(torch.randint(-6, 6, (rows, 1), generator=g, device="cuda").float()).bfloat16()
    groups = 1 if cuts is None else len(cuts) - 1
    w = torch.randn(groups, n, k, generator=g, device="cuda").bfloat16()
    w[:, n // 2:, k // 3:] *= 0.01
    y = _check(env, x, w, cuts, torch.bfloat16)
    if pad:
        out = torch.full((rows, n + pad), 3.0, dtype=torch.bfloat16, device="cuda")
        off = torch.tensor(cuts, dtype=torch.int64, device="cuda")
        got = pmx.fp8_product(*pmx.fp8_store(x), *pmx.fp8_store_weight(w), off, out=out[:, :n])
        assert torch.equal(got, y) and bool((out[:, n:] == 3).all())


def test_large_tiles_without_rows(env):
    """No row, or one, in any group where the rows alone ask for 256 x 256 tiles; the rest of the result is zeros."""
    torch, pmx = env
    x, w = torch.randn(9000, 512, device="cuda").bfloat16(), torch.randn(2, 2304, 512, device="cuda").bfloat16()
    for cuts in ([0, 0, 0], [9000, 9000, 9000], [4000, 4000, 4001]):
        y = _check(env, x, w, cuts, torch.bfloat16)
        live = torch.zeros(9000, dtype=torch.bool, device="cuda")
        live[cuts[0]:cuts[-1]] = True
        assert bool((y[~live] == 0).all())


@pytest.mark.parametrize("out", ["bfloat16", "float32"])
def test_offsets(env, out):
    """Empty groups, rows in no group, int64, offsets out of range or order."""
    torch, pmx = env
    dt = getattr(torch, out)
    for rows, n in ((90, 200), (2000, 700)):
        x, w = torch.randn(rows, 260, device="cuda").to(dt), torch.randn(4, n, 260, device="cuda").to(dt)
        for off in ([0, 0, rows, rows, rows], [5, 20, 20, 60, 70], [rows] * 5, [0, 0, 0, 0, 0], [-3, 30, 10, 50, rows + 9]):
            for it in (torch.int32, torch.int64):
                y = _check(env, x, w, off, dt, it)
            if off == [5, 20, 20, 60, 70]:
                assert bool((y[:5] == 0).all()) and bool((y[70:] == 0).all())


def test_input_gradient_takes_the_transposed(env):
    torch, pmx = env
    for dt in (torch.bfloat16, torch.float32):
        dy = torch.randn(300, 384, device="cuda").to(dt)
        w = torch.randn(3, 384, 200, device="cuda").to(dt)
        y = _check(env, dy, w, [0, 100, 130, 300], dt, transposed=True)
        wq, ws = pmx.fp8_store_weight(w)
        tq, ts = pmx.fp8_store_weight(w, transposed=True)
        assert y.shape == (300, 200) and torch.equal(wq.view(torch.uint8)[:, :, :200].transpose(1, 2), tq.view(torch.uint8)[:, :, :384])
        assert torch.equal(ws.transpose(1, 2), ts)


def test_tiny_and_huge_scales(env):
    torch, pmx = env
    x = torch.randn(70, 256, device="cuda")
    w = torch.randn(1, 130, 256, device="cuda")
    for sx, sw in ((2.0 ** -100, 2.0 ** 90), (2.0 ** 60, 2.0 ** 50), (2.0 ** 100, 2.0 ** -120)):
        for dt in (torch.float32, torch.bfloat16):
            _check(env, (x * sx).to(dt), (w * sw).to(dt), None, dt)
    for dt in (torch.float32, torch.bfloat16):
        z = torch.zeros(70, 256, device="cuda", dtype=dt)
        assert bool((_check(env, z, w.to(dt), None, dt) == 0).all())


def test_nan_stays_in_its_row_and_column(env):
    torch, pmx = env
    for dt in (torch.float32, torch.bfloat16):
        for rows in (20, 600):
            x, w = torch.randn(rows, 300, device="cuda").to(dt), torch.randn(1, 140, 300, device="cuda").to(dt)
            x[3, 299], w[0, 77, 5] = float("inf"), float("nan")
            y = pmx.fp8_product(*pmx.fp8_store(x), *pmx.fp8_store_weight(w), out_dtype=dt)
            bad = torch.zeros(rows, 140, dtype=torch.bool, device="cuda")
            bad[3], bad[:, 77] = True, True
            assert torch.equal(y.isnan(), bad)


def test_what_lies_outside_does_not_enter(env):
    """Neighbouring rows, columns and weights full of NaN; the result's neighbours stay."""
    torch, pmx = env
    nan = 0x7F
    for dt in (torch.float32, torch.bfloat16):
        for rows, n, k in ((9, 70, 384), (150, 300, 384), (2300, 700, 384), (16600, 1111, 640)):
            x, w = torch.randn(rows, k, device="cuda"), torch.randn(2, n, k, device="cuda")
            xq, xs = pmx.fp8_store(x)
            wq, ws = pmx.fp8_store_weight(w)
            off = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
            want = pmx.fp8_product(xq, xs, wq, ws, off, out_dtype=dt)
            e4 = torch.float8_e4m3fn
            bx = torch.full((rows + 2, k + 32), nan, dtype=torch.uint8, device="cuda")
            bw = torch.full((2, n + 1, k + 16), nan, dtype=torch.uint8, device="cuda")
            kb = k // 128
            sx = torch.full((rows + 1, kb + 4), 255, dtype=torch.uint8, device="cuda")
            sw = torch.full((2, ws.shape[1] + 1, kb + 2), 255, dtype=torch.uint8, device="cuda")
            bx[1:-1, 16:16 + k], bw[:, :n, :k], sx[:rows, 1:1 + kb], sw[:, :-1, 2:] = xq.view(torch.uint8), wq.view(torch.uint8), xs, ws
            out = torch.full((rows, n + 5), 3.0, dtype=dt, device="cuda")
            got = pmx.fp8_product(bx.view(e4)[1:-1, 16:16 + k], sx[:rows, 1:1 + kb], bw.view(e4)[:, :n, :k], sw[:, :-1, 2:], off,
                                  out=out[:, 2:n + 2])
            assert torch.equal(got, want) and bool((out[:, :2] == 3).all()) and bool((out[:, n + 2:] == 3).all())


def test_one_weight_for_all_groups_and_no_rows(env):
    torch, pmx = env
    x, w = torch.randn(50, 128, device="cuda"), torch.randn(1, 90, 128, device="cuda")
    xq, xs = pmx.fp8_store(x)
    wq, ws = pmx.fp8_store_weight(w)
    off = torch.tensor([0, 10, 50], dtype=torch.int32, device="cuda")
    shared = pmx.fp8_product(xq, xs, wq.expand(2, -1, -1), ws.expand(2, -1, -1), off)
    assert torch.equal(shared, pmx.fp8_product(xq, xs, wq, ws))
    assert pmx.fp8_product(xq[:0], xs[:0], wq, ws).shape == (0, 90)


def test_refusals(env):
    torch, pmx = env
    xq, xs = pmx.fp8_store(torch.randn(20, 256, device="cuda"))
    wq, ws = pmx.fp8_store_weight(torch.randn(2, 30, 256, device="cuda"))
    off = torch.tensor([0, 5, 20], dtype=torch.int32, device="cuda")

    def refused(f, kind=(ValueError, TypeError)):
        with pytest.raises(kind):
            f()

    refused(lambda: pmx.fp8_product(xq, xs, wq, ws))
    refused(lambda: pmx.fp8_product(xq, xs, wq, ws, off[:2]))
    refused(lambda: pmx.fp8_product(xq, xs, wq, ws, off.float()))
    refused(lambda: pmx.fp8_product(xq[:, :128], xs[:, :1], wq, ws, off))
    refused(lambda: pmx.fp8_product(xq, xs, wq, ws[:, :, :1], off))
    refused(lambda: pmx.fp8_product(xq, xs, wq.view(torch.uint8), ws, off))
    refused(lambda: pmx.fp8_product(xq, xs[:, :1], wq, ws, off))
    refused(lambda: pmx.fp8_product(xq, xs, wq, ws, off, out=torch.empty(20, 31, device="cuda")))
    refused(lambda: pmx.fp8_product(xq, xs, wq, ws, off, out_dtype=torch.float16))
    wide = torch.empty(20, 264, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    refused(lambda: pmx.fp8_product(wide[:, :256], xs, wq, ws, off), pmx.PmxError)
    alias = torch.empty(20 * 256, dtype=torch.uint8, device="cuda")
    refused(lambda: pmx.fp8_product(alias.view(torch.float8_e4m3fn).view(20, 256), xs, wq, ws, off,
                                    out=alias[:20 * 30 * 2].view(torch.bfloat16).view(20, 30)), pmx.PmxError)
