"""What the sums of 8-bit products keep.

fp32 results, and bf16 results of few rows a group: exact products, added in fp32, (66 + k / 128) 2^-24 of the sum of
magnitudes.  bf16 results through tiles: of eight neighbouring products (k = 8 i .. 8 i + 7) each loses what lies below
2^-13 of the power of two of the largest of them, less than 2^-13 of that product, which itself loses nothing: together
less than 7 2^-13 of the eights' largest products, added up, and fp32's share."""
import pytest

from test_gpu_fp8 import _rows_value, _weight_value, env  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def form(rows, k, n, groups, out, units):
    """The kernel that pmx_fp8.hip's rules take (`choose` and `launch` there)."""
    avg, wide = rows // groups, (rows // 128 + groups) * -(-n // 128) >= units
    if avg <= 2 or (avg <= 16 and (not wide or out == "float32")):
        return "stream, own columns" if min(groups, rows) * -(-n // 16) >= 8 * units else "stream, shared"
    if out == "bfloat16" and avg >= 256 and n >= 256 and k >= 512 and rows // 256 * -(-n // 256) >= units:
        return "256"
    return "128" if wide and not (out == "float32" and avg <= 64) else "64"


def units(torch):
    return torch.cuda.get_device_properties(0).multi_processor_count


FORMS = [("stream, shared", 16, 64, 128), ("stream, own columns", 2, 32800, 128), ("64", 600, 600, 128), ("128", 3000, 2100, 128),
         ("256", 9000, 2304, 512)]


def _both(forms):
    return [f + (out,) for f in forms for out in ("bfloat16", "float32") if out == "bfloat16" or f[0] != "256"]


@pytest.mark.parametrize("kind,rows,n,k,out", _both(FORMS))
def test_small_products_beside_large_ones_that_cancel(env, kind, rows, n, k, out):  # noqa: F811
    """+2^16 and -2^16, and `count` products of 2^(16 - b) among the same eight and behind them."""
    torch, pmx = env
    print("fp8 sums", kind, rows, n, k, out, flush=True)
    assert form(rows, k, n, 1, out, units(torch)) == kind
    cuts = out == "bfloat16" and not kind.startswith("stream")
    for first, second, at, count in ((0, 1, 2, 1), (0, 1, 2, 6), (3, 7, 4, 3), (8, 15, 9, 6), (0, 100, 101, 3), (64, 71, 65, 1)):
        for b in (1, 5, 10, 12, 13, 14, 15, 16):
            for sign in (1.0, -1.0):
                ex = min(8, max(-9, (16 - b) // 2))
                x = torch.zeros(rows, k, device="cuda")
                w = torch.zeros(1, n, k, device="cuda")
                x[:, first], x[:, second] = 256.0, 256.0
                w[:, :, first], w[:, :, second] = 256.0, -256.0
                x[:, at:at + count], w[:, :, at:at + count] = sign * 2.0 ** ex, 2.0 ** (16 - b - ex)
                y = pmx.fp8_product(*pmx.fp8_store(x), *pmx.fp8_store_weight(w), out_dtype=getattr(torch, out)).double()
                want = sign * count * 2.0 ** (16 - b)
                if cuts and b > 13:  # cut off, or not: as documented
                    assert bool(((y - want).abs() <= abs(want)).all()), (b, sign)
                else:
                    tol = 0.0 if cuts else 67 * U * (2.0 ** 17 + abs(want)) + (U if out == "float32" else 2.0 ** -8) * abs(want)
                    assert bool(((y - want).abs() <= tol).all()), (b, sign, first, count, float(y[0, 0]), want)


@pytest.mark.parametrize("kind,rows,n,k,out", _both(FORMS + [("64", 300, 515, 1400), ("128", 3000, 1300, 384)]))
def test_bound(env, kind, rows, n, k, out):  # noqa: F811
    """Products of very different sizes, half of them cancelling."""
    torch, pmx = env
    print("fp8 sums, bound", kind, rows, n, k, out, flush=True)
    assert form(rows, k, n, 1, out, units(torch)) == kind
    g = torch.Generator(device="cuda").manual_seed(rows + n)
    x = torch.randn(rows, k, generator=g, device="cuda") * torch.exp2(torch.randint(-7, 8, (rows, k), generator=g, device="cuda").float())
    w = torch.randn(1, n, k, generator=g, device="cuda") * torch.exp2(torch.randint(-7, 8, (1, n, k), generator=g, device="cuda").float())
    x[:, 1::16], w[:, :, 1::16] = x[:, 0:k - 1:16][:, : x[:, 1::16].shape[1]], -w[:, :, 0:k - 1:16][:, :, : x[:, 1::16].shape[1]]
    xq, xs = pmx.fp8_store(x)
    wq, ws = pmx.fp8_store_weight(w)
    y = pmx.fp8_product(xq, xs, wq, ws, out_dtype=getattr(torch, out)).double()
    a, b = _rows_value(torch, xq, xs), _weight_value(torch, wq[0], ws[0])
    r = torch.randperm(rows, generator=g, device="cuda")[:64]
    c = torch.randperm(n, generator=g, device="cuda")[:64]
    p = a[r][:, None, :] * b[c][None, :, :]
    want, size = p.sum(2), p.abs().sum(2)
    tol = (66 + a.shape[1] / 128) * U * size + (U if out == "float32" else 2.0 ** -8) * want.abs()
    if out == "bfloat16" and not kind.startswith("stream"):
        tol = tol + 7 * 2.0 ** -13 * p.abs().view(p.shape[0], p.shape[1], -1, 8).amax(3).sum(2)
    err = (y[r][:, c] - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
