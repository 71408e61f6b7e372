"""What the sums of 8-bit products keep.

fp32 results, and bf16 results of few rows a group: exact products, added in fp32, (66 + k / 128) 2^-24 of the sum of
magnitudes.  bf16 results through tiles: of eight neighbouring products (k = 8 i .. 8 i + 7) each loses what lies below
2^-13 of the largest of their powers of two, those of the operands multiplied, an operand below 2^-6 counting as 2^-6 and
a zero product not: less than 2^-13 of that product, which itself loses nothing where its operands are normal numbers.
Together less than 7 2^-13 (8 2^-13 with smaller operands) of the eights' largest, added up, and fp32's share."""
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


def _ones(torch, q):
    return torch.ones(q.shape, device="cuda").to(torch.float8_e4m3fn)


@pytest.mark.parametrize("kind,rows,n,k,out", _both([f for f in FORMS if not f[0].startswith("stream")]))
def test_operands_below_the_normal_numbers(env, kind, rows, n, k, out):  # noqa: F811
    """+p and -p of an operand 2^ex and one of 2^8, and 2^-b p beside them: kept where it is
    at least 2^-13 of 2^8 max(2^ex, 2^-6)."""
    torch, pmx = env
    for ex in (-4, -6, -7, -8, -9):
        for b in range(4, 18):
            if ex + 8 - b - ex < -9:
                continue
            for swap in (False, True):
                u, v = torch.zeros(k, device="cuda"), torch.zeros(k, device="cuda")
                u[64], v[100] = 256.0, 256.0  # the blocks' powers
                u[0], u[1], u[2] = 2.0 ** ex, 2.0 ** ex, 2.0 ** ex
                v[0], v[1], v[2] = 256.0, -256.0, 2.0 ** (8 - b)
                x, w = (v, u) if swap else (u, v)
                y = pmx.fp8_product(*pmx.fp8_store(x.expand(rows, k).contiguous()),
                                    *pmx.fp8_store_weight(w.expand(1, n, k).contiguous()), out_dtype=getattr(torch, out))
                want = 2.0 ** (ex + 8 - b)
                if out == "float32" or b <= 13 + min(ex + 6, 0):
                    assert bool((y == want).all()), (ex, b, swap, float(y[0, 0]), want)
                else:
                    assert bool(((y.double() - want).abs() <= want).all())


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


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("kind,rows,n,k,out", _both(FORMS + [("64", 300, 515, 1400), ("128", 3000, 1300, 384)]))
def test_bound(env, kind, rows, n, k, out, small):  # noqa: F811
    """Products of very different sizes, some of them cancelling."""
    torch, pmx = env
    print("fp8 sums, bound", kind, rows, n, k, out, flush=True)
    assert form(rows, k, n, 1, out, units(torch)) == kind
    g = torch.Generator(device="cuda").manual_seed(rows + n)
    x = torch.randn(rows, k, generator=g, device="cuda") * torch.exp2(torch.randint(-7, 8, (rows, k), generator=g, device="cuda").float())
    w = torch.randn(1, n, k, generator=g, device="cuda") * torch.exp2(torch.randint(-7, 8, (1, n, k), generator=g, device="cuda").float())
    if small:  # the first value of a block holds its power, the others lie around e4m3's least normal number or below
        x[:, 0::128], w[:, :, 0::128] = 256.0, 256.0
        x = torch.where(x.abs() >= 256, x, x * 2.0 ** -9)
        w[:, :, 64:] *= 2.0 ** -9
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
        # the operands' powers of two before the scales, which are powers themselves and leave 2^-6 in place
        ea, eb = (torch.exp2(torch.floor(torch.log2(q.float().double().abs().clamp(min=2.0 ** -6)))) for q in (xq[r], wq[0][c]))
        fa, fb = ea * _rows_value(torch, _ones(torch, xq[r]), xs[r]), eb * _weight_value(torch, _ones(torch, wq[0]), ws[0])[c]
        top = (fa[:, None, :] * fb[None, :, :] * (p != 0)).view(p.shape[0], p.shape[1], -1, 8).amax(3)
        tol = tol + 8 * 2.0 ** -13 * top.sum(2)
    err = (y[r][:, c] - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
