"""Layer norm of rows whose mean is large beside their spread, and of rows of equal values.

Tolerances (u = 2^-24).  A first mean, of sums through at most 45 additions, is off by e <= E = 46 u max|x|; the
second pass takes the deviations d from it, |d| <= D = |x - m| + E, each rounded once, and their sum, off by 45 u
sum D, which corrects the mean and the variance.  So
  x - m is off by dx = 3 u D + 48 u mean D,
  the variance by at most 150 u (variance + E^2), r by (80 (1 + E^2 / (variance + eps)) + 6) u relative,
  and the mean that the gradient takes, one fp32 number, by dm = u |m| + 49 u mean D.
Equal values: the first mean is off by the same few (up to 31) ulps from all of them, so d is exact, its sum and its
squares' sum are whole numbers below 2^24 of an ulp and of its square, and what is left is 0."""
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


COLS = [33, 100, 300, 1000, 1001, 1024, 2047, 4099, 8193, 16384]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_equal_values(env, cols, dt):
    torch, pmx = env
    values = (3.3, 12345.678, -0.1, 1e-3, 765432.1)
    x = torch.tensor(values).to(getattr(torch, dt))[:, None].expand(-1, cols).contiguous().cuda()
    y, stats = pmx.layer_norm(x)
    assert torch.equal(stats[:, 0], x[:, 0].float())
    assert bool((y == 0).all())
    assert bool((stats[:, 1].double() * 1e-5 ** 0.5 - 1).abs().max() <= 8 * U)  # eps itself is rounded to fp32
    b = torch.randn(cols, device="cuda")
    y, _ = pmx.layer_norm(x, None, b)
    assert torch.equal(y, b.to(x.dtype).expand_as(y))
    y, _ = pmx.layer_norm(x, eps=0.0)
    assert bool(y.isnan().all())
    gx, gw, _ = pmx.layer_norm_grad(torch.randn_like(x), x, stats)
    assert bool((gw == 0).all()) and bool(gx.isfinite().all())


@pytest.mark.parametrize("cols", COLS)
def test_mean_large_beside_spread(env, cols):
    torch, pmx = env
    print("layer norm, large mean", cols, flush=True)
    g = torch.Generator().manual_seed(cols)
    means = torch.tensor([12345.678, 12345.678, 1e6, -3.3, 765432.1, 1e-3])[:, None]
    spread = torch.tensor([0.5, 0.02, 3.0, 1e-4, 1.0, 1e-6])[:, None]
    x = means + spread * torch.randn(6, cols, generator=g)
    dy = torch.randn(6, cols, generator=g)
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    b = torch.randn(cols, generator=g)
    for eps in (1e-5, 1e-12):
        x64, w64 = x.double(), w.double()
        m = x64.mean(1, keepdim=True)
        v = ((x64 - m) ** 2).mean(1, keepdim=True)
        r = 1 / torch.sqrt(v + eps)
        h = (x64 - m) * r
        E = 46 * U * x64.abs().amax(1, keepdim=True)
        D = (x64 - m).abs() + E
        er = (80 * (1 + E ** 2 / (v + eps)) + 6) * U
        y, stats = pmx.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=eps)
        dh = r * (3 * U * D + 48 * U * D.mean(1, keepdim=True)) + h.abs() * er
        want = h * w64 + b.double()
        tol = dh * w64.abs() + 3 * U * ((h * w64).abs() + b.double().abs()) + U * want.abs()
        err = (y.double().cpu() - want).abs()
        assert bool((err <= tol).all()), (eps, (err / tol).amax(1).tolist(), err.amax(1).tolist())
        s = stats.double().cpu()
        dm = 1.01 * U * m.abs() + 49 * U * D.mean(1, keepdim=True)
        assert bool(((s[:, :1] - m).abs() <= dm).all()) and bool(((s[:, 1:] - r).abs() <= er * r).all())
        # the gradients: h as above, but from the rounded mean
        gx, gw, gb = (t.double().cpu() for t in pmx.layer_norm_grad(dy.cuda(), x.cuda(), stats, w.cuda()))
        dh = r * (dm + 2 * U * D) + h.abs() * (er + 2 * U)
        q = dy.double() * w64
        m0, m1 = q.mean(1, keepdim=True), (q * h).mean(1, keepdim=True)
        dx = r * (q - m0 - h * m1)
        e1 = (q.abs() * (dh + 48 * U * h.abs())).mean(1, keepdim=True)
        tol = r * (4 * U * q.abs() + 48 * U * q.abs().mean(1, keepdim=True) + dh * m1.abs() + (h.abs() + dh) * e1
                   + 3 * U * (h * m1).abs()) + dx.abs() * (er + 4 * U)
        assert bool(((gx - dx).abs() <= tol).all()), (eps, ((gx - dx).abs() / tol).amax(1).tolist())
        tw = (dy.double().abs() * dh).sum(0) + 60 * U * (dy.double() * h).abs().sum(0)
        assert bool(((gw - (dy.double() * h).sum(0)).abs() <= tw).all())
        assert bool(((gb - dy.double().sum(0)).abs() <= 60 * U * dy.double().abs().sum(0)).all())
