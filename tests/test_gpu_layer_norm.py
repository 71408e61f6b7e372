"""Layer norm and its gradients against fp64.

Tolerances (u = 2^-24, one fp32 rounding).  A sum over a row passes through at
most 32 additions in a lane and 12 across lanes and waves: the mean is off by at
most 45 u mean|x|, so x - m by dm = 46 u max|x|.  The variance's relative error
is at most 2 (46 u) + 45 u from its sum and, squared, what dm does; with its root
and reciprocal r is off by at most 100 u + dm r relative.  h = (x - m) r is off by
dh = r dm + |h| (102 u + r dm).  Results round once more, by half a step of their
type."""
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


def _half(torch, t):
    return torch.finfo(t).eps / 2


def _data(torch, rows, cols, dt, seed=0, mean=0.3):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * (0.2 + torch.rand(rows, 1, generator=g)) + mean
    return x.to(dt), torch.randn(rows, cols, generator=g).to(dt), (1 + 0.3 * torch.randn(cols, generator=g)), \
        torch.randn(cols, generator=g)


def _ref(torch, x, w, b, eps):
    x = x.double()
    m = x.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + eps)
    h = (x - m) * r
    dm = 46 * U * x.abs().amax(1, keepdim=True)
    dh = r * dm + h.abs() * (102 * U + r * dm)
    return m, r, h, dm, dh, h * w + b


def _ref_grad(torch, dy, r, h, dm, dh, w):
    dy = dy.double()
    g = dy * w
    c = h.shape[1]
    m0, m1 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = r * (g - m0 - h * m1)
    # g rounds once, the two means' sums 46 times, h as above
    e1 = (g.abs() * (dh + 48 * U * h.abs())).mean(1, keepdim=True)
    tol = r * (4 * U * g.abs() + 48 * U * g.abs().mean(1, keepdim=True) + dh * m1.abs() + (h.abs() + dh) * e1
               + 3 * U * (h * m1).abs()) + dx.abs() * (104 * U + r * dm)
    # rows of a thread, the block's teams, the blocks: at most 200 additions here
    dw, db = (dy * h).sum(0), dy.sum(0)
    tw = (dy.abs() * dh).sum(0) + 202 * U * (dy * h).abs().sum(0)
    return dx, tol, dw, tw, db, 200 * U * dy.abs().sum(0)


def _close(torch, got, want, tol, what):
    got, want = got.double().cpu(), want
    bad = ~((got - want).abs() <= tol + _half(torch, torch.float32) * want.abs())
    assert not bool(bad.any()), (what, int(bad.sum()), float((got - want).abs().max()))


SIZES = [(1, 1), (1, 7), (3, 64), (17, 500), (64, 511), (65, 512), (40, 513), (33, 1001), (9, 1024), (5, 1025), (37, 2047),
         (8, 4096), (21, 4099), (6, 8192), (3, 8193), (4, 16384), (2, 16381), (700, 129), (2500, 40), (50, 100), (1100, 2100), (600, 8200),
         (300, 16384)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_forward_and_gradients(env, rows, cols, dt):
    torch, pmx = env
    print("layer norm", rows, cols, dt, flush=True)
    dt = getattr(torch, dt)
    x, dy, w, b = _data(torch, rows, cols, dt, rows + cols)
    w, b = w.to(dt), b.to(dt)
    m, r, h, dm, dh, y = _ref(torch, x, w.double(), b.double(), 1e-5)
    got, stats = pmx.layer_norm(x.cuda(), w.cuda(), b.cuda())
    tol = dh * w.double().abs() + 3 * U * ((h * w.double()).abs() + b.double().abs())
    _close(torch, got, y, tol + _half(torch, dt) * (y.abs() + tol), "y")
    _close(torch, stats[:, :1], m, dm, "mean")
    _close(torch, stats[:, 1:], r, r * (102 * U + r * dm), "r")
    dx, tx, dw, tw, db, tb = _ref_grad(torch, dy, r, h, dm, dh, w.double())
    gx, gw, gb = pmx.layer_norm_grad(dy.cuda(), x.cuda(), stats, w.cuda())
    _close(torch, gx, dx, tx + _half(torch, dt) * (dx.abs() + tx), "dx")
    _close(torch, gw, dw, tw, "dw")
    _close(torch, gb, db, tb, "db")
    again = pmx.layer_norm_grad(dy.cuda(), x.cuda(), stats, w.cuda())
    assert all(torch.equal(p, q) for p, q in zip((gx, gw, gb), again))


def test_parameter_forms(env):
    torch, pmx = env
    x, dy, w, b = _data(torch, 50, 700, torch.bfloat16, 3)
    X, DY, W, B = x.cuda(), dy.cuda(), w.cuda(), b.cuda()  # fp32 parameters of bf16 rows
    one, zero = torch.ones_like(w), torch.zeros_like(b)
    for ww, bb in ((w, b), (w, zero), (one, b), (one, zero)):
        m, r, h, dm, dh, y = _ref(torch, x, ww.double(), bb.double(), 1e-5)
        got, stats = pmx.layer_norm(X, W if ww is w else None, B if bb is b else None)
        tol = dh * ww.double().abs() + 3 * U * (h.abs() * ww.double().abs() + bb.double().abs())
        _close(torch, got, y, tol + _half(torch, torch.bfloat16) * (y.abs() + tol), "y")
        dx, tx, dw, tw, db, tb = _ref_grad(torch, dy, r, h, dm, dh, ww.double())
        gx, gw, gb = pmx.layer_norm_grad(DY, X, stats, W if ww is w else None)
        _close(torch, gx, dx, tx + _half(torch, torch.bfloat16) * (dx.abs() + tx), "dx")
        _close(torch, gw, dw, tw, "dw")
    only, n1, n2 = pmx.layer_norm_grad(DY, X, stats, None, params=False)
    assert n1 is None and n2 is None and torch.equal(only, gx)
    # added to what is there; in dY's place
    dw0, db0 = torch.full((700,), 2.0, device="cuda"), torch.full((700,), -1.0, device="cuda")
    buf = DY.clone()
    g2, aw, ab = pmx.layer_norm_grad(buf, X, stats, None, out=buf, dweight=dw0, dbias=db0, accumulate=True)
    assert g2 is buf and torch.equal(buf, gx) and torch.equal(aw, gw + 2.0) and torch.equal(ab, gb - 1.0)


def test_strides_and_unaligned(env):
    torch, pmx = env
    for dt in (torch.bfloat16, torch.float32):
        big = torch.randn(40, 1200, device="cuda").to(dt)
        x, dy = big[3:30, 1:518], big[10:37, 600:1117]
        out = torch.full((27, 700), 7.0, device="cuda", dtype=dt)
        y, stats = pmx.layer_norm(x, out=out[:, 5:522])
        want, st = pmx.layer_norm(x.contiguous())
        assert torch.equal(y, want) and torch.equal(stats, st)
        assert bool((out[:, :5] == 7).all()) and bool((out[:, 522:] == 7).all())
        g = pmx.layer_norm_grad(dy, x, stats, out=out[:, 100:617])
        g2 = pmx.layer_norm_grad(dy.contiguous(), x.contiguous(), stats)
        assert all(torch.equal(a, b) for a, b in zip(g, g2))


def test_large_mean_and_extremes(env):
    torch, pmx = env
    # a mean of 1000 standard deviations: E x^2 - m^2 would keep no digit of it
    x = (torch.randn(8, 1024, generator=torch.Generator().manual_seed(1)) + 1000).float()
    m, r, h, dm, dh, y = _ref(torch, x, torch.ones(1024).double(), torch.zeros(1024).double(), 1e-5)
    got, _ = pmx.layer_norm(x.cuda())
    _close(torch, got, y, dh + 3 * U * h.abs(), "y")
    flat = torch.full((4, 300), 2.5, device="cuda")
    y, stats = pmx.layer_norm(flat)
    assert bool((y == 0).all()) and bool((stats[:, 0] == 2.5).all())
    bad = flat.clone()
    bad[1, 7], bad[2, 0] = float("inf"), float("nan")
    y, _ = pmx.layer_norm(bad)
    assert bool(y[1].isnan().all()) and bool(y[2].isnan().all()) and bool((y[0] == 0).all()) and bool((y[3] == 0).all())


def test_differences(env):
    """The gradients against central differences of the fp64 formula along one direction: the difference's own
    error is of the order step^2 = 1e-8, the kernel's of 1e-6 of the gradient's size."""
    torch, pmx = env
    x, dy, w, b = _data(torch, 12, 130, torch.float32, 5)
    _, stats = pmx.layer_norm(x.cuda(), w.cuda(), b.cuda())
    gx, gw, gb = (t.double().cpu() for t in pmx.layer_norm_grad(dy.cuda(), x.cuda(), stats, w.cuda()))
    g = torch.Generator().manual_seed(6)
    vx, vw, vb = (torch.randn(t.shape, generator=g, dtype=torch.float64) for t in (x, w, b))
    step = 1e-4

    def value(s):
        return (dy.double() * _ref(torch, x.double() + s * vx, w.double() + s * vw, b.double() + s * vb, 1e-5)[5]).sum()

    want = (value(step) - value(-step)) / (2 * step)
    got = (gx * vx).sum() + (gw * vw).sum() + (gb * vb).sum()
    size = gx.norm() * vx.norm() + gw.norm() * vw.norm() + gb.norm() * vb.norm()
    assert abs(float(got - want)) <= 1e-6 * float(size)


def test_no_rows(env):
    torch, pmx = env
    x = torch.empty(0, 300, device="cuda")
    y, stats = pmx.layer_norm(x)
    assert y.shape == (0, 300) and stats.shape == (0, 2)
    _, gw, gb = pmx.layer_norm_grad(x, x, stats)
    assert bool((gw == 0).all()) and bool((gb == 0).all())


def test_many_rows_and_streams(env):
    torch, pmx = env
    x = torch.randn(40000, 96, device="cuda")
    dy = torch.randn(40000, 96, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, stats = pmx.layer_norm(x)
        dx, dw, db = pmx.layer_norm_grad(dy, x, stats)
    s.synchronize()
    h = (x.double() - stats[:, :1]) * stats[:, 1:]
    # 40000 rows: at most 300 additions in a row of them
    assert bool(((dw - (dy.double() * h).sum(0)).abs() <= 400 * U * (dy.double() * h).abs().sum(0)).all())
    assert bool(((db - dy.double().sum(0)).abs() <= 400 * U * dy.double().abs().sum(0)).all())


def test_refusals(env):
    torch, pmx = env
    x = torch.randn(4, 64, device="cuda")
    _, stats = pmx.layer_norm(x)
    w = torch.ones(64, device="cuda")

    def refused(f, kind=(ValueError, TypeError)):
        with pytest.raises(kind):
            f()

    refused(lambda: pmx.layer_norm(x.half()))
    refused(lambda: pmx.layer_norm(x.cpu()))
    refused(lambda: pmx.layer_norm(x.t()))
    refused(lambda: pmx.layer_norm(x, w[:63]))
    refused(lambda: pmx.layer_norm(x, w, w.bfloat16()))
    refused(lambda: pmx.layer_norm(x, out=torch.empty(4, 63, device="cuda")))
    refused(lambda: pmx.layer_norm(x, eps=-1.0), pmx.PmxError)
    refused(lambda: pmx.layer_norm(x, eps=float("nan")), pmx.PmxError)
    refused(lambda: pmx.layer_norm(x, out=x), pmx.PmxError)
    refused(lambda: pmx.layer_norm(torch.empty(2, pmx.MAX_NORM_COLS + 1, device="cuda")), pmx.PmxError)
    refused(lambda: pmx.layer_norm_grad(x, x.bfloat16(), stats))
    refused(lambda: pmx.layer_norm_grad(x, x, stats[:3]))
    refused(lambda: pmx.layer_norm_grad(x, x, stats, accumulate=True))
    refused(lambda: pmx.layer_norm_grad(x, x, stats, dweight=torch.empty(64, device="cuda", dtype=torch.bfloat16)))
    dy = x.clone()
    refused(lambda: pmx.layer_norm_grad(dy, x, stats, out=x), pmx.PmxError)
    big = torch.empty(65 * 64, device="cuda")
    refused(lambda: pmx.layer_norm_grad(big[:256].view(4, 64), x, stats, out=big[64:320].view(4, 64)), pmx.PmxError)
