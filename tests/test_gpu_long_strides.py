"""Rows, matrices and results beyond 2^31 elements or bytes from a tensor's start: the same bits as packed ones."""
import pytest

from test_gpu_fp8_sums import form, units

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    from preconditioned_optimizer_matrix_amd import pmx
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    return torch, pmx


@pytest.fixture(autouse=True)
def _room():
    import torch
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _far(torch, like, ld):
    """An uninitialised tensor of like's shape whose rows lie `ld` elements apart."""
    rows, cols = like.shape
    size = (rows - 1) * ld + cols
    assert size > 1 << 31
    return torch.empty(size, dtype=like.dtype, device="cuda").as_strided((rows, cols), (ld, 1))


def _spread(torch, t, ld):
    far = _far(torch, t, ld)
    far.copy_(t)
    return far


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_layer_norm(env, dt):
    torch, pmx = env
    x, dy = (torch.randn(5, 1001, device="cuda").to(getattr(torch, dt)) for _ in range(2))
    w = torch.randn(1001, device="cuda")
    ld = (1 << 29) + 8
    fx = _spread(torch, x, ld)
    want, stats = pmx.layer_norm(x, w, w)
    y, st = pmx.layer_norm(fx, w, w, out=_far(torch, x, ld + 3))
    assert torch.equal(y, want) and torch.equal(st, stats)
    del y
    got = pmx.layer_norm_grad(_spread(torch, dy, ld + 1), fx, stats, w, out=_far(torch, x, ld + 5))
    assert all(torch.equal(a, b) for a, b in zip(got, pmx.layer_norm_grad(dy, x, stats, w)))


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("rows,ld", [(5, (1 << 29) + 4), (70, (1 << 25) + 7)])
def test_route(env, rows, ld, dt):
    torch, pmx = env
    z = torch.randn(rows, 40, device="cuda").to(getattr(torch, dt))
    fz = _spread(torch, z, ld)
    kw = dict(balance=0.1, zloss=0.01)
    r, want = pmx.route(fz, 4, **kw), pmx.route(z, 4, **kw)
    assert all(torch.equal(a, b) for a, b in zip(r, want))
    dg = torch.randn(rows, 4, device="cuda")
    dz = pmx.route_grad(fz, r, dg, out=_far(torch, z, ld + 1), **kw)
    assert torch.equal(dz, pmx.route_grad(z, r, dg, **kw))


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_values(env, dt):
    torch, pmx = env
    x = torch.randn(5, 600, device="cuda").to(getattr(torch, dt))
    e4 = torch.float8_e4m3fn
    ld = (1 << 29) + 16
    fx = _spread(torch, x, ld)
    q, s = pmx.fp8_store(x)
    fq, fs = _far(torch, q.view(torch.uint8), ld).view(e4), _far(torch, s, ld + 1)
    pmx.fp8_store(fx, values=fq, scales=fs)
    assert torch.equal(fq.view(torch.uint8), q.view(torch.uint8)) and torch.equal(fs, s)
    assert torch.equal(pmx.fp8_load(fq, fs, 600, out=_far(torch, x, ld + 3)), pmx.fp8_load(q, s, 600, dtype=x.dtype))
    a, q, s = pmx.silu_checkpoint(x, gated=True)
    fq, fs = _far(torch, q.view(torch.uint8), ld).view(e4), _far(torch, s, ld + 1)
    fa, _, _ = pmx.silu_checkpoint(fx, gated=True, out=_far(torch, a, ld + 1), values=fq, scales=fs)
    assert torch.equal(fa, a) and torch.equal(fq.view(torch.uint8), q.view(torch.uint8)) and torch.equal(fs, s)
    da = torch.randn(5, 300, device="cuda").to(x.dtype)
    want = pmx.silu_checkpoint_grad(da, q, s, gated=True)
    fa.copy_(da)
    got = pmx.silu_checkpoint_grad(fa, fq, fs, gated=True, out=fx, act=_far(torch, a, ld + 7))
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("transposed", [False, True])
def test_weights(env, transposed):
    torch, pmx = env
    w = torch.randn(3, 200, 300, device="cuda").bfloat16()
    stride = (1 << 30) + 16
    fw = torch.empty(2 * stride + 200 * 300, dtype=w.dtype, device="cuda").as_strided(w.shape, (stride, 300, 1))
    fw.copy_(w)
    q, s = pmx.fp8_store_weight(w, transposed=transposed)
    fq, fs = (torch.empty(2 * stride + t[0].numel(), dtype=torch.uint8, device="cuda").as_strided(t.shape, (stride, t.shape[2], 1))
              for t in (q, s))
    pmx.fp8_store_weight(fw, transposed=transposed, values=fq.view(torch.float8_e4m3fn), scales=fs)
    assert torch.equal(fq, q.view(torch.uint8)) and torch.equal(fs, s)
    x = torch.randn(500, w.shape[1] if transposed else w.shape[2], device="cuda")
    off = torch.tensor([0, 100, 300, 500], dtype=torch.int32, device="cuda")
    for out in (torch.bfloat16, torch.float32):
        want = pmx.fp8_product(*pmx.fp8_store(x), q, s, off, out_dtype=out)
        assert torch.equal(pmx.fp8_product(*pmx.fp8_store(x), fq.view(torch.float8_e4m3fn), fs, off, out_dtype=out), want)


PRODUCTS = [("stream, shared", 600, 256, 70, 300, 1 << 22, "bfloat16"), ("stream, shared", 600, 256, 70, 300, 1 << 22, "float32"),
            ("stream, own columns", 600, 256, 130, 300, 1 << 22, "bfloat16"), ("64", 600, 300, 515, 8, 1 << 22, "bfloat16"),
            ("64", 600, 300, 515, 8, 1 << 22, "float32"), ("128", 3000, 300, 1300, 4, 1 << 20, "bfloat16"),
            ("128", 3000, 300, 1300, 4, 1 << 20, "float32"), ("256", 9000, 640, 2304, 2, 1 << 18, "bfloat16"),
            ("256", 9000, 640, 2200, 2, 1 << 18, "bfloat16")]


@pytest.mark.parametrize("kind,rows,k,n,groups,ld,out", PRODUCTS)
def test_products(env, kind, rows, k, n, groups, ld, out):
    torch, pmx = env
    print("far products", kind, rows, k, n, groups, ld, out, flush=True)
    assert form(rows, k, n, groups, out, units(torch)) == kind
    e4, dt = torch.float8_e4m3fn, getattr(torch, out)
    g = torch.Generator().manual_seed(rows + n)
    cuts = [0] + torch.sort(torch.randint(0, rows + 1, (groups - 1,), generator=g))[0].tolist() + [rows]
    off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    xq, xs = pmx.fp8_store(torch.randn(rows, k, device="cuda"))
    wq, ws = pmx.fp8_store_weight(torch.randn(groups, n, k, device="cuda"))
    want = pmx.fp8_product(xq, xs, wq, ws, off, out_dtype=dt)
    fx, fs = _spread(torch, xq.view(torch.uint8), ld).view(e4), _spread(torch, xs, ld)
    got = pmx.fp8_product(fx, fs, wq, ws, off, out=_far(torch, want, ld))
    assert torch.equal(got, want)


def test_rows_behind_the_last_group_stay(env):
    """A result inside a longer buffer: the tiles' rows past the last group's end are not written."""
    torch, pmx = env
    for rows, n, cuts in ((9000, 2304, [0, 8999, 9000]), (8961, 2304, [0, 8961]), (9000, 2200, [0, 8960, 9000]), (3001, 1300, [0, 3001]),
                          (601, 515, [0, 601]), (17, 33000, [0, 17])):
        x, w = torch.randn(rows, 640, device="cuda"), torch.randn(len(cuts) - 1, n, 640, device="cuda")
        off = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        q = (*pmx.fp8_store(x), *pmx.fp8_store_weight(w), off)
        for dt in (torch.bfloat16, torch.float32):
            buf = torch.full((rows + 600, n), 3.0, dtype=dt, device="cuda")
            assert torch.equal(pmx.fp8_product(*q, out=buf[:rows]), pmx.fp8_product(*q, out_dtype=dt))
            assert bool((buf[rows:] == 3).all())


def test_most_rows_of_a_norm_and_of_values(env):
    """2^25 rows of 65: more than 2^31 elements; the ends and the middle against fp64, the gradients' sums whole."""
    torch, pmx = env
    rows, cols, step = 1 << 25, 65, 1 << 21
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dy = torch.empty_like(x).normal_(generator=g)
    y, stats = pmx.layer_norm(x)
    dx, dw, db = pmx.layer_norm_grad(dy, x, stats)
    sw, sb, mw, mb = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(4))
    for a in range(0, rows, step):
        h = (x[a:a + step].double() - stats[a:a + step, :1]) * stats[a:a + step, 1:]
        d = dy[a:a + step].double()
        sw += (d * h).sum(0)
        sb += d.sum(0)
        mw += (d * h).abs().sum(0)
        mb += d.abs().sum(0)
    # a thread adds up 2^25 / (256 blocks of 32 rows at least) = 4096 rows, then teams and blocks
    assert bool(((dw - sw).abs() <= 4200 * U * mw).all()) and bool(((db - sb).abs() <= 4200 * U * mb).all())
    q, s = pmx.fp8_store(x)
    back = pmx.fp8_load(q, s, cols)
    act, aq, asc = pmx.silu_checkpoint(x)
    dh, again = pmx.silu_checkpoint_grad(dy, aq, asc)
    for a in (0, rows // 2 - 1000, rows - 3000):
        part = slice(a, a + 3000)
        # alone they are the first rows
        xs, ds = x[part].clone(), dy[part].clone()
        assert all(torch.equal(p[part], w) for p, w in zip((y, stats), pmx.layer_norm(xs)))
        assert torch.equal(dx[part], pmx.layer_norm_grad(ds, xs, stats[part].clone(), params=False)[0])
        q2, s2 = pmx.fp8_store(xs)
        assert torch.equal(q[part].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[part], s2)
        assert torch.equal(back[part], pmx.fp8_load(q2, s2, cols))
        a2, q2, s2 = pmx.silu_checkpoint(xs)
        assert torch.equal(act[part], a2) and torch.equal(aq[part].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(asc[part], s2)
        assert all(torch.equal(p[part], w) for p, w in zip((dh, again), pmx.silu_checkpoint_grad(ds, q2, s2)))
