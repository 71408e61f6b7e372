"""Values in 8 bits whose rows, scales and matrices lie at distances of their own: the bytes are those of a packed
call, what lies between them stays, and what reads them reads the same."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    from preconditioned_optimizer_matrix_amd import pmx
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    return torch, pmx


def _room(torch, rows, wide, blocks):
    """A view of rows x wide bytes at a row distance of a multiple of 16, its buffer, and the same for the scales."""
    v = torch.full((rows + 2, wide + 48), 3, dtype=torch.uint8, device="cuda")
    s = torch.full((rows + 2, blocks + 5), 9, dtype=torch.uint8, device="cuda")
    return v.view(torch.float8_e4m3fn)[1:1 + rows, 32:32 + wide], v, s[1:1 + rows, 2:2 + blocks], s


def _kept(view, buf, fill):
    """The buffer holds `fill` wherever the view does not lie."""
    copy = buf.clone()
    rows, wide = view.shape[-2:]
    at = (view.data_ptr() - buf.data_ptr())
    copy.as_strided(view.shape, view.stride(), at).fill_(fill)
    return bool((copy == fill).all())


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (23, 403), (5, 128), (40, 1000), (300, 129)])
def test_rows(env, rows, cols, dt):
    torch, pmx = env
    print("8-bit rows at distances", rows, cols, dt, flush=True)
    dt = getattr(torch, dt)
    x = torch.randn(rows, cols, device="cuda").to(dt)
    wide = -(-cols // 128) * 128
    q, s = pmx.fp8_store(x)
    v, vb, c, cb = _room(torch, rows, wide, wide // 128)
    assert v.stride(0) % 16 == 0 and (rows == 1 or v.stride(0) > wide)
    got = pmx.fp8_store(x, values=v, scales=c)
    assert got[0] is v and got[1] is c
    assert torch.equal(v.contiguous().view(torch.uint8), q.view(torch.uint8)) and torch.equal(c, s)
    assert _kept(v.view(torch.uint8), vb, 3) and _kept(c, cb, 9)
    for out in (torch.bfloat16, torch.float32):
        assert torch.equal(pmx.fp8_load(v, c, cols, dtype=out), pmx.fp8_load(q, s, cols, dtype=out))


@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 3), (23, 200), (7, 256), (130, 515)])
def test_checkpoint(env, rows, cols, gated, dt):
    torch, pmx = env
    print("checkpoint at distances", rows, cols, gated, dt, flush=True)
    dt = getattr(torch, dt)
    halves = 2 if gated else 1
    big = torch.randn(rows + 1, halves * cols + 9, device="cuda").to(dt)
    h = big[1:, 5:5 + halves * cols]
    wide = halves * (-(-cols // 128) * 128)
    a, q, s = pmx.silu_checkpoint(h.contiguous(), gated=gated)
    v, vb, c, cb = _room(torch, rows, wide, wide // 128)
    ab = torch.full((rows, cols + 4), 5.0, device="cuda", dtype=dt)
    a2, _, _ = pmx.silu_checkpoint(h, gated=gated, out=ab[:, 3:3 + cols], values=v, scales=c)
    assert torch.equal(a2, a) and bool((ab[:, :3] == 5).all()) and bool((ab[:, 3 + cols:] == 5).all())
    assert torch.equal(v.contiguous().view(torch.uint8), q.view(torch.uint8)) and torch.equal(c, s)
    assert _kept(v.view(torch.uint8), vb, 3) and _kept(c, cb, 9)
    da = torch.randn(rows, cols, device="cuda").to(dt)
    want = pmx.silu_checkpoint_grad(da, q, s, gated=gated)
    got = pmx.silu_checkpoint_grad(da, v, c, gated=gated)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("groups,n,k", [(1, 1, 1), (3, 130, 127), (2, 257, 515), (4, 64, 300)])
def test_weights(env, groups, n, k, transposed):
    torch, pmx = env
    print("8-bit weights at distances", groups, n, k, transposed, flush=True)
    for dt in (torch.bfloat16, torch.float32):
        big = torch.randn(groups, n + 2, k + 3, device="cuda").to(dt)
        w = big[:, 1:1 + n, 2:2 + k]
        q, s = pmx.fp8_store_weight(w.contiguous(), transposed=transposed)
        r, wide = q.shape[1:]
        vb = torch.full((groups, r + 2, wide + 32), 3, dtype=torch.uint8, device="cuda")
        cb = torch.full((groups, s.shape[1] + 1, s.shape[2] + 3), 9, dtype=torch.uint8, device="cuda")
        v, c = vb.view(torch.float8_e4m3fn)[:, 1:1 + r, 16:16 + wide], cb[:, :s.shape[1], 1:1 + s.shape[2]]
        pmx.fp8_store_weight(w, transposed=transposed, values=v, scales=c)
        assert torch.equal(v.contiguous().view(torch.uint8), q.view(torch.uint8)) and torch.equal(c, s)
        assert _kept(v.view(torch.uint8), vb, 3) and _kept(c, cb, 9)
