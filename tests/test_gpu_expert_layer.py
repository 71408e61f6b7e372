"""The expert layer's operators run together: examples/expert_layer.py, and the same calls captured into a HIP graph.

The fp32 gradients are compared with the same pass in fp64, whose products take the values that e4m3 keeps of their
operands.  Tolerance, of each gradient's norm: an operand that differs by 1e-5 relative (what fp32 sums before it
leave) lands on the other side of a rounding border with a chance of 1e-5 / 2^-4, and is then off by 2^-3 at most:
2^-3 sqrt(1.6e-4) = 1.6e-3 of the norm at each of the three roundings of a gradient's way, 5e-3 together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return torch, m


def _kept(torch, v, tiles=False):
    """What 8 bits keep of v: blocks of 128 of a row, or 128 x 128 tiles."""
    r, c = v.shape
    p = torch.nn.functional.pad(v.double(), (0, -c % 128, 0, -r % 128 if tiles else 0))
    t = p.view(p.shape[0] // 128, 128, -1, 128) if tiles else p.view(p.shape[0], 1, -1, 128)
    amax = t.abs().amax(3, keepdim=True).amax(1, keepdim=True)
    power = torch.tensor([2.0 ** k for k in range(-126, 128)], dtype=torch.float64, device=v.device)
    scale = torch.where(amax > 0, power[torch.searchsorted(448 * power, amax).clamp(max=253)], torch.ones_like(amax))
    return ((t / scale).float().to(torch.float8_e4m3fn).double() * scale).reshape(p.shape)[:r, :c]


def _plain(torch, params, x, dy, top, balance, zloss):
    p = {k: v.double() for k, v in params.items()}
    x, dy = x.double(), dy.double()
    rows, dim = x.shape
    experts, hidden = p["down"].shape[0], p["down"].shape[2]
    m = x.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + 1e-5)
    xh = (x - m) * r
    n = xh * p["weight"] + p["bias"]
    z = n @ p["router"].t()
    ids = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :top]
    zr = z.clone().requires_grad_()
    gates = torch.softmax(zr.gather(1, ids), 1)
    counts = torch.bincount(ids.flatten(), minlength=experts).double()
    loss = balance * experts / (top * rows) * (counts * torch.softmax(zr, 1).mean(0)).sum() + zloss * (torch.logsumexp(zr, 1) ** 2).mean()
    dn = torch.zeros_like(n)
    y, dgates = x.clone(), torch.zeros_like(gates)
    grads = {k: torch.zeros_like(v) for k, v in p.items()}
    for e in range(experts):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        up, down = _kept(torch, params["up"][e], True), _kept(torch, params["down"][e], True)
        n8 = _kept(torch, n[t])
        h = n8 @ up.t()
        gate, val = h[:, :hidden], h[:, hidden:]
        a = gate * torch.sigmoid(gate) * val
        o = _kept(torch, a) @ down.t()
        g = gates[t, j].detach()[:, None]
        y.index_add_(0, t, g * o)
        dgates[t, j] = (o * dy[t]).sum(1)
        do = g * dy[t]
        da = _kept(torch, do) @ down
        k1, k2 = _kept(torch, gate), _kept(torch, val)
        s = torch.sigmoid(k1)
        dh = torch.cat([da * k2 * s * (1 + k1 * (1 - s)), da * k1 * s], 1)
        grads["down"][e] = do.t() @ (k1 * s * k2)
        grads["up"][e] = dh.t() @ n8
        dn.index_add_(0, t, _kept(torch, dh) @ up)
    (loss + (gates * dgates).sum()).backward()
    dz = zr.grad
    dn += dz @ p["router"]
    grads["router"] = dz.t() @ n
    gw = dn * p["weight"]
    dx = r * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True)) + dy
    grads["weight"], grads["bias"] = (dn * xh).sum(0), dn.sum(0)
    return y, loss.detach(), dx, grads


@pytest.mark.parametrize("tokens,dim,hidden,experts,top", [(300, 200, 150, 5, 2), (1000, 256, 384, 8, 3)])
def test_gradients(example, tokens, dim, hidden, experts, top):
    torch, m = example
    print("expert layer", tokens, dim, flush=True)
    params = m.make(dim, hidden, experts, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    params["weight"] += 0.2 * torch.randn(dim, generator=g, device="cuda")
    params["bias"] += 0.2 * torch.randn(dim, generator=g, device="cuda")
    x, dy = torch.randn(tokens, dim, generator=g, device="cuda"), torch.randn(tokens, dim, generator=g, device="cuda")
    weights = m.to_8bit(params)
    y, loss, saved = m.forward(params, weights, x, top=top, balance=0.1, zloss=0.01)
    dx, grads = m.backward(params, weights, saved, dy)
    wy, wloss, wdx, want = _plain(torch, params, x, dy, top, 0.1, 0.01)
    assert abs(float(loss) - float(wloss)) <= 1e-5 * float(wloss)
    for name, a, b in [("y", y, wy), ("dx", dx, wdx)] + [(k, grads[k], want[k]) for k in want]:
        assert float((a.double() - b).norm()) <= 5e-3 * float(b.norm()), name


def test_training_runs(example):
    _, m = example
    losses = m.train(steps=4, tokens=512)
    assert all(v == v and v < float("inf") for v in losses)


@pytest.mark.parametrize("tokens", [16, 700])
def test_captured_into_a_graph(example, tokens):
    """The whole pass replayed on new inputs, between eager work, gives the eager bits."""
    torch, m = example
    from preconditioned_optimizer_matrix_amd import pmx
    params = m.make(seed=5)
    weights = m.to_8bit(params)
    dim = params["weight"].numel()
    x, dy = (torch.zeros(tokens, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    one = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    router = params["router"].bfloat16()[None]
    up, down = torch.tensor(1.0, device="cuda"), weights["down"]

    def work():
        n, stats = pmx.layer_norm(x, params["weight"], params["bias"])
        z = pmx.grouped_product(n, router, one, trans_b=True, out_dtype=torch.float32)
        kw = dict(balance=0.1, zloss=0.01)
        r = pmx.route(z, 2, **kw)
        rows = pmx.fp8_store(pmx.embedding(n, r.tokens))
        h = pmx.fp8_product(*rows, *weights["up"][0], r.offsets)
        a, *hidden = pmx.silu_checkpoint(h, gated=True)
        o = pmx.fp8_product(*pmx.fp8_store(a), *down[0], r.offsets)
        do = pmx.embedding(dy, r.tokens)
        da = pmx.fp8_product(*pmx.fp8_store(do), *down[1], r.offsets)
        dh, again = pmx.silu_checkpoint_grad(da, *hidden, gated=True)
        dr = pmx.fp8_product(*pmx.fp8_store(dh), *weights["up"][1], r.offsets, out_dtype=torch.float32)
        dz = pmx.route_grad(z, r, r.gates, upstream=up, **kw)
        dn = pmx.embedding_grad(dr, r.tokens, tokens, out_dtype=torch.bfloat16)
        dx, dw, db = pmx.layer_norm_grad(dn, x, stats, params["weight"])
        return (o, again, dz, dx, dw, db, pmx.fp8_load(*rows)) + tuple(r)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for seed in range(4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(tokens, dim, generator=g, device="cuda"))
        dy.copy_(torch.randn(tokens, dim, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed


def test_two_streams_at_once(example):
    """Two passes on two streams, each with its own workspaces, do not disturb each other."""
    torch, m = example
    params = m.make(seed=6)
    weights = m.to_8bit(params)
    dim = params["weight"].numel()
    g = torch.Generator(device="cuda").manual_seed(7)
    xs = [torch.randn(900, dim, generator=g, device="cuda").bfloat16() for _ in range(2)]

    def work(x):
        y, loss, saved = m.forward(params, weights, x)
        dx, grads = m.backward(params, weights, saved, x)
        return [y, loss, dx] + list(grads.values())

    want = [work(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for s, x in zip(streams, xs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(work(x))
        torch.cuda.synchronize()
        # index_put of the example's own gates apart, every step is bit-exact
        assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q))
