"""Router: the launch between the two at few experts, and logits beyond 2^31 of them."""
import pytest

from test_gpu_route import _check, env  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


# counts of all chunks are more than every block reads: chunks^2 experts > 2^25, 64 tokens a chunk
@pytest.mark.parametrize("rows,experts,top", [(70001, 32, 3), (66000, 64, 4), (131072, 8, 2), (40003, 128, 8), (30000, 200, 5)])
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_launch_between(env, rows, experts, top, dt):  # noqa: F811
    torch, pmx = env
    print("route, launch between", rows, experts, top, dt, flush=True)
    g = torch.Generator().manual_seed(rows + experts)
    z = torch.randn(rows, experts, generator=g).to(getattr(torch, dt)).cuda()
    live = (torch.rand(rows, generator=g) < 0.9).cuda()
    r, _ = _check(env, z, top, live=live)
    bare = pmx.route(z, top, live=live, balance=1e-2, zloss=1e-3, order=False)
    assert torch.equal(bare.tally, r.tally) and torch.equal(bare.offsets, r.offsets) and torch.equal(bare.loss, r.loss)


@pytest.mark.parametrize("rows,experts", [(1 << 25, 65), ((1 << 25) - 77, 70)])
def test_most_rows(env, rows, experts):  # noqa: F811
    """2^25 tokens, more than 2^31 logits: ids, gates, counts, order and the gradient, by torch on the GPU."""
    torch, pmx = env
    print("route, most rows", rows, experts, flush=True)
    top = 2
    g = torch.Generator(device="cuda").manual_seed(rows)
    z = torch.empty(rows, experts, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    z += torch.arange(experts, device="cuda").bfloat16() * 0.01
    kw = dict(balance=0.5, zloss=0.0)
    r = pmx.route(z, top, **kw)
    step = 1 << 22
    share = torch.zeros(experts, dtype=torch.float64, device="cuda")
    for a in range(0, rows, step):
        part = z[a:a + step].float()
        # ties to the lowest index
        order = torch.sort(part, dim=1, descending=True, stable=True)[1][:, :top]
        assert torch.equal(r.ids[a:a + step].long(), order)
        chosen = torch.softmax(part.gather(1, order), 1)
        assert bool(((r.gates[a:a + step] - chosen).abs() <= 100 * 2.0 ** -24 * chosen).all())
        share += torch.softmax(part, 1).sum(0, dtype=torch.float64)
    counts = torch.zeros(experts, dtype=torch.int64, device="cuda")
    for e in range(experts):
        counts[e] = (r.ids == e).sum()
    assert torch.equal(r.counts.long(), counts) and int(r.tally[-1]) == rows and int(r.offsets[-1]) == rows * top
    assert torch.equal(r.offsets.long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]))
    want = 0.5 * experts / (top * rows) * float((counts.double() * share / rows).sum())
    assert abs(float(r.loss) - want) <= 600 * 2.0 ** -24 * want
    # slots and tokens: each expert's tokens ascend, and slots is their inverse
    slots = r.slots.view(-1).long()
    flat = torch.arange(rows * top, device="cuda", dtype=torch.int32) // top
    assert torch.equal(r.tokens[slots], flat)
    del slots, flat
    up = r.tokens[1:] > r.tokens[:-1]
    border = torch.zeros(rows * top, dtype=torch.bool, device="cuda")
    border[r.offsets[1:-1].long()] = True
    assert bool((up | border[1:]).all())
    del up, border
    dz = pmx.route_grad(z, r, **kw)
    a = 0.5 * experts * counts.double() / (top * float(rows) * rows)
    for lo in (0, rows // 2, rows - 5000):
        p = torch.softmax(z[lo:lo + 5000].double(), 1)
        w = p * (a - (p * a).sum(1, keepdim=True))
        size = p * (a + (p * a).sum(1, keepdim=True))
        assert bool(((dz[lo:lo + 5000].double() - w).abs() <= 2.0 ** -8 * w.abs() + 400 * 2.0 ** -24 * size).all())
    del dz
    torch.cuda.empty_cache()
