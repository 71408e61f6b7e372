"""Router, balance loss and their gradients against fp64 and plain sorting.

Tolerances (u = 2^-24): a difference z - max rounds once, which moves its
exponential by |z - max| u; the exponential itself is off by at most 4 u; a row's
sum passes through at most 22 additions.  So p and the gates are off by at most
(60 + 2 D) u relative, D the row's largest distance of finite logits.  Sums over
tokens pass through at most 300 additions here, of terms of one sign."""
import math

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


def _plain(torch, z, top, live, balance, zloss, normalize, dg, up):
    """Token by token, in fp64 on the CPU."""
    z64 = z.double().cpu()
    rows, experts = z64.shape
    ids = torch.full((rows, top), -1, dtype=torch.int32)
    use = torch.ones(rows, dtype=torch.bool) if live is None else live.bool().cpu()
    use = use & (z64 > -math.inf).any(1)
    order = torch.sort(z64, dim=1, descending=True, stable=True)[1][:, :top]
    ok = use[:, None] & (z64.gather(1, order) > -math.inf)
    ids = torch.where(ok, order, torch.full_like(order, -1))
    n = int(use.sum())
    zl = torch.where(use[:, None], z64, torch.zeros_like(z64)).requires_grad_()
    p = torch.softmax(zl, 1)
    sel = p.gather(1, ids.clamp(min=0)) * ok
    gates = sel / sel.sum(1, keepdim=True).clamp(min=1e-300) if normalize else sel
    counts = torch.bincount(ids[ids >= 0].flatten(), minlength=experts)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    flat = ids.flatten()
    key = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    perm = torch.sort(key, stable=True)[1]
    m = int(offsets[-1])
    slots = torch.full((rows * top,), -1, dtype=torch.int64)
    slots[perm[:m]] = torch.arange(m)
    tokens = torch.full((rows * top,), -1, dtype=torch.int64)
    tokens[:m] = perm[:m] // top
    one = use.double()
    lse = torch.logsumexp(zl, 1)
    loss = torch.zeros((), dtype=torch.float64)
    mag = 0.0
    if n:
        share = (p * one[:, None]).sum(0) / n
        loss = balance * experts / (top * n) * (counts.double() * share).sum() + zloss * (lse ** 2 * one).sum() / n
        mag = float(loss.detach().abs() + abs(zloss) * ((1 + lse.detach().abs()) ** 2 * one).sum() / n)
    # the z term's gradient is written out: the softmax that automatic differentiation takes as exp(z - lse) is off by a
    # factor of `experts` where lse rounds to the largest logit (-3.4e38 + log 10 in fp64)
    total = up * (loss - (zloss * (lse ** 2 * one).sum() / n if n else 0.0))
    if dg is not None:
        total = total + (gates * dg.double().cpu() * one[:, None]).sum()
    dz = torch.zeros_like(z64)
    if n:
        total.backward()
        dz = (zl.grad + up * zloss * 2 / n * lse.detach()[:, None] * p.detach()) * one[:, None]
    return dict(ids=ids, gates=gates.detach() * one[:, None], counts=counts, offsets=offsets, slots=slots.view(rows, top),
                tokens=tokens, loss=float(loss), n=n, dz=dz, mag=mag, p=p.detach(), lse=lse.detach())


def _check(env, z, top, live=None, balance=1e-2, zloss=1e-3, normalize=True, seed=0):
    torch, pmx = env
    rows, experts = z.shape
    g = torch.Generator().manual_seed(seed)
    dg = torch.randn(rows, top, generator=g).cuda()
    up = torch.tensor(0.7, device="cuda")
    kw = dict(live=live, balance=balance, zloss=zloss, normalize=normalize)
    r = pmx.route(z, top, **kw)
    w = _plain(torch, z, top, live, balance, zloss, normalize, dg, float(up))
    for k in ("ids", "counts", "offsets", "slots", "tokens"):
        assert torch.equal(getattr(r, k).long().cpu(), w[k].long()), k
    assert int(r.tally[-1]) == w["n"]
    zf = z.double().cpu()
    fin = torch.where(torch.isfinite(zf), zf, zf.amax(1, keepdim=True).clamp(min=-1e300))
    D = (fin.amax(1) - fin.amin(1)).clamp(max=120.0)[:, None]
    rel = (60 + 2 * D) * U
    assert bool(((r.gates.double().cpu() - w["gates"]).abs() <= rel * w["gates"] + 1e-38).all())
    # beyond fp32's largest number its rounding is infinity
    want = w["loss"] if abs(w["loss"]) < 3.4e38 else math.copysign(math.inf, w["loss"])
    assert float(r.loss) == want or abs(float(r.loss) - want) <= (400 + 2 * float(D.max() if rows else 0)) * U * w["mag"] + 1e-38
    dz = pmx.route_grad(z, r, dg, upstream=up, **kw)
    # the terms' sizes: p (a + sum p a + z part + gates' part), and the gates' own
    n = max(w["n"], 1)
    a = 0.7 * abs(balance) * experts / (top * n * n) * w["counts"].double()
    gd = (w["gates"] * dg.double().cpu()).abs()
    p = torch.nan_to_num(w["p"])
    size = p * (a + (p * a).sum(1, keepdim=True) + 1.4 * abs(zloss) / n * (1 + w["lse"].abs() + fin.abs().amax(1))[:, None]
                + (0 if normalize else 1) * gd.sum(1, keepdim=True))
    own = gd + (w["gates"] * gd.sum(1, keepdim=True) if normalize else 0)
    size = size.scatter_add(1, w["ids"].long().clamp(min=0), own * (w["ids"] >= 0))
    tol = (3 * rel + 100 * U) * size + torch.finfo(z.dtype).eps / 2 * w["dz"].abs() + 1e-37
    bad = ~((dz.double().cpu() - w["dz"]).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float((dz.double().cpu() - w["dz"]).abs().max()))
    r2 = pmx.route(z, top, **kw)
    assert all(torch.equal(x, y) for x, y in zip(r, r2)) and torch.equal(dz, pmx.route_grad(z, r2, dg, upstream=up, **kw))
    return r, dz


CASES = [(1, 1, 1), (1, 2, 1), (5, 3, 3), (16, 32, 2), (64, 64, 4), (65, 64, 8), (63, 16, 16), (100, 17, 2), (129, 65, 5),
         (300, 128, 8), (257, 129, 3), (90, 256, 16), (80, 257, 7), (70, 512, 6), (200, 513, 4), (33, 1000, 16), (66, 1000, 1),
         (16383, 8, 2), (16384, 8, 2), (20011, 33, 3), (8192, 257, 3), (8195, 300, 5),
         (3001, 1000, 4), (16, 700, 8), (17, 700, 8), (32, 300, 4), (64, 400, 6)]


@pytest.mark.parametrize("rows,experts,top", CASES)
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_against_plain(env, rows, experts, top, dt):
    torch, pmx = env
    print("route", rows, experts, top, dt, flush=True)
    g = torch.Generator().manual_seed(rows * 7 + experts)
    z = (torch.randn(rows, experts, generator=g) * 1.5).to(getattr(torch, dt)).cuda()
    live = (torch.rand(rows, generator=g) < 0.8).cuda()
    _check(env, z, top, live=live)
    _check(env, z, top, normalize=False)


def test_ties_take_the_lowest_index(env):
    torch, pmx = env
    for experts in (8, 64, 100, 300, 1000):
        z = torch.zeros(70, experts, device="cuda")
        z[:, ::3] = -0.0  # equal to 0.0
        r, _ = _check(env, z, min(experts, 6))
        assert bool((r.ids == torch.arange(6, device="cuda")).all())
        z = torch.randint(0, 3, (130, experts), generator=torch.Generator().manual_seed(experts)).float().cuda()
        _check(env, z, 5)


def test_masked_experts_and_rows(env):
    torch, pmx = env
    inf = math.inf
    for experts in (10, 200):
        z = torch.randn(150, experts, generator=torch.Generator().manual_seed(3)).cuda()
        z[3] = -inf                 # nothing left: not a live token
        z[4, 1:] = -inf             # one expert left of four
        z[5, :-2] = -inf            # two
        z[100] = -inf
        live = torch.ones(150, dtype=torch.uint8, device="cuda")
        live[6] = 0
        z[7] = torch.finfo(torch.float32).min  # the type's lowest value is a value
        z[8, 0] = 3e38
        r, dz = _check(env, z, 4, live=live)
        assert r.ids[4].tolist() == [0, -1, -1, -1] and r.gates[4].tolist() == [1, 0, 0, 0]
        assert bool((r.ids[3] == -1).all()) and bool((dz[3] == 0).all()) and bool((dz[6] == 0).all())
        assert r.ids[7].tolist() == [0, 1, 2, 3]
        # what a dead row holds does not matter
        z2 = z.clone()
        z2[6] = float("nan")
        r2 = pmx.route(z2, 4, live=live, balance=1e-2, zloss=1e-3)
        assert torch.equal(r2.loss, r.loss) and torch.equal(r2.ids, r.ids) and torch.equal(r2.gates, r.gates)
        dz2 = pmx.route_grad(z2, r2, None, live=live, balance=1e-2, zloss=1e-3)
        assert bool(dz2.isfinite().all())


def test_no_live_tokens(env):
    torch, pmx = env
    for rows in (0, 5, 100):
        z = torch.randn(rows, 12, device="cuda")
        live = torch.zeros(rows, dtype=torch.bool, device="cuda")
        r = pmx.route(z, 3, live=live, balance=1.0, zloss=1.0)
        assert float(r.loss) == 0 and int(r.tally.sum()) == 0 and int(r.offsets.sum()) == 0
        assert bool((r.ids == -1).all()) and bool((r.tokens == -1).all()) and bool((r.slots == -1).all())
        dz = pmx.route_grad(z, r, torch.ones(rows, 3, device="cuda"), live=live, balance=1.0, zloss=1.0)
        assert bool((dz == 0).all())


def test_nan_and_inf_rows(env):
    torch, pmx = env
    for rows in (20, 200):
        z = torch.randn(rows, 40, device="cuda")
        z[2, 5], z[9, 39] = float("nan"), math.inf
        r = pmx.route(z, 4, balance=1e-2, zloss=1e-3)
        for t in (2, 9):
            assert bool((r.ids[t] == -1).all()) and bool((r.slots[t] == -1).all()) and bool(r.gates[t].isnan().all())
        assert bool(r.loss.isnan()) and int(r.tally[-1]) == rows and int(r.offsets[-1]) == 4 * (rows - 2)
        dz = pmx.route_grad(z, r, torch.ones(rows, 4, device="cuda"), balance=1e-2, zloss=1e-3)
        bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
        bad[2] = bad[9] = True
        assert bool(dz[bad].isnan().all()) and bool(dz[~bad].isfinite().all())


def test_strides_in_place_and_without_order(env):
    torch, pmx = env
    for dt in (torch.float32, torch.bfloat16):
        big = torch.randn(90, 100, device="cuda").to(dt)
        z = big[5:85, 3:74]
        kw = dict(balance=0.1, zloss=0.01)
        r, want = pmx.route(z, 4, **kw), pmx.route(z.contiguous(), 4, **kw)
        assert all(torch.equal(a, b) for a, b in zip(r, want))
        bare = pmx.route(z, 4, order=False, **kw)
        assert bare.slots is None and bare.tokens is None and torch.equal(bare.ids, r.ids) and torch.equal(bare.offsets, r.offsets)
        dg = torch.randn(80, 4, device="cuda")
        dz = pmx.route_grad(z.contiguous(), r, dg, **kw)
        keep = big.clone()
        assert pmx.route_grad(z, r, dg, out=z, **kw) is z and torch.equal(z, dz)
        keep[5:85, 3:74] = dz
        assert torch.equal(big, keep)


def test_differences(env):
    """dz against central differences of the fp64 loss with the choice held: step 1e-4, error of order 1e-8."""
    torch, pmx = env
    g = torch.Generator().manual_seed(8)
    z = torch.randn(30, 20, generator=g)
    dg = torch.randn(30, 3, generator=g)
    v = torch.randn(30, 20, generator=g, dtype=torch.float64)
    for normalize in (True, False):
        kw = dict(balance=0.5, zloss=0.1, normalize=normalize)
        r = pmx.route(z.cuda(), 3, **kw)
        dz = pmx.route_grad(z.cuda(), r, dg.cuda(), **kw).double().cpu()
        ids, c = r.ids.long().cpu(), r.counts.double().cpu()

        def value(s):
            p = torch.softmax(z.double() + s * v, 1)
            sel = p.gather(1, ids)
            if normalize:
                sel = sel / sel.sum(1, keepdim=True)
            return (sel * dg.double()).sum() + 0.5 * 20 / (3 * 30) * (c * p.mean(0)).sum() \
                + 0.1 * (torch.logsumexp(z.double() + s * v, 1) ** 2).mean()

        want = (value(1e-4) - value(-1e-4)) / 2e-4
        assert abs(float((dz * v).sum() - want)) <= 1e-6 * float(dz.norm() * v.norm())


def test_global_counts(env):
    """The gradient takes the tally it is given: two halves with the summed tally are the whole."""
    torch, pmx = env
    z = torch.randn(128, 24, device="cuda")
    kw = dict(balance=0.3, zloss=0.0)
    whole = pmx.route(z, 2, **kw)
    dz = pmx.route_grad(z, whole, **kw)
    a, b = pmx.route(z[:64], 2, **kw), pmx.route(z[64:], 2, **kw)
    tally = a.tally + b.tally
    assert torch.equal(tally, whole.tally)
    parts = [pmx.route_grad(z[i:i + 64], r._replace(tally=tally), **kw) for i, r in ((0, a), (64, b))]
    assert torch.equal(torch.cat(parts), dz)


def test_refusals(env):
    torch, pmx = env
    z = torch.randn(6, 8, device="cuda")
    r = pmx.route(z, 2)

    def refused(f, kind=(ValueError, TypeError)):
        with pytest.raises(kind):
            f()

    refused(lambda: pmx.route(z, 0), pmx.PmxError)
    refused(lambda: pmx.route(z, 9), pmx.PmxError)
    refused(lambda: pmx.route(torch.randn(6, 40, device="cuda"), 17), pmx.PmxError)
    refused(lambda: pmx.route(torch.randn(2, pmx.MAX_GROUPS + 1, device="cuda"), 2), pmx.PmxError)
    refused(lambda: pmx.route(z, 2, balance=float("inf")), pmx.PmxError)
    refused(lambda: pmx.route(z, -1))
    refused(lambda: pmx.route(z, (1 << 32) + 2))
    refused(lambda: pmx.route(z.half(), 2))
    refused(lambda: pmx.route(z.t(), 2))
    refused(lambda: pmx.route(z, 2, live=torch.ones(5, dtype=torch.bool, device="cuda")))
    refused(lambda: pmx.route(z, 2, live=torch.ones(6, device="cuda")))
    refused(lambda: pmx.route_grad(z[:5], r))
    refused(lambda: pmx.route_grad(z, r, torch.ones(6, 3, device="cuda")))
    refused(lambda: pmx.route_grad(z, r, upstream=torch.ones(2, device="cuda")))
    refused(lambda: pmx.route_grad(z, r._replace(tally=r.tally[:-1])))
    refused(lambda: pmx.route_grad(z, r, out=torch.empty(6, 9, device="cuda")))


def test_rows_left_out_without_normalization(env):
    """Rows with nothing left, and rows that are not live whatever they hold, have gates 0 and gradient 0."""
    torch, pmx = env
    for experts, top, rows in ((10, 4, 60), (200, 4, 150), (700, 2, 40)):
        z = torch.randn(rows, experts, generator=torch.Generator().manual_seed(5)).cuda()
        z[3] = -math.inf
        live = torch.ones(rows, dtype=torch.uint8, device="cuda")
        live[6] = live[7] = live[8] = 0
        z[8] = -math.inf
        _check(env, z, top, live=live, normalize=False)
        z[6], z[7, 1] = float("nan"), math.inf
        kw = dict(live=live, balance=1e-2, zloss=1e-3, normalize=False)
        r = pmx.route(z, top, **kw)
        dz = pmx.route_grad(z, r, torch.ones(rows, top, device="cuda"), **kw)
        assert bool(r.loss.isfinite()) and bool(dz.isfinite().all())
        for t in (3, 6, 7, 8):
            assert bool((r.ids[t] == -1).all()) and bool((r.gates[t] == 0).all()) and bool((dz[t] == 0).all())
