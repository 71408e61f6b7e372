"""The distillation loss and its gradient against a plain fp64 implementation.

Tolerance.  An exponential exp(x), x <= 0, is computed as 2^(x log2 e) with two
fp32 roundings of the argument: relative error at most (2 |x| + 2) 2^-24, below
6e-6 for |x| <= 45; smaller terms (e^-45 of the largest) do not show in any sum.
A sum over the vocabulary adds at most 512 of a thread's own terms and a tree:
530 x 2^-24 = 3.2e-5.  With D = 5e-5 for both together,
  |dz error|   <= D w (mix tau (q + p) + (1 - mix) (s + [label])) (+ bf16 rounding 2^-8),
  |loss error| <= D (mix tau^2 (1 + sum p (|log p| + |log q|)) + (1 - mix) (1 + |log s|)).
The total adds the rows in fp64: the sum of the rows' bounds and one rounding."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
D = 5e-5


@pytest.fixture(scope="module")
def env():
    import torch
    from preconditioned_optimizer_matrix_amd import pmx
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    return torch, pmx, dev


def _log_softmax(x):
    m = x.max()
    if m == -np.inf:
        return None
    return x - m - np.log(np.exp(x - m).sum())


def reference(z, ids, teacher, tau, mix, labels, weights, up=1.0):
    """Row losses, total, gradient and their bounds, in fp64, row by row."""
    rows, vocab = z.shape
    loss, lb = np.zeros(rows), np.zeros(rows)
    dz, db = np.zeros((rows, vocab)), np.zeros((rows, vocab))
    w = np.full(rows, 1.0 / rows) if weights is None else weights
    for t in range(rows):
        if w[t] == 0:
            continue
        ls, lq = _log_softmax(z[t]), _log_softmax(z[t] / tau)
        if ls is None:
            continue
        if mix > 0:
            ok = [i for i in range(ids.shape[1]) if 0 <= ids[t, i] < vocab and teacher[t, i] > -np.inf]
            if ok:
                lp = _log_softmax(teacher[t, ok] / tau)
                p = np.exp(lp)
                at = lq[ids[t, ok]]
                live = p > 1e-38  # fp32 keeps nothing below
                loss[t] += mix * tau ** 2 * (p[live] * (lp - at)[live]).sum()
                lb[t] += mix * tau ** 2 * (1 + (p[live] * (np.abs(lp) + np.abs(at))[live]).sum())
                q = np.exp(lq)
                dz[t] += mix * tau * q
                db[t] += mix * tau * q
                np.add.at(dz[t], ids[t, ok], -mix * tau * p)
                np.add.at(db[t], ids[t, ok], mix * tau * p)
        if mix < 1 and 0 <= labels[t] < vocab:
            s = np.exp(ls)
            loss[t] -= (1 - mix) * ls[labels[t]]
            lb[t] += (1 - mix) * (1 + abs(ls[labels[t]]))
            dz[t] += (1 - mix) * s
            db[t] += (1 - mix) * s
            dz[t, labels[t]] -= 1 - mix
            db[t, labels[t]] += 1 - mix
        dz[t] *= w[t] * up
        db[t] *= abs(w[t] * up)
    return loss, D * lb, (w * loss)[w != 0].sum(), D * (np.abs(w) * lb)[w != 0].sum(), dz, D * db + 1e-37


def _inputs(torch, dev, rows, vocab, top, dtype, seed, spread=4.0, ldp=0):
    g = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    z = (torch.randn(rows, vocab + ldp, generator=g) * spread).to(dt)
    ids = torch.stack([torch.randperm(vocab, generator=g)[:top] for _ in range(rows)]) if top else torch.zeros(rows, 0, dtype=torch.int64)
    teacher = (torch.randn(rows, top, generator=g) * 3 + 2).to(dt)
    labels = torch.randint(0, vocab, (rows,), generator=g)
    weights = torch.rand(rows, generator=g) + 0.1
    return z.to(dev)[:, :vocab], ids.to(dev), teacher.to(dev), labels.to(dev), weights.to(dev)


def _np(t):
    return None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _compare(torch, total, rows, dz, ref, bf16, lossy=True):
    loss, lb, tot, tb, g, gb = ref
    with np.errstate(invalid="ignore"):
        if rows is not None:
            r = _np(rows)
            assert ((np.abs(r - loss) <= lb + 2.0 ** -23 * np.abs(loss)) | (r == loss)).all()
            x = float(total)
            assert abs(x - tot) <= tb + 2.0 ** -23 * abs(tot) or x == tot
        if dz is not None:
            extra = 2.0 ** -8 * (1 + 1e-6) * np.abs(g) + 1e-40 if bf16 else 0.0
            assert (np.abs(_np(dz) - g) <= gb * (1 + 2.0 ** -8 * bf16) + extra).all()


# vocabularies of every register class, exact fits and one more, odd row
# starts, and rows too long for the registers
SHAPES = [(1, 1, 1), (2, 7, 3), (5, 300, 20), (3, 4088, 5), (3, 4097, 64), (4, 8185, 9), (2, 16376, 17), (2, 16385, 4), (3, 33001, 30),
          (2, 65528, 8), (2, 66000, 8), (1, 131064, 128), (2, 131073, 6), (40, 515, 515)]


@pytest.mark.parametrize("rows,vocab,top", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tau,mix", [(1.0, 1.0), (2.0, 0.7), (1.5, 0.25), (1.0, 0.5), (3.0, 0.0), (4.0, 1.0), (8.0, 0.5)])
def test_loss_and_gradient(env, rows, vocab, top, dtype, tau, mix):
    torch, pmx, dev = env
    print("distill", rows, vocab, top, dtype, tau, mix, flush=True)
    z, ids, teacher, labels, weights = _inputs(torch, dev, rows, vocab, top, dtype, vocab + rows)
    kw = dict(tau=tau, mix=mix, labels=labels if mix < 1 else None, weights=weights)
    ref = reference(_np(z), _np(ids), _np(teacher), tau, mix, _np(labels), _np(weights))
    total, r, _, dz = pmx.distill_loss(z, ids, teacher, grad=True, **kw)
    _compare(torch, total, r, dz, ref, dtype == "bf16")
    total, r, stats, none = pmx.distill_loss(z, ids, teacher, **kw)
    assert none is None
    _compare(torch, total, r, None, ref, False)
    up = torch.tensor(-3.0, device=dev)
    dz = pmx.distill_grad(z, ids, teacher, stats, upstream=up, **kw)
    loss, lb, tot, tb, g, gb = ref
    _compare(torch, None, None, dz, (loss, lb, tot, tb, -3 * g, 3 * gb), dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(6, 77), (4, 9001), (3, 140001)])
def test_strides_types_and_in_place(env, dtype, rows, vocab):
    """Row distances beyond the vocabulary (so every row starts at another
    alignment), int32 indices, a teacher of the other type, equal weights, and
    the gradient written over the logits; what lies between the rows stays."""
    torch, pmx, dev = env
    print("strides", dtype, rows, vocab, flush=True)
    z, ids, teacher, labels, _ = _inputs(torch, dev, rows, vocab, 12, dtype, 5, ldp=3)
    other = teacher.float() if dtype == "bf16" else teacher.bfloat16()
    ref = reference(_np(z), _np(ids), _np(other), 2.5, 0.6, _np(labels), None)
    kw = dict(tau=2.5, mix=0.6, labels=labels.int())
    total, r, _, dz = pmx.distill_loss(z, ids.int(), other, grad=True, **kw)
    _compare(torch, total, r, dz, ref, dtype == "bf16")
    buf = torch.full((rows, vocab + 6), 9.0, dtype=z.dtype, device=dev)
    pmx.distill_loss(z, ids.int(), other, out=buf[:, 1:1 + vocab], **kw)
    assert torch.equal(buf[:, 1:1 + vocab], dz) and (buf[:, :1] == 9).all() and (buf[:, 1 + vocab:] == 9).all()
    _, _, stats, _ = pmx.distill_loss(z, ids.int(), other, **kw)
    late = pmx.distill_grad(z, ids.int(), other, stats, **kw)
    _compare(torch, None, None, late, ref, dtype == "bf16")
    for split in (False, True):
        zz = torch.full((rows, vocab + 3), 9.0, dtype=z.dtype, device=dev)
        zz[:, :vocab] = z
        v = zz[:, :vocab]
        if split:
            pmx.distill_grad(v, ids.int(), other, stats, out=v, **kw)
            assert torch.equal(v, late)
        else:
            pmx.distill_loss(v, ids.int(), other, out=v, **kw)
            assert torch.equal(v, dz)
        assert (zz[:, vocab:] == 9).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("mix", [1.0, 0.5, 0.0])
@pytest.mark.parametrize("vocab", [50, 140000])
def test_masks(env, dtype, mix, vocab):
    """Ignored rows full of NaN, labels and ids outside the vocabulary, ids
    listed twice, teacher logits of -inf, masked student logits (-inf and the
    type's lowest value), rows whose mask leaves nothing."""
    torch, pmx, dev = env
    print("masks", dtype, mix, vocab, flush=True)
    inf = float("inf")
    z, ids, teacher, labels, weights = _inputs(torch, dev, 12, vocab, 8, dtype, 9)
    low = torch.finfo(z.dtype).min
    z[0] = float("nan")
    weights[0] = 0.0
    labels[1] = -100
    labels[2] = vocab
    ids[3] = -1
    ids[4, 3:] = vocab + 5
    ids[5, 1] = ids[5, 0]
    teacher[6, :7] = -inf
    teacher[7] = -inf
    keep = ids[8]
    masked = torch.full((vocab,), -inf, device=dev, dtype=z.dtype)
    masked[keep] = z[8, keep]
    masked[labels[8]] = 1.0
    z[8] = masked
    z[9] = low
    ids[10] = keep  # (weight on a place of the lowest value is a loss beyond fp32's range)
    labels[10] = labels[8]
    z[10] = torch.where(torch.isinf(masked), torch.full_like(masked, low), masked)
    z[11] = -inf
    ref = reference(_np(z), _np(ids), _np(teacher), 2.0, mix, _np(labels), _np(weights))
    kw = dict(tau=2.0, mix=mix, labels=labels, weights=weights)
    total, r, _, dz = pmx.distill_loss(z, ids, teacher, grad=True, **kw)
    finite = bool(torch.isfinite(dz).all()), torch.isfinite(r).tolist()
    assert finite == (True, [True] * 12)
    _compare(torch, total, r, dz, ref, dtype == "bf16")
    assert (r[0] == 0) and (dz[0] == 0).all() and (r[11] == 0) and (dz[11] == 0).all()
    _, _, stats, _ = pmx.distill_loss(z, ids, teacher, **kw)
    late = pmx.distill_grad(z, ids, teacher, stats, **kw)
    _compare(torch, None, None, late, ref, dtype == "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_and_nan(env, dtype):
    torch, pmx, dev = env
    z, ids, teacher, labels, _ = _inputs(torch, dev, 5, 400, 6, dtype, 10)
    z[0, ids[0, 2]] = -float("inf")  # the teacher has weight where the student has none
    z[1, 7] = float("nan")
    z[2, 9] = float("inf")
    teacher[3, 1] = float("nan")
    total, r, stats, dz = pmx.distill_loss(z, ids, teacher, tau=2.0, grad=True)
    assert r[0] == float("inf") and torch.isfinite(dz[0]).all() and float(dz[0, ids[0, 2]]) < 0
    assert torch.isnan(r[1:4]).all() and torch.isfinite(r[4]) and torch.isfinite(dz[4]).all()
    for t in (1, 2, 3):
        assert torch.isnan(dz[t]).any()


def test_no_rows(env):
    torch, pmx, dev = env
    z, ids = torch.empty(0, 30, device=dev), torch.empty(0, 4, dtype=torch.int64, device=dev)
    total, r, stats, dz = pmx.distill_loss(z, ids, torch.empty(0, 4, device=dev), grad=True)
    assert float(total) == 0 and r.shape == (0,) and dz.shape == (0, 30)
    total, r, stats, _ = pmx.distill_loss(z, ids, torch.empty(0, 4, device=dev))
    assert pmx.distill_grad(z, ids, torch.empty(0, 4, device=dev), stats).shape == (0, 30)


@pytest.mark.parametrize("tau,mix", [(2.0, 0.7), (1.5, 1.0), (1.0, 0.0)])
def test_gradient_against_differences(env, tau, mix):
    """Central differences along a random unit direction v with step h = 2^-4:
    the third derivative of total along v is at most sum w (mix / tau + 1 - mix)
    (softmax third cumulants, |v_j| <= 1), so the quotient is off by h^2 / 6 of
    that; fp32 noise of the total over 2 h adds 2 tb / (2 h) with tb the total's
    bound, tightened to the rows' typical error sqrt(rows) below it."""
    torch, pmx, dev = env
    rows, vocab = 24, 400
    z, ids, teacher, labels, weights = _inputs(torch, dev, rows, vocab, 16, "f32", 12, spread=2.0)
    weights /= weights.sum()
    kw = dict(tau=tau, mix=mix, labels=labels, weights=weights)
    v = torch.randn(rows, vocab, device=dev)
    v /= v.abs().max()
    h = 2.0 ** -4
    f = lambda x: float(pmx.distill_loss(x, ids, teacher, **kw)[0])
    dz = pmx.distill_loss(z, ids, teacher, grad=True, **kw)[3]
    quotient = (f(z + h * v) - f(z - h * v)) / (2 * h)
    tb = reference(_np(z), _np(ids), _np(teacher), tau, mix, _np(labels), _np(weights))[3]
    assert abs(quotient - float((dz.double() * v.double()).sum())) <= h * h / 6 * (mix / tau + 1 - mix) + tb / h


def test_same_bits_and_graph(env):
    torch, pmx, dev = env
    for rows, vocab in ((50, 2000), (3, 50000)):
        z, ids, teacher, labels, weights = _inputs(torch, dev, rows, vocab, 10, "bf16", 13)
        kw = dict(tau=2.0, mix=0.5, labels=labels, weights=weights)
        keep = []

        def call():
            total, r, _, dz = pmx.distill_loss(z, ids, teacher, grad=True, **kw)
            _, _, stats, _ = pmx.distill_loss(z, ids, teacher, **kw)
            keep[:] = [total, r, dz, stats, pmx.distill_grad(z, ids, teacher, stats, **kw)]

        call()
        torch.cuda.synchronize()
        ref = [t.clone() for t in keep]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(keep, ref))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for _ in range(3):
            for t in keep:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(keep, ref))
            x = torch.randn(300, 300, device=dev)
            float((x @ x).sum())


def test_refusals(env):
    torch, pmx, dev = env
    z, ids, teacher, labels, weights = _inputs(torch, dev, 6, 40, 5, "f32", 14)
    for bad in (lambda: pmx.distill_loss(z.half(), ids, teacher), lambda: pmx.distill_loss(z, ids.float(), teacher),
                lambda: pmx.distill_loss(z, ids, teacher.double()), lambda: pmx.distill_loss(z, ids, teacher, weights=weights.double()),
                lambda: pmx.distill_loss(z, ids, teacher, mix=0.5, labels=labels.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: pmx.distill_loss(z.t(), ids, teacher), lambda: pmx.distill_loss(z, ids[:5], teacher),
                lambda: pmx.distill_loss(z, ids, teacher[:, :4]), lambda: pmx.distill_loss(z, ids, teacher, mix=0.5, labels=labels[:5]),
                lambda: pmx.distill_loss(z, ids, teacher, weights=weights[:3]), lambda: pmx.distill_loss(z.cpu(), ids, teacher),
                lambda: pmx.distill_loss(z, ids, teacher, out=torch.empty(6, 41, device=dev)),
                lambda: pmx.distill_grad(z, ids, teacher, torch.empty(5, 3, device=dev))):
        with pytest.raises(ValueError):
            bad()
    wide = torch.zeros(6, 90, device=dev)
    for bad, code in ((lambda: pmx.distill_loss(z, ids, teacher, tau=0.0), pmx.ERR_INVALID_VALUE),
                      (lambda: pmx.distill_loss(z, ids, teacher, tau=float("nan")), pmx.ERR_INVALID_VALUE),
                      (lambda: pmx.distill_loss(z, ids, teacher, tau=float("inf")), pmx.ERR_INVALID_VALUE),
                      (lambda: pmx.distill_loss(z, ids, teacher, mix=1.5), pmx.ERR_INVALID_VALUE),
                      (lambda: pmx.distill_loss(z, ids, teacher, mix=float("nan")), pmx.ERR_INVALID_VALUE),
                      (lambda: pmx.distill_loss(z, ids, teacher, mix=0.5), pmx.ERR_INVALID_VALUE),
                      (lambda: pmx.distill_loss(z, None, None), pmx.ERR_INVALID_VALUE),
                      (lambda: pmx.distill_loss(wide[:, :40], ids, teacher, out=wide[:, 20:60]), pmx.ERR_ALIAS)):
        with pytest.raises(pmx.PmxError) as e:
            bad()
        assert e.value.code == code
    # plain cross entropy needs no teacher
    total, r, _, dz = pmx.distill_loss(z, None, None, mix=0.0, labels=labels, grad=True)
    assert torch.allclose(r, torch.logsumexp(z, 1) - z.gather(1, labels[:, None])[:, 0], atol=1e-4)
    # the C ABI: nothing is enqueued on an error
    q = pmx._distill_problem(z, ids, teacher, 1.0, 1.0, None, None)
    out = torch.full((7,), 5.0, device=dev)
    import ctypes

    def loss(total=out.data_ptr(), rows=out.data_ptr() + 4):
        return pmx.lib.pmx_distill_loss(pmx.handle(0), ctypes.byref(q), rows, total, None, None, 0, None, 0, None)

    inv = pmx.ERR_INVALID_VALUE
    assert loss(total=None) == inv and loss(rows=None) == inv and loss(total=out.data_ptr() + 1) == inv
    assert loss(total=out.data_ptr() + 4) == pmx.ERR_ALIAS
    for field, value in (("struct_version", 2), ("reserved", 1), ("dtype", 7), ("rows", -1), ("vocab", 0), ("vocab", pmx.MAX_VOCAB + 1),
                         ("top", -1), ("top", pmx.MAX_TOP + 1), ("ldz", 39), ("ld_ids", 4), ("ld_teacher", 4), ("ids_type", 2),
                         ("teacher_dtype", -1), ("z", None), ("teacher", None), ("teacher_ids", None)):
        old = getattr(q, field)
        setattr(q, field, value)
        assert loss() == inv, field
        setattr(q, field, old)
    torch.cuda.synchronize()
    assert (out == 5).all()


@pytest.mark.parametrize("rows,vocab,dtype", [(700, 4097, "f32"), (2100, 515, "bf16"), (300, 33001, "bf16"), (140, 16500, "f32"),
                                              (530, 66001, "bf16"), (270, 40003, "f32"), (131, 131100, "bf16"), (600, 7, "f32")])
@pytest.mark.parametrize("ignored", [0.0, 0.4, 1.0])
def test_many_rows(env, rows, vocab, dtype, ignored):
    """More rows than blocks, so that a block works through several, in each
    class of row length; some, or all, of the rows ignored (and full of NaN)."""
    torch, pmx, dev = env
    print("many rows", rows, vocab, dtype, ignored, flush=True)
    top = min(vocab, 6)
    z, _, teacher, labels, weights = _inputs(torch, dev, rows, vocab, 0, dtype, 31)
    ids = torch.randint(0, vocab, (rows, top), device=dev)  # some listed twice
    teacher = torch.randn(rows, top, device=dev).to(z.dtype)
    off = torch.rand(rows, device=dev) < ignored
    weights[off] = 0.0
    z[off] = float("nan")
    kw = dict(tau=2.0, mix=0.75, labels=labels, weights=weights)
    ref = reference(_np(z), _np(ids), _np(teacher), 2.0, 0.75, _np(labels), _np(weights))
    total, r, _, dz = pmx.distill_loss(z, ids, teacher, grad=True, **kw)
    _compare(torch, total, r, dz, ref, dtype == "bf16")
    total, r, stats, _ = pmx.distill_loss(z, ids, teacher, **kw)
    _compare(torch, total, r, None, ref, False)
    late = pmx.distill_grad(z, ids, teacher, stats, **kw)
    _compare(torch, None, None, late, ref, dtype == "bf16")
    inplace = z.clone()
    pmx.distill_loss(inplace, ids, teacher, out=inplace, **kw)
    assert torch.equal(inplace, dz)


@pytest.mark.parametrize("vocab,dtype", [(66001, "bf16"), (40003, "f32")])
@pytest.mark.parametrize("first", [1, 257, 600])
def test_claimed_rows_after_ignored_ones(env, vocab, dtype, first):
    """Blocks that claim their rows, each beginning with ignored ones (a padded batch's leading rows): all waves of a
    block go on with the row that it claimed."""
    torch, pmx, dev = env
    rows, top = 640, 5
    print("claimed", vocab, dtype, first, flush=True)
    z, _, teacher, labels, weights = _inputs(torch, dev, rows, vocab, 0, dtype, 37)
    ids = torch.randint(0, vocab, (rows, top), device=dev)
    teacher = torch.randn(rows, top, device=dev).to(z.dtype)
    weights[:first] = 0.0
    weights[first::3] = 0.0
    z[weights == 0] = float("nan")
    kw = dict(tau=2.0, mix=0.75, labels=labels, weights=weights)
    ref = reference(_np(z), _np(ids), _np(teacher), 2.0, 0.75, _np(labels), _np(weights))
    total, r, _, dz = pmx.distill_loss(z, ids, teacher, grad=True, **kw)
    _compare(torch, total, r, dz, ref, dtype == "bf16")
    total, r, _, _ = pmx.distill_loss(z, ids, teacher, **kw)
    _compare(torch, total, r, None, ref, False)
    pmx.distill_loss(z, ids, teacher, out=z, **kw)
    assert torch.equal(z, dz)


@pytest.mark.parametrize("rows,vocab", [(9, 300), (9, 33001), (9, 140001), (200, 700)])
@pytest.mark.parametrize("tau", [0.1, 0.3, 3.0])
def test_large_teacher_logits(env, rows, vocab, tau):
    """The teacher's logits count by their differences: a large common offset, values near the type's largest, and
    a row of nothing but its lowest value (equal shares), at temperatures that are no powers of two."""
    torch, pmx, dev = env
    print("large teacher logits", rows, vocab, tau, flush=True)
    z, ids, teacher, labels, weights = _inputs(torch, dev, rows, vocab, 7, "f32", 41)
    teacher = teacher * 0.25
    teacher[0] += 12345.0
    teacher[1] -= 98765.0
    teacher[2] = 3e38
    teacher[2, 4:] = 2e38
    teacher[3] = torch.finfo(torch.float32).min
    teacher[4] = torch.finfo(torch.float32).min
    teacher[4, 2] = 5.0
    kw = dict(tau=tau, mix=0.8, labels=labels, weights=weights)
    ref = reference(_np(z), _np(ids), _np(teacher), tau, 0.8, _np(labels), _np(weights))
    total, r, _, dz = pmx.distill_loss(z, ids, teacher, grad=True, **kw)
    _compare(torch, total, r, dz, ref, False)
    total, r, stats, _ = pmx.distill_loss(z, ids, teacher, **kw)
    _compare(torch, total, r, None, ref, False)
    _compare(torch, None, None, pmx.distill_grad(z, ids, teacher, stats, **kw), ref, False)


@pytest.mark.parametrize("rows,vocab", [(6, 300), (6, 33001), (6, 140001), (300, 515)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_teacher_part_whatever_it_holds(env, rows, vocab, dtype):
    """mix = 0: a teacher's list full of NaN and infinities changes nothing."""
    torch, pmx, dev = env
    print("no teacher part", rows, vocab, dtype, flush=True)
    z, ids, teacher, labels, weights = _inputs(torch, dev, rows, vocab, 7, dtype, 43)
    ids[1, 2] = labels[1]
    teacher[0:3] = float("nan")
    teacher[3] = float("inf")
    teacher[4] = -float("inf")
    kw = dict(tau=3.0, mix=0.0, labels=labels, weights=weights)
    ref = reference(_np(z), None, None, 3.0, 0.0, _np(labels), _np(weights))
    total, r, _, dz = pmx.distill_loss(z, ids, teacher, grad=True, **kw)
    _compare(torch, total, r, dz, ref, dtype == "bf16")
    total, r, stats, _ = pmx.distill_loss(z, ids, teacher, **kw)
    _compare(torch, total, r, None, ref, False)
    _compare(torch, None, None, pmx.distill_grad(z, ids, teacher, stats, **kw), ref, dtype == "bf16")


def test_smallest_temperatures(env):
    """Down to 2^-100 the softmax is the largest logit's alone, with finite results; below, tau is refused."""
    torch, pmx, dev = env
    z, ids, teacher, labels, weights = _inputs(torch, dev, 6, 500, 5, "f32", 47)
    kw = dict(mix=0.5, labels=labels, weights=weights)
    total, r, _, dz = pmx.distill_loss(z, ids, teacher, tau=2.0 ** -100, grad=True, **kw)
    _compare(torch, total, r, dz, reference(_np(z), _np(ids), _np(teacher), 2.0 ** -100, 0.5, _np(labels), _np(weights)), False)
    for tau in (2.0 ** -101, 1e-38, 1e-42, -1.0):
        with pytest.raises(pmx.PmxError) as e:
            pmx.distill_loss(z, ids, teacher, tau=tau, **kw)
        assert e.value.code == pmx.ERR_INVALID_VALUE
