"""Products grouped by expert against a plain fp64 implementation.

Tolerance, per element: the kernel adds K products in fp32 in some fixed
order, so its sum is off by at most (K + 2) 2^-24 sum |a| |b| (the textbook
bound of a K-term sum with exact or once-rounded products); a bf16 result
adds its rounding (8 significant bits), 2^-8 of the value, an accumulated one the rounding of the
addition."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    from preconditioned_optimizer_matrix_amd import pmx
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    return torch, pmx, dev


def _offsets(rows, groups, seed, first=0, last=None):
    """Uneven groups over [first, last), some of them empty."""
    rng = np.random.default_rng(seed)
    last = rows if last is None else last
    cuts = np.sort(rng.integers(first, last + 1, groups - 1)) if groups > 1 else np.empty(0, int)
    if groups > 3:
        cuts[1] = cuts[0]  # an empty group
    return np.concatenate([[first], cuts, [last]]).astype(np.int64)


def _bound(val, absum, k, bf16_out):
    return (k + 2) * 2.0 ** -24 * absum + (2.0 ** -8 * (1 + 1e-6) * np.abs(val) if bf16_out else 2.0 ** -24 * np.abs(val)) + 1e-37


def _ref_product(A, B, off, trans):
    C = np.zeros((A.shape[0], B.shape[1] if trans else B.shape[2]))
    S = np.zeros_like(C)
    for e in range(B.shape[0]):
        a, b = off[e], off[e + 1]
        W = B[e].T if trans else B[e]
        C[a:b] = A[a:b] @ W
        S[a:b] = np.abs(A[a:b]) @ np.abs(W)
    return C, S


def _make(torch, dev, dtype, shape, seed, pad=0):
    """Seeded values of `dtype` as (device view of row distance cols + pad, fp64 values)."""
    g = torch.Generator().manual_seed(seed)
    full = torch.randn(*shape[:-1], shape[-1] + pad, generator=g).to(dtype)
    v = full.to(dev)[..., :shape[-1]]
    return v, full[..., :shape[-1]].double().numpy()


# rows, groups, k, n: one row; sides under a 16-byte piece; odd sides; tiles
# filled exactly and by one more; groups of every size class
SIZES = [(1, 1, 1, 1), (3, 2, 5, 3), (17, 4, 64, 128), (40, 5, 33, 129), (100, 3, 65, 7),
         (257, 2, 200, 136), (300, 2, 129, 515), (1000, 6, 72, 264), (31, 300, 48, 40)]


@pytest.mark.parametrize("rows,groups,k,n", SIZES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("trans", [True, False])
def test_product(env, rows, groups, k, n, dtype, out, trans):
    torch, pmx, dev = env
    dts = {"bf16": torch.bfloat16, "f32": torch.float32}
    print("product", rows, groups, k, n, dtype, out, trans, flush=True)
    off = _offsets(rows, groups, rows + k)
    A, An = _make(torch, dev, dts[dtype], (rows, k), 1)
    B, Bn = _make(torch, dev, dts[dtype], (groups, n, k) if trans else (groups, k, n), 2)
    C = pmx.grouped_product(A, B, torch.from_numpy(off).to(dev), trans_b=trans, out_dtype=dts[out])
    ref, s = _ref_product(An, Bn, off, trans)
    err = np.abs(C.double().cpu().numpy() - ref)
    assert C.dtype == dts[out]
    assert (err <= _bound(ref, s, k, out == "bf16")).all()


@pytest.mark.parametrize("rows,groups,m,n", SIZES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_outer(env, rows, groups, m, n, dtype, out, accumulate):
    torch, pmx, dev = env
    dts = {"bf16": torch.bfloat16, "f32": torch.float32}
    print("outer", rows, groups, m, n, dtype, out, accumulate, flush=True)
    off = _offsets(rows, groups, rows + m)
    A, An = _make(torch, dev, dts[dtype], (rows, m), 3)
    B, Bn = _make(torch, dev, dts[dtype], (rows, n), 4)
    C, C0 = _make(torch, dev, dts[out], (groups, m, n), 5)
    pmx.grouped_outer(A, B, torch.from_numpy(off).int().to(dev), out=C, accumulate=accumulate)
    Cn = C.double().cpu().numpy()
    for e in range(groups):
        a, b = off[e], off[e + 1]
        ref = An[a:b].T @ Bn[a:b] + (C0[e] if accumulate else 0.0)
        s = np.abs(An[a:b]).T @ np.abs(Bn[a:b]) + (np.abs(C0[e]) if accumulate else 0.0)
        assert (np.abs(Cn[e] - ref) <= _bound(ref, s, b - a + 1, out == "bf16")).all(), e


# the tile classes and the split contraction that only larger calls reach
@pytest.mark.parametrize("rows,groups,k,n", [(16384, 4, 72, 1024), (16500, 9, 136, 1030), (70, 2, 4100, 130), (200, 1, 3000, 33)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_larger_products(env, rows, groups, k, n, dtype):
    torch, pmx, dev = env
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    off = _offsets(rows, groups, 77)
    o = torch.from_numpy(off).to(dev)
    for trans in (True, False):
        print("larger product", rows, groups, k, n, dtype, trans, flush=True)
        A, An = _make(torch, dev, dt, (rows, k), 6)
        B, Bn = _make(torch, dev, dt, (groups, n, k) if trans else (groups, k, n), 7)
        C = pmx.grouped_product(A, B, o, trans_b=trans)
        ref, s = _ref_product(An, Bn, off, trans)
        assert (np.abs(C.double().cpu().numpy() - ref) <= _bound(ref, s, k, dtype == "bf16")).all()


@pytest.mark.parametrize("rows,groups,m,n", [(4200, 16, 1024, 1030), (9000, 2, 130, 96), (20000, 1, 64, 64), (5000, 40, 520, 768)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_larger_outer(env, rows, groups, m, n, dtype, accumulate):
    torch, pmx, dev = env
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    print("larger outer", rows, groups, m, n, dtype, accumulate, flush=True)
    off = _offsets(rows, groups, 78)
    A, An = _make(torch, dev, dt, (rows, m), 8)
    B, Bn = _make(torch, dev, dt, (rows, n), 9)
    C, C0 = _make(torch, dev, torch.float32, (groups, m, n), 10)
    pmx.grouped_outer(A, B, torch.from_numpy(off).to(dev), out=C, accumulate=accumulate)
    Cn = C.double().cpu().numpy()
    for e in range(groups):
        a, b = off[e], off[e + 1]
        ref = An[a:b].T @ Bn[a:b] + (C0[e] if accumulate else 0.0)
        s = np.abs(An[a:b]).T @ np.abs(Bn[a:b]) + (np.abs(C0[e]) if accumulate else 0.0)
        assert (np.abs(Cn[e] - ref) <= _bound(ref, s, b - a + 1, False)).all(), e


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("trans", [True, False])
def test_strides_and_rows_of_no_group(env, dtype, trans):
    """Padded rows at odd alignments, one weight matrix shared by all groups,
    rows before the first and after the last group, and what lies around the
    outputs stays as it was."""
    torch, pmx, dev = env
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    for rows, groups, k, n in ((150, 3, 77, 45), (900, 3, 80, 136)):
        print("strides", rows, dtype, trans, flush=True)
        off = _offsets(rows, groups, 5, first=9, last=rows - 14)
        A, An = _make(torch, dev, dt, (rows, k), 11, pad=3)
        A[:9] = float("nan")
        A[rows - 14:] = float("inf")
        W, Wn = _make(torch, dev, dt, (n, k) if trans else (k, n), 12, pad=1)
        B = W.unsqueeze(0).expand(groups, -1, -1)
        buf = torch.full((rows, n + 5), 7.0, dtype=dt, device=dev)
        C = pmx.grouped_product(A, B, torch.from_numpy(off).to(dev), trans_b=trans, out=buf[:, 2:2 + n])
        An = np.where(np.isfinite(An), An, 0.0)
        ref, s = _ref_product(An, np.broadcast_to(Wn, (groups,) + Wn.shape), off, trans)
        Cn = C.double().cpu().numpy()
        assert (Cn[:9] == 0).all() and (Cn[rows - 14:] == 0).all()
        assert (np.abs(Cn - ref) <= _bound(ref, s, k, dtype == "bf16")).all()
        assert (buf[:, :2] == 7).all() and (buf[:, 2 + n:] == 7).all()
        # the weight gradient does not see the rows of no group either
        D, Dn = _make(torch, dev, dt, (rows, n), 13, pad=1)
        D[rows - 14:] = float("nan")
        out = torch.full((groups, k + 1, n + 3), 7.0, device=dev)
        G = pmx.grouped_outer(A, D, torch.from_numpy(off).to(dev), out=out[:, :k, :n])
        Gn = G.double().cpu().numpy()
        for e in range(groups):
            a, b = off[e], off[e + 1]
            ref = An[a:b].T @ Dn[a:b]
            s = np.abs(An[a:b]).T @ np.abs(Dn[a:b])
            assert (np.abs(Gn[e] - ref) <= _bound(ref, s, b - a, False)).all(), e
        assert (out[:, k:] == 7).all() and (out[:, :, n:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_group_does_not_reach_another(env, dtype):
    """NaN in one expert's weights, or infinities in its rows, stay its own."""
    torch, pmx, dev = env
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    rows, k, n = 90, 70, 50
    off = torch.tensor([0, 31, 60, 90], device=dev)
    A = torch.randn(rows, k, device=dev).to(dt)
    B = torch.randn(3, n, k, device=dev).to(dt)
    clean = pmx.grouped_product(A, B, off, trans_b=True)
    B[1] = float("nan")
    C = pmx.grouped_product(A, B, off, trans_b=True)
    assert torch.isnan(C[31:60]).all()
    assert torch.equal(C[:31], clean[:31]) and torch.equal(C[60:], clean[60:])
    D = torch.randn(rows, n, device=dev).to(dt)
    clean = pmx.grouped_outer(A, D, off, out_dtype=torch.float32)
    A2 = A.clone()
    A2[31:60] = float("inf")
    G = pmx.grouped_outer(A2, D, off, out_dtype=torch.float32)
    assert torch.equal(G[0], clean[0]) and torch.equal(G[2], clean[2]) and not torch.isfinite(G[1]).any()


def test_offsets_out_of_order_stay_inside(env):
    """Offsets are clamped to [0, rows] and made non-decreasing."""
    torch, pmx, dev = env
    A = torch.randn(20, 16, device=dev)
    B = torch.randn(4, 16, 24, device=dev)
    for dt in (torch.int32, torch.int64):
        C = pmx.grouped_product(A, B, torch.tensor([-5, 8, 3, 50, 12], dtype=dt, device=dev))
        # groups: [0, 8), [8, 8), [8, 20), [20, 20)
        ref = torch.cat([A[:8] @ B[0], A[8:] @ B[2]])
        assert torch.allclose(C, ref, atol=1e-4)
        G = pmx.grouped_outer(A, C, torch.tensor([-5, 8, 3, 50, 12], dtype=dt, device=dev))
        assert (G[1] == 0).all() and (G[3] == 0).all()
        assert torch.allclose(G[2], A[8:].t() @ C[8:], atol=1e-2)


def test_empty(env):
    torch, pmx, dev = env
    for dt in (torch.bfloat16, torch.float32):
        A = torch.empty(0, 24, dtype=dt, device=dev)
        B = torch.randn(3, 24, 40, device=dev).to(dt)
        off = torch.zeros(4, dtype=torch.int32, device=dev)
        assert pmx.grouped_product(A, B, off).shape == (0, 40)
        G = pmx.grouped_outer(A, torch.empty(0, 40, dtype=dt, device=dev), off)
        assert G.shape == (3, 24, 40) and (G == 0).all()
        keep = torch.ones(3, 24, 40, device=dev)
        pmx.grouped_outer(A, torch.empty(0, 40, dtype=dt, device=dev), off, out=keep, accumulate=True)
        assert (keep == 1).all()


@pytest.mark.parametrize("rows,groups,k,n", [(60, 4, 40, 56), (500, 3, 136, 72)])
def test_gradients_against_differences(env, rows, groups, k, n):
    """f(X, W) = sum R * Y is linear in X and in W, so a difference quotient over
    a unit step is exact but for rounding: |f| is at most sum |R| |Y|, whose fp32
    rounding (K + 2) 2^-24 bounds the quotient's error on each side."""
    torch, pmx, dev = env
    off = _offsets(rows, groups, 21)
    o = torch.from_numpy(off).to(dev)
    X, Xn = _make(torch, dev, torch.float32, (rows, k), 14)
    W, Wn = _make(torch, dev, torch.float32, (groups, n, k), 15)
    R, Rn = _make(torch, dev, torch.float32, (rows, n), 16)
    VX, VXn = _make(torch, dev, torch.float32, (rows, k), 17)
    VW, VWn = _make(torch, dev, torch.float32, (groups, n, k), 18)
    f = lambda x, w: float((pmx.grouped_product(x, w, o, trans_b=True).double() * R.double()).sum())
    dX = pmx.grouped_product(R, W, o).double().cpu().numpy()
    dW = pmx.grouped_outer(R, X, o).double().cpu().numpy()
    size = 0.0
    for e in range(groups):
        a, b = off[e], off[e + 1]
        x = np.abs(Xn[a:b]) + np.abs(VXn[a:b])
        w = np.abs(Wn[e]) + np.abs(VWn[e])
        size += (np.abs(Rn[a:b]) * (x @ w.T)).sum()
    tol = 4 * (max(k, n, rows) + 2) * 2.0 ** -24 * size
    gx = (f(X + VX, W) - f(X - VX, W)) / 2
    gw = (f(X, W + VW) - f(X, W - VW)) / 2
    assert abs(gx - (dX * VXn).sum()) <= tol
    assert abs(gw - (dW * VWn).sum()) <= tol


def test_same_bits_and_graph(env):
    """A call gives the same bits every time, on another stream and replayed
    from a graph."""
    torch, pmx, dev = env
    off = torch.from_numpy(_offsets(700, 5, 3)).to(dev)
    A = torch.randn(700, 1100, device=dev).bfloat16()
    B = torch.randn(5, 120, 1100, device=dev).bfloat16()
    D = torch.randn(700, 120, device=dev).bfloat16()
    out, G = torch.empty(700, 120, dtype=torch.bfloat16, device=dev), torch.empty(5, 120, 1100, device=dev)
    ws1 = pmx.workspace(pmx._need("pmx_grouped_product_workspace_size", 700, 1100, 120, 5, pmx.BF16), dev)
    ws2 = pmx.workspace(pmx._need("pmx_grouped_outer_workspace_size", 700, 120, 1100, 5, pmx.BF16), dev)

    def call():
        pmx.grouped_product(A, B, off, trans_b=True, out=out, ws=ws1)
        pmx.grouped_outer(D, A, off, out=G, ws=ws2)

    call()
    torch.cuda.synchronize()
    ref = out.clone(), G.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out, ref[0]) and torch.equal(G, ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        out.zero_()
        G.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(G, ref[1])
        x = torch.randn(300, 300, device=dev)
        float((x @ x).sum())


def test_refusals(env):
    torch, pmx, dev = env
    A = torch.randn(8, 16, device=dev)
    B = torch.randn(2, 16, 12, device=dev)
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device=dev)
    for bad in (lambda: pmx.grouped_product(A, B.bfloat16(), off),
                lambda: pmx.grouped_product(A.half(), B.half(), off),
                lambda: pmx.grouped_product(A, B, off.float()),
                lambda: pmx.grouped_outer(A, B[0].bfloat16()[:8], off)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: pmx.grouped_product(A, B, off[:2]),
                lambda: pmx.grouped_product(A, B, off, trans_b=True),
                lambda: pmx.grouped_product(A.t(), B, off),
                lambda: pmx.grouped_product(A[0], B, off),
                lambda: pmx.grouped_product(A, B, off, out=torch.empty(8, 11, device=dev)),
                lambda: pmx.grouped_outer(A, A[:7], off),
                lambda: pmx.grouped_outer(A, A, off, accumulate=True),
                lambda: pmx.grouped_product(A.cpu(), B, off)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pmx.PmxError) as e:
        pmx.grouped_product(A, B, off, out_dtype=torch.bfloat16)
    assert e.value.code == pmx.ERR_NOT_SUPPORTED
    buf = torch.zeros(8, 28, device=dev)
    with pytest.raises(pmx.PmxError) as e:
        pmx.grouped_product(buf[:, :16], B, off, out=buf[:, 16:])
    assert e.value.code == pmx.ERR_ALIAS
    # through the C ABI: sizes, strides, null pointers, a workspace too small
    L, h, p = pmx.lib, pmx.handle(0), lambda t: t.data_ptr()
    C = torch.full((8, 12), 5.0, device=dev)

    def product(rows=8, k=16, lda=16, n=12, ldb=12, sb=192, trans=0, it=pmx.I32, groups=2, ldc=12, a=p(A), b=p(B),
                o=p(off), c=p(C), dt=pmx.F32, odt=pmx.F32):
        return L.pmx_grouped_product(h, a, dt, rows, k, lda, b, n, ldb, sb, trans, o, it, groups, c, odt, ldc, None, 0, None)

    inv = pmx.ERR_INVALID_VALUE
    assert product(rows=-1) == inv and product(k=0) == inv and product(n=0) == inv and product(groups=0) == inv
    assert product(groups=pmx.MAX_GROUPS + 1) == inv and product(lda=15) == inv and product(ldb=11) == inv
    assert product(ldc=11) == inv and product(sb=100) == inv and product(sb=-1) == inv and product(trans=2) == inv
    assert product(a=None) == inv and product(b=None) == inv and product(o=None) == inv and product(c=None) == inv
    assert product(it=2) == inv and product(dt=2) == inv and product(odt=5) == inv and product(a=p(A) + 1) == inv
    assert product(c=p(A)) == pmx.ERR_ALIAS and product(rows=1 << 40) == inv
    big = pmx._need("pmx_grouped_product_workspace_size", 8, 4096, 12, 2, pmx.F32)
    assert big > 0
    A2, B2 = torch.zeros(8, 4096, device=dev), torch.zeros(2, 4096, 12, device=dev)
    small = pmx.workspace(big, dev)
    args = lambda w, nb: L.pmx_grouped_product(h, p(A2), pmx.F32, 8, 4096, 4096, p(B2), 12, 12, 4096 * 12, 0, p(off),
                                               pmx.I32, 2, p(C), pmx.F32, 12, w, nb, None)
    assert args(None, 0) == pmx.ERR_WORKSPACE and args(p(small), big - 1) == pmx.ERR_WORKSPACE
    assert args(p(small) + 4, big) == pmx.ERR_WORKSPACE
    torch.cuda.synchronize()
    assert (C == 5).all()  # nothing was enqueued


@pytest.mark.parametrize("rows,groups,m,n", [(5000, 40, 520, 768), (3000, 33, 512, 1032), (2600, 65, 256, 512)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_outer_of_large_aligned_tiles(env, rows, groups, m, n, out, accumulate):
    """Large tiles of aligned operands: groups of every length modulo the k tile,
    sides that end inside a tile, both result types."""
    torch, pmx, dev = env
    print("large aligned outer", rows, groups, m, n, out, accumulate, flush=True)
    off = _offsets(rows, groups, 91)
    A, An = _make(torch, dev, torch.bfloat16, (rows, m), 21)
    B, Bn = _make(torch, dev, torch.bfloat16, (rows, n), 22)
    C, C0 = _make(torch, dev, {"bf16": torch.bfloat16, "f32": torch.float32}[out], (groups, m, n), 23)
    pmx.grouped_outer(A, B, torch.from_numpy(off).to(dev), out=C, accumulate=accumulate)
    Cn = C.double().cpu().numpy()
    for e in range(groups):
        a, b = off[e], off[e + 1]
        ref = An[a:b].T @ Bn[a:b] + (C0[e] if accumulate else 0.0)
        s = np.abs(An[a:b]).T @ np.abs(Bn[a:b]) + (np.abs(C0[e]) if accumulate else 0.0)
        assert (np.abs(Cn[e] - ref) <= _bound(ref, s, b - a + 1, out == "bf16")).all(), e


@pytest.mark.parametrize("k,n", [(2048, 1000), (2051, 1021)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_last_tiles_in_quarters(env, k, n, out):
    """A few tiles more than whole rounds: 68 rows of tiles by 4, the last ones cut, quarters of them outside."""
    torch, pmx, dev = env
    off = np.cumsum([0, 4000, 300, 0, 6000, 6500])
    rows, groups = int(off[-1]), len(off) - 1
    t = torch.from_numpy(off).to(dev)
    odt = torch.float32 if out == "f32" else torch.bfloat16
    A, a = _make(torch, dev, torch.bfloat16, (rows, k), 3)
    for trans in (True, False):
        print("quarters", k, n, out, trans, flush=True)
        B, b = _make(torch, dev, torch.bfloat16, (groups, n, k) if trans else (groups, k, n), 4)
        C = torch.full((rows, n + 3), 7.0, device=dev).to(odt)
        pmx.grouped_product(A, B, t, trans_b=trans, out=C[:, :n])
        ref, mag = _ref_product(a, b, off, trans)
        assert (np.abs(C[:, :n].double().cpu().numpy() - ref) <= _bound(ref, mag, k, out == "bf16")).all()
        assert (C[:, n:] == 7).all()


# groups of middle size: enough 128 x 128 tiles, too few larger ones; the last sizes also split the contraction
@pytest.mark.parametrize("rows,groups,k,n", [(6000, 30, 200, 1000), (5001, 21, 131, 1029), (1500, 5, 1100, 1500)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_middle_products(env, rows, groups, k, n, dtype):
    test_larger_products(env, rows, groups, k, n, dtype)


@pytest.mark.parametrize("rows,groups,m,n", [(3000, 50, 260, 390), (3001, 50, 129, 515), (2200, 2, 1200, 1201)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_middle_outer(env, rows, groups, m, n, dtype, accumulate):
    test_larger_outer(env, rows, groups, m, n, dtype, accumulate)


# 256 large tiles, where they begin to be taken, a column of tiles more, and 255 (smaller tiles)
@pytest.mark.parametrize("rows,groups,m,n", [(1100, 1, 4096, 4096), (4200, 4, 2048, 2048), (2100, 1, 4096, 4360), (2100, 1, 3840, 4344)])
@pytest.mark.parametrize("out,accumulate", [("f32", False), ("f32", True), ("bf16", False)])
def test_outer_where_large_tiles_begin(env, rows, groups, m, n, out, accumulate):
    """Long groups and as many large tiles as units: whole results, nothing read from the workspace.  Operands that
    are aligned, and rows at odd distances."""
    torch, pmx, dev = env
    off = _offsets(rows, groups, 92)
    o = torch.from_numpy(off).to(dev)
    odt = {"bf16": torch.bfloat16, "f32": torch.float32}[out]
    for pad in (0, 3):
        print("large tiles begin", rows, groups, m, n, out, accumulate, pad, flush=True)
        A, An = _make(torch, dev, torch.bfloat16, (rows, m), 24, pad=pad)
        B, Bn = _make(torch, dev, torch.bfloat16, (rows, n), 25, pad=pad)
        C, C0 = _make(torch, dev, odt, (groups, m, n), 26)
        ws = torch.full((1 << 28,), 0xFF, dtype=torch.uint8, device=dev)  # NaN
        pmx.grouped_outer(A, B, o, out=C, accumulate=accumulate, ws=ws)
        Cn = C.double().cpu().numpy()
        for e in range(groups):
            a, b = off[e], off[e + 1]
            ref = An[a:b].T @ Bn[a:b] + (C0[e] if accumulate else 0.0)
            s = np.abs(An[a:b]).T @ np.abs(Bn[a:b]) + (np.abs(C0[e]) if accumulate else 0.0)
            assert (np.abs(Cn[e] - ref) <= _bound(ref, s, b - a + 1, out == "bf16")).all(), e


@pytest.mark.parametrize("rows,groups,k,n", [(64, 64, 4096, 4096), (779, 21, 4032, 336), (900, 3, 16384, 1030), (3000, 40, 4100, 1100)])
def test_long_fp32_contractions(env, rows, groups, k, n):
    """The root mean square error of long fp32 sums.  Over n roundings of a sum of terms of random sign it is about
    2^-24 sqrt(n / 6) of the result's; sums over 128 values of k, two to a matrix instruction, joined by a second sum
    make n = 64 + K / 128.  Twice that is asked for; one chain of K / 2 would be off by 2.3 times as much at K = 4096
    and 3.3 times at 16384."""
    torch, pmx, dev = env
    print("long fp32 contraction", rows, groups, k, n, flush=True)
    off = np.linspace(0, rows, groups + 1).astype(np.int64)
    o = torch.from_numpy(off).to(dev)

    def check(got, ref, K):
        d = got.double().cpu().numpy() - ref
        tol = 2 * 2.0 ** -24 * ((64 + K / 128) / 6) ** 0.5
        assert (d ** 2).sum() ** 0.5 <= tol * (ref ** 2).sum() ** 0.5

    A, An = _make(torch, dev, torch.float32, (rows, k), 27)
    for trans in (True, False):
        B, Bn = _make(torch, dev, torch.float32, (groups, n, k) if trans else (groups, k, n), 28)
        check(pmx.grouped_product(A, B, o, trans_b=trans), _ref_product(An, Bn, off, trans)[0], k)
    # the same as rows of the outer form: one group of k rows
    one = torch.tensor([0, k], device=dev)
    check(pmx.grouped_outer(A.t().contiguous(), B[0].contiguous(), one)[0], An @ Bn[0], k)
