"""Products of 8-bit values: each kernel at the shapes that its rules give it, which `form` states, so that a change of
the rules cannot drop a case without notice: few rows over many columns, a column tail of the 128 x 128 tiles, all
rows in one of many groups, rows in no group, and neighbours full of NaN."""
import pytest

from test_gpu_fp8 import _check, env  # noqa: F401  (the fixture)
from test_gpu_fp8_sums import form, units

pytestmark = pytest.mark.gpu

OWN, SHARED = "stream, own columns", "stream, shared"
CASES = [
    # kind, rows, k, n, groups, type, offsets (None: uneven)
    (OWN, 16, 1100, 4099, 32, "bfloat16", None), (OWN, 16, 1100, 4099, 32, "float32", None),
    (OWN, 33, 130, 4096, 32, "bfloat16", None), (OWN, 33, 130, 4096, 32, "float32", None),
    (OWN, 33, 1100, 4099, 32, "bfloat16", [0] * 8 + [33] * 25), (OWN, 33, 1100, 4099, 32, "float32", [0] * 8 + [33] * 25),
    (OWN, 33, 600, 4099, 32, "bfloat16", [3] * 5 + [25] * 10 + [31] * 18), (OWN, 33, 600, 4099, 32, "float32", [3] * 5 + [25] * 10 + [31] * 18),
    (OWN, 250, 1100, 4099, 16, "float32", None), (OWN, 250, 1100, 4099, 16, "float32", [0] * 3 + [250] * 14),
    (OWN, 2000, 384, 100, 1000, "bfloat16", [0] * 999 + [2000] * 2), (OWN, 1, 128, 33000, 1, "bfloat16", [0, 1]),
    (SHARED, 40, 1100, 65, 40, "bfloat16", [0] * 40 + [40]), (SHARED, 40, 1100, 65, 40, "float32", [1] * 20 + [39] * 21),
    (SHARED, 100, 4096, 1001, 8, "bfloat16", [0] * 8 + [100]), (SHARED, 5, 128, 20, 1, "float32", [0, 5]),
    ("64", 600, 300, 515, 8, "bfloat16", [0] * 8 + [600]), ("64", 600, 300, 515, 8, "float32", [0] * 8 + [600]),
    ("64", 300, 640, 130, 2, "bfloat16", [17, 17, 251]), ("64", 4000, 200, 1300, 64, "float32", None),
    ("128", 3000, 384, 1300, 4, "bfloat16", None), ("128", 3000, 384, 1300, 4, "float32", None),
    ("128", 3000, 300, 1217, 4, "bfloat16", [5, 700, 700, 701, 2990]), ("128", 3000, 300, 1217, 4, "float32", [5, 700, 700, 701, 2990]),
    ("128", 3000, 300, 1217, 16, "bfloat16", [0] * 9 + [3000] * 8), ("128", 1200, 600, 2003, 30, "bfloat16", None),
    ("256", 9000, 640, 2304, 30, "bfloat16", [0] * 12 + [9000] * 19), ("256", 9000, 520, 2500, 30, "bfloat16", None),
]


def _cuts(torch, rows, groups, seed):
    g = torch.Generator().manual_seed(seed)
    return [0] + torch.sort(torch.randint(0, rows + 1, (groups - 1,), generator=g))[0].tolist() + [rows]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_each_kernel(env, case):  # noqa: F811
    torch, pmx = env
    kind, rows, k, n, groups, out, cuts = CASES[case]
    print("fp8 forms", CASES[case][:6], flush=True)
    assert form(rows, k, n, groups, out, units(torch)) == kind
    cuts = cuts or _cuts(torch, rows, groups, case)
    assert len(cuts) == groups + 1
    g = torch.Generator(device="cuda").manual_seed(case)
    dt = getattr(torch, out)
    x = torch.randn(rows, k, generator=g, device="cuda") * torch.exp2(torch.randint(-6, 6, (rows, 1), generator=g, device="cuda").float())
    w = torch.randn(groups, n, k, generator=g, device="cuda") * torch.exp2(torch.randint(-6, 6, (groups, 1, 1), generator=g, device="cuda").float())
    y = _check(env, x.to(dt), w.to(dt), cuts, dt)
    assert bool((y[:cuts[0]] == 0).all()) and bool((y[cuts[-1]:] == 0).all())


@pytest.mark.parametrize("case", [0, 1, 6, 7, 8, 13, 18, 22, 23, 26])
def test_neighbours_do_not_enter(env, case):  # noqa: F811
    """The operands inside buffers of NaN, the result inside one that stays as it was."""
    torch, pmx = env
    kind, rows, k, n, groups, out, cuts = CASES[case]
    print("fp8 neighbours", CASES[case][:6], flush=True)
    dt = getattr(torch, out)
    cuts = cuts or _cuts(torch, rows, groups, case)
    off = torch.tensor(cuts, dtype=torch.int64, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(case)
    x = torch.randn(rows, k, generator=g, device="cuda").to(dt)
    w = torch.randn(groups, n, k, generator=g, device="cuda").to(dt)
    xq, xs = pmx.fp8_store(x)
    wq, ws = pmx.fp8_store_weight(w)
    want = pmx.fp8_product(xq, xs, wq, ws, off, out_dtype=dt)
    kp, kb, sn = xq.shape[1], xs.shape[1], ws.shape[1]
    e4 = torch.float8_e4m3fn
    bx = torch.full((rows + 3, kp + 48), 0x7F, dtype=torch.uint8, device="cuda")
    sx = torch.full((rows + 2, kb + 3), 255, dtype=torch.uint8, device="cuda")
    bw = torch.full((groups, n + 2, kp + 32), 0x7F, dtype=torch.uint8, device="cuda")
    sw = torch.full((groups, sn + 1, kb + 3), 255, dtype=torch.uint8, device="cuda")
    bx[1:1 + rows, 16:16 + kp], sx[1:1 + rows, 2:2 + kb] = xq.view(torch.uint8), xs
    bw[:, 1:1 + n, 16:16 + kp], sw[:, :sn, 1:1 + kb] = wq.view(torch.uint8), ws
    buf = torch.full((rows + 2, n + 5), 3.0, dtype=dt, device="cuda")
    got = pmx.fp8_product(bx.view(e4)[1:1 + rows, 16:16 + kp], sx[1:1 + rows, 2:2 + kb], bw.view(e4)[:, 1:1 + n, 16:16 + kp],
                          sw[:, :sn, 1:1 + kb], off, out=buf[1:1 + rows, 3:3 + n])
    assert torch.equal(got, want) and bool(want.isfinite().all())
    buf[1:1 + rows, 3:3 + n] = 3.0
    assert bool((buf == 3).all())
