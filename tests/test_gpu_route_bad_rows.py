"""Router: rows of NaN or +inf without any loss term."""
import math

import pytest

from test_gpu_route import env  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,experts", [(20, 40), (200, 40), (70001, 32), (300, 700)])
def test_bad_rows_make_the_loss_nan_whatever_its_terms(env, rows, experts):  # noqa: F811
    torch, pmx = env
    print("route, bad rows", rows, experts, flush=True)
    z = torch.randn(rows, experts, device="cuda")
    for balance, zloss in ((0.0, 0.0), (0.1, 0.0), (0.0, 0.1)):
        clean = pmx.route(z, 4, balance=balance, zloss=zloss)
        assert bool(clean.loss.isfinite()) and (float(clean.loss) == 0 or balance or zloss)
        for value in (math.nan, math.inf):
            bad = z.clone()
            bad[rows // 2, 3] = value
            r = pmx.route(bad, 4, balance=balance, zloss=zloss)
            assert bool(r.loss.isnan()), (balance, zloss, value)
            dz = pmx.route_grad(bad, r, balance=balance, zloss=zloss)
            assert bool(dz[rows // 2].isnan().all())
            # not live: it does not count
            live = torch.ones(rows, dtype=torch.bool, device="cuda")
            live[rows // 2] = False
            assert bool(pmx.route(bad, 4, live=live, balance=balance, zloss=zloss).loss.isfinite())
    # a z-loss beyond fp32 is no reason for NaN where it has no weight
    z[1] = 3e38
    assert float(pmx.route(z, 4).loss) == 0.0
