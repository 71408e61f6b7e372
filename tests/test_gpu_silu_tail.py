"""silu and its gradient in fp32 where exp(-|x|) is small, element by element.

Tolerances (u = 2^-24), relative and independent of x: with t = exp(-|x|), the exponential is off by at most 4 u, 1 + t
by 1 u and half of t's, its reciprocal by 2 u, their product by 1 u: s and 1 - s by at most 10 u.  x s and x s u round
once each: 12 u.  The slope s (1 + x (1 - s)) is off by at most 18 u s (1 + |x| (1 - s)) with the products by u and dA.
Results below fp32's normal numbers may be 0, and so may exp(-|x|) below 2^-126, the least that the exponential
instruction returns (|x| > 87.3, which 8 bits make of 86: 88): s is then off by less than 2^-126, x s by |x| 2^-126, the
slope by (1 + |x|) 2^-126, and what they are multiplied by."""
import math

import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def env():
    import torch
    from preconditioned_optimizer_matrix_amd import pmx
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    return torch, pmx


def _parts(torch, x):
    t = torch.exp(-x.abs())
    s = torch.where(x >= 0, torch.ones_like(t), t) / (1 + t)
    c = torch.where(x >= 0, t, torch.ones_like(t)) / (1 + t)
    return s, c


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("cols", [1, 130, 515, 4096])
def test_every_size_of_x(env, cols, gated):
    torch, pmx = env
    print("silu tail", cols, gated, flush=True)
    g = torch.Generator().manual_seed(cols)
    rows = 24
    x = torch.rand(rows, cols, generator=g) * 126 - 86  # -86 .. 40
    x[1] = torch.rand(cols, generator=g) * 2 - 1
    x[2] *= 1e-3
    x[3] = -86.0
    up = torch.randn(rows, cols, generator=g) if gated else torch.ones(rows, cols)
    h = torch.cat([x, up], 1) if gated else x
    da = torch.randn(rows, cols, generator=g)
    a, q, s = pmx.silu_checkpoint(h.cuda(), gated=gated)
    sg, _ = _parts(torch, x.double())
    want = x.double() * sg * up.double()
    err = (a.double().cpu() - want).abs()
    assert bool((err <= 12 * U * want.abs() + TINY).all()), float((err / (want.abs() + TINY)).max() / U)
    wide = -(-cols // 128) * 128
    kept = pmx.fp8_load(q[:, :wide], s[:, : wide // 128], cols, dtype=torch.float32).double().cpu()
    ku = pmx.fp8_load(q[:, wide:], s[:, wide // 128:], cols, dtype=torch.float32).double().cpu() if gated else torch.ones_like(kept)
    dh, again = pmx.silu_checkpoint_grad(da.cuda(), q, s, gated=gated)
    dh, again, d = dh.double().cpu(), again.double().cpu(), da.double()
    sg, c = _parts(torch, kept)
    y = kept * sg
    low = (1 + kept.abs()) * TINY  # of s below 2^-126
    assert bool(((again - y * ku).abs() <= 12 * U * (y * ku).abs() + low * ku.abs() + TINY).all())
    slope = sg * (1 + kept * c)
    tol = (18 * U * sg * (1 + kept.abs() * c) + low) * (d * ku).abs() + TINY
    err = (dh[:, :cols] - d * ku * slope).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    if gated:
        assert bool(((dh[:, cols:] - d * y).abs() <= 12 * U * (d * y).abs() + low * d.abs() + TINY).all())


def test_ends(env):
    """Far out silu is 0 and x, its slope 0 and 1; NaN stays."""
    torch, pmx = env
    x = torch.tensor([[-1e30, -3e3, -200.0, 0.0, -0.0, 90.0, 1e4, 3e38]], device="cuda")
    a, _, _ = pmx.silu_checkpoint(x)
    assert a[0].tolist() == [0.0, 0.0, 0.0, 0.0, 0.0, 90.0, 1e4, float(x[0, 7])]
    for v, slope in ((-256.0, 0.0), (0.0, 0.5), (256.0, 1.0)):
        h = torch.full((1, 8), v, device="cuda")
        _, q, s = pmx.silu_checkpoint(h)
        dh, _ = pmx.silu_checkpoint_grad(torch.ones_like(h), q, s)
        assert bool((dh == slope).all()), v
    h = torch.full((2, 8), math.nan, device="cuda")
    a, q, s = pmx.silu_checkpoint(h)
    dh, again = pmx.silu_checkpoint_grad(torch.ones_like(h), q, s)
    assert bool(a.isnan().all()) and bool(dh.isnan().all()) and bool(again.isnan().all())
