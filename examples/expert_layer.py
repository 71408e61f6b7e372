"""One expert layer with its products in 8 bits, forward and backward.

    x -> layer norm -> router -> the chosen experts (gated silu between two
    products) -> their results by the gates, added to x

What the backward pass needs of the experts is kept in 8 bits: their inputs,
which are the first product's operand anyway, and the hidden layer, stored as
silu reads it.  train() takes the gradients to the optimizers: the experts'
are orthogonalised by polar (Muon), the router goes through a Shampoo plan.

    python examples/expert_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from preconditioned_optimizer_matrix_amd import pmx  # noqa: E402


def make(dim=256, hidden=384, experts=8, seed=0, device="cuda"):
    """fp32 parameters: norm, router, the experts' two matrices (out x in; the first has a gate and a value half)."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5

    return {"weight": torch.ones(dim, device=device), "bias": torch.zeros(dim, device=device), "router": normal(experts, dim),
            "up": normal(experts, 2 * hidden, dim), "down": normal(experts, dim, hidden)}


def to_8bit(params):
    """The experts' weights as both passes take them: (values, scales), and of the transposed."""
    return {k: (pmx.fp8_store_weight(params[k]), pmx.fp8_store_weight(params[k], transposed=True)) for k in ("up", "down")}


def forward(params, weights, x, top=2, balance=1e-2, zloss=1e-3, live=None):
    """(y, loss of the router, what backward needs)."""
    one = torch.tensor([0, x.shape[0]], dtype=torch.int32, device=x.device)
    n, stats = pmx.layer_norm(x, params["weight"], params["bias"])
    z = pmx.grouped_product(n, params["router"].to(x.dtype)[None], one, trans_b=True, out_dtype=torch.float32)
    kw = dict(live=live, balance=balance, zloss=zloss)
    r = pmx.route(z, top, **kw)
    rows = pmx.fp8_store(pmx.embedding(n, r.tokens))  # of the pairs, by expert; zeros behind the last
    h = pmx.fp8_product(*rows, *weights["up"][0], r.offsets, out_dtype=x.dtype)
    a, *hidden = pmx.silu_checkpoint(h, gated=True)
    o = pmx.fp8_product(*pmx.fp8_store(a), *weights["down"][0], r.offsets, out_dtype=x.dtype)
    mixed = pmx.embedding(o, r.slots).float() * r.gates[:, :, None]  # slots of -1 give zeros
    y = x + mixed.sum(1).to(x.dtype)
    return y, r.loss, (x, stats, z, r, rows, hidden, o, kw, one)


def backward(params, weights, saved, dy, upstream=None):
    """(dx, gradients): of sum(y dy) + upstream (default 1) times the router's loss."""
    x, stats, z, r, rows, hidden, o, kw, one = saved
    f32 = torch.float32
    dim = x.shape[1]
    dgates = (pmx.embedding(o, r.slots).float() * dy.float()[:, None]).sum(2)
    # each row's gate, and its share of dy
    gate = torch.zeros(r.tokens.numel() + 1, device=x.device)
    gate[torch.where(r.slots < 0, r.tokens.numel(), r.slots).long().flatten()] = r.gates.flatten()
    do = (pmx.embedding(dy, r.tokens).float() * gate[:-1, None]).to(x.dtype)
    da = pmx.fp8_product(*pmx.fp8_store(do), *weights["down"][1], r.offsets, out_dtype=x.dtype)
    dh, a = pmx.silu_checkpoint_grad(da, *hidden, gated=True)
    d_down = pmx.grouped_outer(do, a, r.offsets, out_dtype=f32)
    d_rows = pmx.fp8_product(*pmx.fp8_store(dh), *weights["up"][1], r.offsets, out_dtype=x.dtype)
    d_up = pmx.grouped_outer(dh, pmx.fp8_load(*rows, dim, dtype=x.dtype), r.offsets, out_dtype=f32)
    dz = pmx.route_grad(z, r, dgates, upstream=upstream, **kw).to(x.dtype)
    # a token's rows add up as the rows of a table do
    dn = pmx.embedding_grad(d_rows, r.tokens, x.shape[0], out_dtype=f32)
    dn = (dn + pmx.grouped_product(dz, params["router"].to(x.dtype)[None], one, out_dtype=f32)).to(x.dtype)
    n, _ = pmx.layer_norm(x, params["weight"], params["bias"])
    d_router = pmx.grouped_outer(dz, n, one, out_dtype=f32)[0]
    dx, dw, db = pmx.layer_norm_grad(dn, x, stats, params["weight"])
    return dx + dy, {"weight": dw, "bias": db, "router": d_router, "up": d_up, "down": d_down}


def train(steps=20, tokens=1024, lr=0.05, device="cuda"):
    """The layer learns what another one computes; the mean squared difference of each step."""
    params, other = make(device=device), make(seed=1, device=device)
    target = to_8bit(other)
    plan = pmx.ShampooPlan([tuple(params["router"].shape)], device, pmx.shampoo_config(lr=lr))
    losses = []
    for t in range(1, steps + 1):
        g = torch.Generator(device=device).manual_seed(t)
        x = torch.randn(tokens, params["router"].shape[1], generator=g, device=device).bfloat16()
        weights = to_8bit(params)
        want, _, _ = forward(other, target, x)
        y, _, saved = forward(params, weights, x)
        diff = y.float() - want.float()
        _, grads = backward(params, weights, saved, (diff * (2.0 / diff.numel())).bfloat16())
        plan.step([params["router"]], [grads["router"]], t)
        for name in ("up", "down"):
            step, _ = pmx.polar(grads[name])
            params[name] -= lr * step
        for name in ("weight", "bias"):
            params[name] -= lr * grads[name]
        losses.append(diff.square().mean())
    return [float(v) for v in losses]


if __name__ == "__main__":
    for i, v in enumerate(train()):
        print("step %2d  loss %.5f" % (i + 1, v))
