"""A small mixture-of-experts student learns from a teacher's top logits.

    tokens -> embedding -> one expert each (SiLU between two products) + the
    embedding -> head -> distillation loss

forward_backward() is one pass with its gradients, all products through
grouped_product and grouped_outer (the head is one group).  train() takes
them to the optimizers: the experts' gradients are orthogonalised by polar
(Muon), the table and the head go through a Shampoo plan.

    python examples/moe_distill.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from preconditioned_optimizer_matrix_amd import pmx  # noqa: E402


def make(vocab=2000, dim=128, hidden=256, experts=8, seed=0, device="cuda"):
    """fp32 parameters: the table, the experts' two matrices (out x in), the head."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5

    return {"table": normal(vocab, dim), "up": normal(experts, hidden, dim), "down": normal(experts, dim, hidden),
            "head": normal(vocab, dim)}


def route(ids, experts):
    """Order of the tokens by expert, and the experts' row offsets: token i goes to expert i mod experts."""
    which = ids % experts
    order = torch.sort(which, stable=True).indices
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(torch.bincount(which, minlength=experts), 0)
    return order, offsets


def forward_backward(params, ids, batch, dtype=torch.bfloat16, tau=2.0, mix=0.75, padding_idx=-1):
    """Loss and fp32 gradients of one batch.  batch: the teacher's ids and
    logits (tokens x top), labels and weights of the tokens."""
    table, up, down, head = (params[k].to(dtype) for k in ("table", "up", "down", "head"))
    vocab, dim = table.shape
    scale = dim ** 0.5
    order, groups = route(ids, up.shape[0])
    ids = ids[order]
    top_ids, top, labels, weights = (t[order] for t in batch)
    one = torch.tensor([0, ids.numel()], dtype=torch.int32, device=ids.device)

    x = pmx.embedding(table, ids, scale=scale)
    h = pmx.grouped_product(x, up, groups, trans_b=True)
    gate = torch.sigmoid(h)
    a = h * gate
    u = x + pmx.grouped_product(a, down, groups, trans_b=True)
    z = pmx.grouped_product(u, head[None], one, trans_b=True)
    # the logits' gradient takes the logits' place
    total, _, _, dz = pmx.distill_loss(z, top_ids, top, tau=tau, mix=mix, labels=labels, weights=weights, out=z)

    f32 = torch.float32
    d_head = pmx.grouped_outer(dz, u, one, out_dtype=f32)[0]
    du = pmx.grouped_product(dz, head[None], one)
    d_down = pmx.grouped_outer(du, a, groups, out_dtype=f32)
    dh = pmx.grouped_product(du, down, groups) * (gate + a * (1 - gate))
    d_up = pmx.grouped_outer(dh, x, groups, out_dtype=f32)
    dx = du + pmx.grouped_product(dh, up, groups)
    d_table = pmx.embedding_grad(dx, ids, vocab, scale=scale, padding_idx=padding_idx, out_dtype=f32)
    return total, {"table": d_table, "up": d_up, "down": d_down, "head": d_head}


def teacher_batch(tokens, vocab, top, seed, device="cuda"):
    """Tokens, and a teacher that has one fixed opinion of every token."""
    g = torch.Generator(device=device).manual_seed(seed)
    ids = torch.randint(0, vocab, (tokens,), generator=g, device=device)
    step = torch.arange(top, device=device)
    top_ids = (ids[:, None] * 7 + 1 + step * (vocab // top)) % vocab
    top = 6.0 - 0.5 * step.float().expand(tokens, top)
    weights = torch.full((tokens,), 1.0 / tokens, device=device)
    return ids, (top_ids, top.contiguous(), top_ids[:, 0].contiguous(), weights)


def train(steps=30, tokens=2048, top=16, lr=0.05, device="cuda"):
    params = make(device=device)
    vocab = params["head"].shape[0]
    plan = pmx.ShampooPlan([tuple(params["table"].shape), tuple(params["head"].shape)], device,
                           pmx.shampoo_config(lr=lr))
    losses = []
    for t in range(1, steps + 1):
        ids, batch = teacher_batch(tokens, vocab, top, t, device)
        total, grads = forward_backward(params, ids, batch)
        plan.step([params["table"], params["head"]], [grads["table"], grads["head"]], t)
        for name in ("up", "down"):
            step, _ = pmx.polar(grads[name])
            params[name] -= lr * step
        losses.append(total)
    return [float(v) for v in losses]


if __name__ == "__main__":
    for i, v in enumerate(train()):
        print("step %2d  loss %.4f" % (i + 1, v))
