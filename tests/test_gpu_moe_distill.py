"""The embedding, the products grouped by expert and the distillation loss
run together: examples/moe_distill.py.

The fp32 gradients are compared with fp64 automatic differentiation of the
plain formulas.  Tolerance, relative to the largest gradient entry of each
parameter: a path has at most six products of up to K = 128 .. 500 terms, each
off by at most K 2^-24 of the sum of its terms' magnitudes, which for such
random data is about sqrt(K) times the sum itself: 6 * 500^1.5 * 2^-24 = 4e-3
at worst; rounding errors of random sign stay sqrt(K) below that, 2e-4."""
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
    spec = importlib.util.spec_from_file_location("moe_distill", os.path.join(ROOT, "examples", "moe_distill.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return torch, m


def _plain(torch, params, ids, batch, experts, tau, mix, padding_idx):
    p = {k: v.double().cpu().requires_grad_() for k, v in params.items()}
    ids = ids.cpu()
    top_ids, top, labels, weights = (t.cpu() for t in batch)
    x = p["table"][ids] * p["table"].shape[1] ** 0.5
    if padding_idx >= 0:
        x = torch.where((ids == padding_idx)[:, None], x.detach(), x)
    e = ids % experts
    h = torch.bmm(p["up"][e], x[:, :, None])[:, :, 0]
    u = x + torch.bmm(p["down"][e], torch.nn.functional.silu(h)[:, :, None])[:, :, 0]
    z = u @ p["head"].T
    q = torch.softmax(top.double() / tau, 1)
    # tau^2 KL(teacher's top || the student's softmax over the vocabulary)
    kd = tau * tau * (q * (q.log() - torch.log_softmax(z / tau, 1).gather(1, top_ids))).sum(1)
    ce = -torch.log_softmax(z, 1).gather(1, labels[:, None])[:, 0]
    total = (weights.double() * (mix * kd + (1 - mix) * ce)).sum()
    total.backward()
    return float(total), {k: v.grad for k, v in p.items()}


def test_gradients(example):
    torch, m = example
    print("moe gradients", flush=True)
    params = m.make(vocab=500, dim=64, hidden=128, experts=5, seed=1)
    ids, batch = m.teacher_batch(300, 500, 8, 2)
    total, grads = m.forward_backward(params, ids, batch, dtype=torch.float32, padding_idx=int(ids[0]))
    ref, want = _plain(torch, params, ids, batch, 5, 2.0, 0.75, int(ids[0]))
    assert abs(float(total) - ref) <= 2e-4 * abs(ref)
    for k, w in want.items():
        assert (grads[k].double().cpu() - w).abs().max() <= 2e-4 * w.abs().max(), k


def test_training_lowers_the_loss(example):
    _, m = example
    print("moe training", flush=True)
    losses = m.train(steps=20)
    assert losses[-1] < 0.9 * losses[0] and all(v == v for v in losses)
