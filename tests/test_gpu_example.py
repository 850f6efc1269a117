"""examples/train_step.py: the operators and the all-reduce together."""
import importlib.util
import os

import pytest
import torch

import ring_all_reduce_allreduce_amd as rs
from tests._gpu import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("train_step", os.path.join(ROOT, "examples", "train_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_training_lowers_the_loss_and_keeps_the_ranks_equal(ex):
    for dtype in (torch.float32, torch.bfloat16):
        say(f"train {dtype}")
        losses, norms, group = ex.train(ranks=3, steps=8, tokens=64, width=256, hidden=384, blocks=2, dtype=dtype)
        assert losses[-1] < losses[0] - 0.005, losses
        assert all(n > 0 for n in norms)
        for r in group[1:]:
            assert all(torch.equal(a, b) for a, b in zip(group[0].weights, r.weights))


def test_gradients_equal_autograd(ex):
    """One rank's gradients in fp32 against torch's autograd of the same
    network in 64 bits. Every product is a library matrix product in fp32 over
    at most 384 terms, and four layers of them follow one another: 1e-4 of the
    largest gradient is 800 roundings."""
    width, hidden, tokens = 256, 384, 64
    rank = ex.Rank(width, hidden, 2, torch.float32)
    gen = torch.Generator().manual_seed(3)
    x = torch.empty(tokens, width).normal_(generator=gen)
    target = torch.empty(tokens, width).normal_(generator=gen)
    loss = rank.forward_backward(x.cuda(), target.cuda())
    ws = [w.double().cpu().requires_grad_() for w in rank.weights]

    def norm(h, w):
        return h / torch.sqrt(h.square().mean(-1, keepdim=True) + ex.EPS) * w

    h = x.double()
    for i in range(2):
        gain, up, down = ws[3 * i:3 * i + 3]
        h = h + torch.nn.functional.silu(norm(h, gain) @ up) @ down
    want = 0.5 * (norm(h, ws[-1]) - target.double()).square().mean()
    want.backward()
    assert abs(float(loss) - float(want.detach())) < 1e-5 * float(want.detach())
    for got, w in zip(rank.grads, ws):
        assert float((got.double().cpu() - w.grad).abs().max()) <= 1e-4 * float(w.grad.abs().max())


def test_serving_form(ex):
    rank = ex.Rank(512, 64, 1, torch.bfloat16)
    token = torch.randn(1, 512, device="cuda").bfloat16()
    q, scales, read = ex.serve_one(rank, token)
    assert q.dtype is torch.float8_e4m3fn and scales.shape == (1, 4)
    plain = rs.rms_norm(token, rank.last, eps=ex.EPS).out.float()
    # half a step of e4m3 and of bf16, or half the smallest e4m3 step
    assert bool(((read - plain).abs() <= plain.abs() * (2.0 ** -4 + 2.0 ** -7) + float(scales.max()) * 2.0 ** -9).all())
