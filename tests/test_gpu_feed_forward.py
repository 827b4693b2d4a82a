"""The gated feed-forward block of examples/gated_feed_forward.py: its parts work together.

Each NVFP4 operand is off by at most a quarter of a value's own size (half of E2M1's largest relative step,
1/3 of the way, and the E4M3 block scale's 2^-4), in the root mean square below a tenth; a gradient here
passes up to six quantized operands, so its error stays below half of it, a cosine above 0.86."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_feed_forward.py")
    spec = importlib.util.spec_from_file_location("gated_feed_forward", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def cosine(a, b):
    return float((a.double().flatten() @ b.double().flatten()) / (a.double().norm() * b.double().norm()))


def test_one_step_against_autograd_and_tokens():
    m = example()
    T, H, F = 512, 512, 768
    block = m.GatedFeedForward(H, F)
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16)
    dy = (torch.randn((T, H), generator=g) * 0.01).to(torch.bfloat16)
    y, saved = block.forward(x.cuda(), 7)
    dx, d1, d2 = block.backward(dy.cuda(), saved, 7)
    w1, w2 = block.w1.cpu().requires_grad_(), block.w2.cpu().requires_grad_()
    xr = x.float().requires_grad_()
    p = xr @ w1.t()
    want = (torch.nn.functional.silu(p[:, :F]) * p[:, F:]) @ w2.t()
    want.backward(dy.float())
    for got, ref, name in ((y, want, "y"), (dx, xr.grad, "dx"), (d1, w1.grad, "d_w1"), (d2, w2.grad, "d_w2")):
        assert cosine(got.cpu(), ref.detach()) > 0.86, name
    # a token from the quantized weights, itself not quantized
    assert cosine(block.token(x[:3].cuda()).cpu(), want[:3].detach()) > 0.86
    assert cosine(block.token(x[:1].cuda()).cpu(), want[:1].detach()) > 0.86


def test_clipped_steps_follow_a_target():
    m = example()
    block, target = m.GatedFeedForward(512, 768), m.GatedFeedForward(512, 768, seed=1)
    g = torch.Generator().manual_seed(4)
    losses = []
    for i in range(12):
        x = torch.randn((1024, 512), generator=g).to(torch.bfloat16).cuda()
        y, saved = block.forward(x, i)
        err = y.float() - target.forward(x, i)[0].float()
        losses.append(float(err.square().mean()))
        _, *grads = block.backward((err / 1024).to(torch.bfloat16), saved, i)
        before = [t.clone() for t in grads]
        norm = block.step(grads, lr=2.0, max_norm=1.0)
        n = sum(float(t.double().square().sum()) for t in before) ** 0.5
        assert abs(float(norm) - n) <= 1e-6 * n
        assert sum(float(t.double().square().sum()) for t in grads) ** 0.5 <= 1.0 + 1e-6
    assert losses[-1] < losses[0]
