"""The loss operators, the activation checkpoints and the optimizer step together, as the example runs them."""
import math
import os
import sys

import pytest
import torch

import clip_tensor_adamw_gb300 as mica

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import preference_step  # noqa: E402


def test_example_learns():
    losses = preference_step.run(steps=12, pairs=4, length=40, width=128, vocab=1009, lr=1e-3)
    # the first step's policy is the reference but for the activations' rounding: log 2
    assert abs(losses[0] - math.log(2.0)) < 0.02
    assert losses[-1] < 0.2 * losses[0] and all(math.isfinite(v) for v in losses)


def test_gradients_against_autograd():
    """One step's weight gradients against autograd in float64 through the same bfloat16 weights. Differences: bfloat16
    activations and gradients (2^-9 each, a handful of them in a row) and the checkpoints' half steps (at most 1/127 of a
    block's largest, some 1/300 of a typical value's root mean square): under 2% of a gradient's norm."""
    model = preference_step.Block(128, 1009)
    x, y, ends = preference_step.make_batch(4, 40, 128, 1009)
    ref = mica.mica_token_logps(model.forward(x), y) + 0.05 * torch.randn(x.shape[0], device="cuda")
    logits = model.forward(x, keep=True)
    r = mica.mica_preference_loss(logits, y, ends, ref, beta=0.1)
    model.backward(r.dlogits)
    w1, w2, w3 = (w.double().requires_grad_() for w in model.half)
    xd = x.double()
    z = xd + torch.nn.functional.gelu(xd @ w1, approximate="tanh") @ w2
    lp = torch.log_softmax(z @ w3, 1).gather(1, y.clamp(min=0)[:, None])[:, 0]
    d = torch.where(y >= 0, lp - ref.double(), 0.0)
    e = ends.tolist()
    s = torch.stack([d[a:b].sum() for a, b in zip(e[:-1], e[1:])])
    loss = -torch.nn.functional.logsigmoid(0.1 * (s[0::2] - s[1::2])).mean()
    want = torch.autograd.grad(loss, (w1, w2, w3))
    for got, g in zip(model.g, want):
        assert (got.double() - g).norm() < 0.02 * g.norm()
