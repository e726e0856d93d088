"""The losses from hidden states and the orthogonalised step as a training step uses them, together with the joint norm and
AdamW: the example's gradients against autograd in float64, a step's weights against the definitions, and that it runs."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_example_runs():
    import pretrain_step
    losses = pretrain_step.run(steps=3, rows=256, width=128, vocab=1009)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)


def test_gradients_of_the_whole_step():
    """Against autograd in float64 through the same bfloat16 weights. The hidden states are rounded to bfloat16 at every
    product (2^-9 relative on average, and so are the gradients on their way back), so gradients agree to a few 2^-8 of their
    norm; an error in a formula, a missing row or a wrong scale shows as tenths."""
    import pretrain_step
    model = pretrain_step.Model(128, 2, 1009, seed=3)
    tokens, targets = pretrain_step.make_batch(300, 1009, seed=4)
    loss = model.backward(tokens, targets)
    half = [w.bfloat16().double().requires_grad_(True) for w in model.params]
    x = half[-2][tokens]
    for w, v in zip(half[0:-2:2], half[1:-2:2]):
        x = x + torch.nn.functional.gelu(model.norm(x) @ w, approximate="tanh") @ v
    z = (model.norm(x) * half[-1]) @ half[-2].t()
    want = torch.nn.functional.cross_entropy(z, targets, ignore_index=-100)
    assert abs(float(loss) - float(want.detach())) <= 2.0 ** -7 * abs(float(want.detach()))
    grads = torch.autograd.grad(want, half)
    for got, add, d in zip(model.grads, model.added, grads):
        assert float((got.double() + add.double() - d).norm()) <= 8 * 2.0 ** -8 * float(d.norm())


def test_step_of_the_whole_model():
    """What one step does to every weight: the joint norm over all gradients, one factor for both optimizers, Muon's weights
    against the iteration in float64 (within what its binary16 storage does, 2^-8 of the update), AdamW's first step against
    its closed form."""
    import pretrain_step
    from test_gpu_muon import iterate
    model = pretrain_step.Model(128, 1, 501, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    for t in model.grads:
        t.normal_(generator=g)
    n = len(model.hidden)
    model.added[n].normal_(generator=g)
    before = [p.double() for p in model.params]
    grads = [(a + b).double() for a, b in zip(model.grads, model.added)]
    lr = 1e-2
    norm = model.step(lr, max_norm=1.0)
    want = math.sqrt(sum(float(x.square().sum()) for x in grads))
    assert abs(float(norm) - want) <= 1e-5 * want
    f = 1.0 / (want + 1e-6)
    for k in range(n):
        gh = f * grads[k]
        m = 0.05 * gh
        update = lr * 0.2 * math.sqrt(max(gh.shape)) * iterate(gh + 0.95 * (m - gh))
        w = before[k] * (1 - lr * 0.01) - update
        assert float((model.params[k].double() - w).norm()) <= 2.0 ** -8 * float(update.norm()) + 1e-6 * float(w.norm())
    for k in (n, n + 1):
        gh = f * grads[k]
        w = before[k] - lr * gh / (gh.abs() + 1e-8)
        assert float((model.params[k].double() - w).abs().max()) <= 1e-5
