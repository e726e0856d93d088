"""Preference fine-tuning steps with nothing but this package's kernels and plain matrix products: logits -> preference
loss and its gradient -> weight gradients from 8-bit activation checkpoints -> clip + AdamW.

The model is a residual MLP block and an output projection over frozen embeddings, in bfloat16 with float32 master weights.
Everything that the backward pass needs of the forward pass is kept as 8-bit checkpoints (a little over half of the
bfloat16 activations' memory), and the logits' gradient is written over the logits.

    python examples/preference_step.py [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import clip_tensor_adamw_gb300 as mica  # noqa: E402


class Block:
    """z = x + gelu(x W1) W2, logits = z W3, with its backward pass written out."""

    def __init__(self, width: int, vocab: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        shapes = [(width, 4 * width), (4 * width, width), (width, vocab)]
        self.w = [torch.randn(s, generator=g, device=device) * s[0] ** -0.5 for s in shapes]
        self.g = [torch.zeros_like(w) for w in self.w]
        self.half = [w.bfloat16() for w in self.w]
        self.W, self.G = mica.TensorList(self.w), mica.TensorList(self.g)
        self.M, self.V = (mica.TensorList([torch.zeros_like(w) for w in self.w]) for _ in range(2))
        self.steps = 0

    def forward(self, x: torch.Tensor, keep: bool = False) -> torch.Tensor:
        w1, w2, w3 = self.half
        h = x @ w1
        if not keep:
            y = torch.nn.functional.gelu(h, approximate="tanh")
            return (x + y @ w2) @ w3
        packed_h, y = mica.mica_act_pack(h, "gelu_tanh")
        z = x + y @ w2
        self.kept = [mica.mica_act_pack(x), packed_h, mica.mica_act_pack(y), mica.mica_act_pack(z)]
        return z @ w3

    def backward(self, dlogits: torch.Tensor) -> None:
        """Writes the weights' gradients (float32) from the checkpoints that forward(keep=True) left."""
        _, w2, w3 = self.half
        x, h, y, z = self.kept
        mica.mica_packed_wgrad(z, dlogits, out=self.g[2])
        dz = dlogits @ w3.t()
        mica.mica_packed_wgrad(y, dz, out=self.g[1])
        dh = dz @ w2.t()
        mica.mica_act_grad(h, dh, "gelu_tanh", out=dh)
        mica.mica_packed_wgrad(x, dh, out=self.g[0])

    def step(self, lr: float, max_norm: float = 1.0) -> torch.Tensor:
        self.steps += 1
        norm, _ = mica.mica_clip_adamw_step(self.W, self.G, self.M, self.V, max_norm=max_norm, lr=lr, beta1=0.9,
                                            beta2=0.95, eps=1e-8, weight_decay=0.0, step=self.steps)
        for half, w in zip(self.half, self.w):
            half.copy_(w)
        return norm


def make_batch(pairs: int, length: int, width: int, vocab: int, seed: int = 1):
    """Embeddings, targets (the first quarter of each sequence is prompt and not scored) and sequence bounds."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = [length - (7 * i) % max(1, length // 3) for i in range(2 * pairs)]
    ends = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    rows = sum(lens)
    x = torch.randn(rows, width, generator=g, device="cuda").bfloat16()
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    at = 0
    for n in lens:
        targets[at:at + n // 4] = -100
        at += n
    return x, targets, ends


def run(steps: int = 20, pairs: int = 8, length: int = 96, width: int = 384, vocab: int = 5003,
        lr: float = 2e-5) -> list[float]:
    model = Block(width, vocab)
    x, targets, ends = make_batch(pairs, length, width, vocab)
    reference = mica.mica_token_logps(model.forward(x), targets)  # the frozen policy's scores: the model's own, before
    losses = []
    for _ in range(steps):
        logits = model.forward(x, keep=True)
        r = mica.mica_preference_loss(logits, targets, ends, reference, beta=0.1, out=logits)
        model.backward(r.dlogits)
        model.step(lr)
        losses.append(r.loss)
    mica.mica_sync()
    return [v.item() for v in losses]


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=20)
    for i, loss in enumerate(run(parser.parse_args().steps)):
        print(f"step {i + 1}: loss {loss:.4f}")
