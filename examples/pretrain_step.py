"""Pre-training steps with this package's kernels and plain matrix products: hidden states -> cross entropy without stored logits,
with both gradients -> one clip over all gradients -> Muon for the hidden matrices, AdamW for the tied embedding and the gains.

The model is a stack of residual MLP blocks between an embedding and the same embedding as output layer, in bfloat16 with
float32 master weights. The embedding's gradient has two contributions, the output layer's and the input's: the second is
added to the first in the pass that takes the joint norm.

    python examples/pretrain_step.py [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import clip_tensor_adamw_gb300 as mica  # noqa: E402


class Model:
    """x_0 = E[tokens], x_{i+1} = x_i + gelu(n(x_i) W_i) V_i with n(x) = x / rms(x), logits = (gain * n(x)) E^T."""

    def __init__(self, width: int, blocks: int, vocab: int, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        shapes = [s for _ in range(blocks) for s in ((width, 4 * width), (4 * width, width))]
        self.hidden = [torch.randn(s, generator=g, device=device) * s[0] ** -0.5 for s in shapes]
        self.embedding = torch.randn(vocab, width, generator=g, device=device) * width ** -0.5
        self.gain = torch.ones(width, device=device)
        self.params = [*self.hidden, self.embedding, self.gain]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.added = [torch.zeros_like(p) for p in self.params]  # the gradients' other contributions: the input embedding's
        n = len(shapes)
        self.G, self.A = mica.TensorList(self.grads), mica.TensorList(self.added)
        self.muon = [mica.TensorList(x) for x in (self.hidden, self.grads[:n], [torch.zeros_like(w) for w in self.hidden])]
        rest = self.params[n:]
        self.adamw = [mica.TensorList(x) for x in (rest, self.grads[n:], *([torch.zeros_like(w) for w in rest] for _ in range(2)))]
        self.steps = 0

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)

    def forward(self, tokens, half):
        """The hidden states before the output layer, with the graph of everything before it."""
        x = half[-2].detach()[tokens].float().requires_grad_(True)
        self.first = x
        for w, v in zip(half[0:-2:2], half[1:-2:2]):
            x = x + (torch.nn.functional.gelu(self.norm(x).bfloat16() @ w, approximate="tanh") @ v).float()
        return (self.norm(x) * half[-1].float()).bfloat16()

    def backward(self, tokens, targets):
        """Writes every gradient (float32) and returns the loss."""
        half = [w.bfloat16().requires_grad_(True) for w in self.params]
        h = self.forward(tokens, half)
        n = len(self.hidden)
        r = mica.mica_linear_cross_entropy(h.detach(), half[n].detach(), targets, dw=self.grads[n])
        inner = [*half[:n], half[n + 1], self.first]
        found = torch.autograd.grad(h, inner, r.dh)
        for g, d in zip([*self.grads[:n], self.grads[n + 1]], found):
            g.copy_(d)
        self.added[n].zero_().index_add_(0, tokens, found[-1])
        return r.loss

    def step(self, lr: float, max_norm: float = 1.0) -> torch.Tensor:
        self.steps += 1
        norm, factor = mica.mica_accumulate_clip_grad_norms(self.G, self.A, max_norm=max_norm)
        mica.mica_muon_steps(*self.muon, lr=lr, momentum=0.95, weight_decay=0.01, adjust="match_rms_adamw", factor=factor)
        mica.mica_adamw_steps(*self.adamw, lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, step=self.steps, factor=factor)
        return norm


def make_batch(rows: int, vocab: int, seed: int = 1):
    """Tokens and the next ones; the first of each run of 64 is a prompt and not scored."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    targets = (tokens * 31 + 7) % vocab
    targets[torch.arange(rows, device="cuda") % 64 == 0] = -100
    return tokens, targets


def run(steps: int = 20, rows: int = 1024, width: int = 384, blocks: int = 2, vocab: int = 5003, lr: float = 2e-3) -> list[float]:
    model = Model(width, blocks, vocab)
    tokens, targets = make_batch(rows, vocab)
    losses = []
    for _ in range(steps):
        losses.append(model.backward(tokens, targets))
        model.step(lr)
    mica.mica_sync()
    return [v.item() for v in losses]


if __name__ == "__main__":
    parser = argparse.ArgumentParser()
    parser.add_argument("--steps", type=int, default=20)
    for i, loss in enumerate(run(parser.parse_args().steps)):
        print(f"step {i + 1}: loss {loss:.4f}")
