"""The losses from hidden states against their definitions in float64, over element types, sizes, strides, masks and the
values that end in infinities and NaNs.

Tolerances, with u = 2^-24 and E = 2^-9 (bfloat16) or 2^-12 (binary16), the most that a rounding to the type is off by,
relative (half a unit in the last place: 2^-8 / 2 and 2^-11 / 2 of the next power of two, so E of a value at its lower end is
twice that: e(x) = 2 E |x|).

  logits   The products are exact and there are `features` of them; each of the features / 16 additions to the accumulator
           truncates, at 2^-23 of the largest term at hand, and within 16 products the alignment drops as much: a logit is off
           by at most 2 (features / 16 + 2) 2^-23 sum_k |h_k w_k| / T =: t.
  lse      A sum of `vocabulary` positive terms, each off by t + 4u|z| and 2^-22 (the hardware's power of two), added 8 in a
           row four times over, 4 chunks and vocabulary / 128 parts: at most t + 4u|z| + 2^-22 + (vocabulary / 1024 + 64) u.
  d        An element c (1[target] - p) has p's relative error, the same as exp(lse)'s and the logit's together (2 lse errors),
           and is rounded once: e(d) (binary16: and half of 2^-24 of the largest |c| 2^-14, the smallest step).
  dh, dw   Errors of d add up at worst: sum_j err_j |w_j|; the sums in float32 truncate: (terms / 16 + 2) 2^-22 sum |d_j w_j|;
           then one rounding.
"""
import math

import pytest
import torch

import clip_tensor_adamw_gb300 as mica

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}
HALVES = [torch.float16, torch.bfloat16]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def strided(g, rows, cols, ld, offset, dtype, scale=1.0):
    flat = torch.randn(offset + max(rows, 1) * max(ld, cols), generator=g, device="cuda") * scale
    return flat.to(dtype)[offset:].as_strided((rows, cols), (ld, 1))


def make(rows, features, vocab, dtype, seed=0, skip=0.3, ld_h=None, ld_w=None, offset=0, index=torch.int64):
    g = gen(seed)
    h = strided(g, rows, features, ld_h or features, offset, dtype)
    w = strided(g, vocab, features, ld_w or features, offset, dtype, 1.5 / math.sqrt(features))
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    y[torch.rand(rows, generator=g, device="cuda") < skip] = -100
    return h, w, y.to(index)


class Want:
    """The definitions in float64 with the bounds of the errors."""

    def __init__(self, h, w, y, temperature=1.0):
        self.h, self.w, self.y, self.t = h.double(), w.double(), y.long(), temperature
        self.on = self.y >= 0
        self.h = torch.where(self.on[:, None], self.h, 0.0)
        features, vocab = h.shape[1], w.shape[0]
        self.z = self.h @ self.w.t() / temperature
        self.t_err = (2 * (features / 16 + 2) * 2.0 ** -23 * (self.h.abs() @ self.w.abs().t()) / temperature).amax(1)
        self.lse = torch.logsumexp(self.z, 1)
        self.at = self.z.gather(1, self.y.clamp(min=0)[:, None])[:, 0]
        self.logps = torch.where(self.on, self.at - self.lse, 0.0)
        top = self.z.abs().amax(1)
        self.err = self.t_err + 6 * U * (top + 1) + 2.0 ** -22 + (vocab / 1024 + 64) * U
        self.p = torch.exp(self.z - self.lse[:, None])

    def grads(self, dlogps, dtype, add=None):
        """(dh, its bound, dw, its bound), before the last rounding"""
        c = torch.where(self.on, dlogps.double() / self.t, 0.0)[:, None]
        one = torch.zeros_like(self.p).scatter_(1, self.y.clamp(min=0)[:, None], 1.0)
        d = c * (one - self.p)
        err = c.abs() * (2 * self.err[:, None] * self.p + 4 * U) + ROUND[dtype] * d.abs()
        if dtype == torch.float16:
            err += 2.0 ** -25 * 2.0 ** -13 * c.abs().amax() * (c != 0)
        rows, vocab = d.shape
        long = lambda n: (n / 16 + 4) * 2.0 ** -22  # noqa: E731
        dh, dw = d @ self.w, d.t() @ self.h
        dh_err = err @ self.w.abs() + long(vocab) * (d.abs() @ self.w.abs())
        dw_err = err.t() @ self.h.abs() + long(rows) * (d.abs().t() @ self.h.abs())
        if add is not None:
            dw = dw + add.double()
            dw_err = dw_err + 2 * U * dw.abs()
        return dh, dh_err, dw, dw_err


def close(a, b, tol):
    a = a.double()
    bad = ~((a - b).abs() <= tol) & ~(a.isnan() & b.isnan()) & ~(a == b)
    assert not bad.any(), (int(bad.sum()), a[bad][:4], b[bad][:4], (tol[bad] if torch.is_tensor(tol) else tol))


def rounded(got, want, err):
    close(got, want, err + (want.abs() + err) * ROUND[got.dtype] + TINY[got.dtype])


SHAPES = [(1, 1, 1), (3, 16, 7), (5, 33, 129), (2, 64, 257), (64, 128, 256), (65, 100, 1000), (300, 387, 515), (257, 72, 4099),
          (1, 768, 50257), (40, 200, 30011), (700, 513, 130)]


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("rows,features,vocab", SHAPES)
def test_logps(rows, features, vocab, dtype):
    h, w, y = make(rows, features, vocab, dtype, seed=rows + vocab, skip=0.0 if rows == 1 else 0.3)
    for t in (1.0, 0.7):
        want = Want(h, w, y, t)
        lp, lse = mica.mica_linear_logps(h, w, y, temperature=t, lse=True)
        close(lp, want.logps, 2 * want.err)
        close(lse, torch.where(want.on, want.lse, 0.0), want.err + U * want.lse.abs())
        assert torch.equal(lp, mica.mica_linear_logps(h, w, y, temperature=t))


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("rows,features,vocab", SHAPES)
def test_logps_grad(rows, features, vocab, dtype):
    h, w, y = make(rows, features, vocab, dtype, seed=3 * rows + vocab, skip=0.0 if rows == 1 else 0.3, index=torch.int32)
    want = Want(h, w, y, 0.9)
    c = torch.randn(rows, generator=gen(5), device="cuda")
    if rows > 2:
        c[::3] = 0.0
    dh, dh_err, dw, dw_err = want.grads(c, dtype)
    lse = want.lse.float()
    for out in (dtype, torch.float32):
        got_h, got_w = mica.mica_linear_logps_grad(h, w, y, lse, c, temperature=0.9, dw_dtype=out)
        assert got_h.dtype == dtype and got_w.dtype == out
        rounded(got_h, dh, dh_err)
        rounded(got_w, dw, dw_err)
        assert not got_h[(y < 0) | (c == 0)].any()


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("rows,features,vocab", SHAPES)
def test_cross_entropy(rows, features, vocab, dtype):
    h, w, y = make(rows, features, vocab, dtype, seed=7 * rows + vocab, skip=0.0 if rows == 1 else 0.3)
    want = Want(h, w, y)
    scale = 64.0
    for denom in (None, 5.0):
        n = max(1, int(want.on.sum())) if denom is None else denom
        r = mica.mica_linear_cross_entropy(h, w, y, denom=denom, grad_scale=scale)
        close(r.logps, want.logps, 2 * want.err)
        close(r.loss[0], -want.logps.sum() / n, 2 * want.err.sum() / n + 4 * U * want.logps.abs().sum() / n)
        dh, dh_err, dw, dw_err = want.grads(torch.full((rows,), -scale / n, device="cuda"), dtype)
        rounded(r.dh, dh, dh_err)
        rounded(r.dw, dw, dw_err)
    r2 = mica.mica_linear_cross_entropy(h, w, y, denom=5.0, grad=False)
    assert r2.dh is None and r2.dw is None and torch.equal(r2.loss, r.loss) and torch.equal(r2.logps, r.logps)
