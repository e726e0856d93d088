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
           Cross entropy in bfloat16 leaves exp(z - z_target) in d's place, rounded once like it, and multiplies dh's rows and,
           rounded once more, h's rows by what is left: another e(d) and another error of exp(lse).
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

    def grads(self, dlogps, dtype, add=None, once=False):
        """(dh, its bound, dw, its bound), before the last rounding. once: with h's rows scaled by the rest of the softmax, and
        rounded once more, and d counted from another origin"""
        c = torch.where(self.on, dlogps.double() / self.t, 0.0)[:, None]
        one = torch.zeros_like(self.p).scatter_(1, self.y.clamp(min=0)[:, None], 1.0)
        d = c * (one - self.p)
        err = c.abs() * (2 * self.err[:, None] * self.p + 4 * U) + ROUND[dtype] * d.abs()
        if dtype == torch.float16:
            err += 2.0 ** -25 * 2.0 ** -13 * c.abs().amax() * (c != 0)
        if once and dtype == torch.bfloat16:
            err += ROUND[dtype] * d.abs() * 1.01 + c.abs() * 2 * self.err[:, None] * self.p
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
        dh, dh_err, dw, dw_err = want.grads(torch.full((rows,), -scale / n, device="cuda"), dtype, once=True)
        rounded(r.dh, dh, dh_err)
        rounded(r.dw, dw, dw_err)
    r2 = mica.mica_linear_cross_entropy(h, w, y, denom=5.0, grad=False)
    assert r2.dh is None and r2.dw is None and torch.equal(r2.loss, r.loss) and torch.equal(r2.logps, r.logps)


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("rows,features,vocab,skip", [(300, 517, 70001, 0.3), (1100, 256, 40003, 0.5), (513, 1000, 20011, 0.0),
                                                      (90, 520, 213001, 0.2)])
def test_cross_entropy_of_many(rows, features, vocab, skip, dtype):
    h, w, y = make(rows, features, vocab, dtype, seed=rows, skip=skip)
    for scale, t in ((64.0, 1.0), (-3.0, 0.8)):
        want = Want(h, w, y, t)
        n = max(1, int(want.on.sum()))
        r = mica.mica_linear_cross_entropy(h, w, y, grad_scale=scale, temperature=t)
        close(r.logps, want.logps, 2 * want.err)
        close(r.loss[0], -want.logps.sum() / n, 2 * want.err.sum() / n + 4 * U * want.logps.abs().sum() / n)
        c = torch.full((rows,), -scale / n, device="cuda")
        dh, dh_err, dw, dw_err = want.grads(c, dtype, once=True)
        rounded(r.dh, dh, dh_err)
        rounded(r.dw, dw, dw_err)


@pytest.mark.parametrize("rows,features,vocab", [(2500, 300, 5000), (4000, 520, 9000), (700, 800, 40_000), (5200, 100, 700), (2100, 2000, 3000)])
def test_work_of_both_gradients(rows, features, vocab):
    """How both gradients' tiles are dealt: dh's split along the vocabulary or not, dw's going on in turn."""
    h, w, y = make(rows, features, vocab, torch.bfloat16, seed=rows, skip=0.05)
    lp, lse = mica.mica_linear_logps(h, w, y, lse=True)
    c = torch.randn(rows, generator=gen(2), device="cuda")
    got = mica.mica_linear_logps_grad(h, w, y, lse, c)
    dh, dh_err, dw, dw_err = Want(h, w, y).grads(c, torch.bfloat16)
    rounded(got[0], dh, dh_err)
    rounded(got[1], dw, dw_err)
    one = mica.mica_linear_logps_grad(h, w, y, lse, c, want_dh=False)[1]
    two = mica.mica_linear_logps_grad(h, w, y, lse, c, want_dw=False)[0]
    rounded(one, dw, dw_err)
    rounded(two, dh, dh_err)


def test_offsets_past_32_bits():
    """An embedding, its gradient and hidden states of more than 2^31 elements; the rows at their ends against float64."""
    rows, features, vocab = 40, 40_000, 60_000
    g = gen(31)
    w = torch.empty(vocab, features, dtype=torch.bfloat16, device="cuda").normal_(0.0, features ** -0.5, generator=g)
    h = torch.empty(70_000, features, dtype=torch.bfloat16, device="cuda")[::1790]  # 40 rows, the last past 2^31 elements
    h.normal_(generator=g)
    assert h.shape[0] == rows and w.numel() > 2 ** 31 and h.stride(0) * (rows - 1) > 2 ** 31
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    y[0], y[1], y[2] = 0, vocab - 1, vocab - 2
    z = torch.cat([h.double() @ w[a:a + 5000].double().t() for a in range(0, vocab, 5000)], 1)
    lse = torch.logsumexp(z, 1)
    want = z.gather(1, y[:, None])[:, 0] - lse
    r = mica.mica_linear_cross_entropy(h, w, y)
    # the longest sum: 2,500 additions of 16 products each, truncated; 2 (features / 16 + 2) 2^-23 sum |h w| as above
    err = 2 * (features / 16 + 2) * 2.0 ** -23 * float((h.double().abs() @ w[:1000].double().abs().t()).max()) * 1.5 + 1e-4
    close(r.logps, want, err)
    d = (torch.exp(z - lse[:, None]) - torch.nn.functional.one_hot(y, vocab)) / rows
    for at in (slice(0, 3), slice(vocab - 3, vocab), slice(int(y[5]), int(y[5]) + 1)):
        dw = d[:, at].t() @ h.double()
        assert float((r.dw[at].double() - dw).norm()) <= 0.02 * float(dw.norm())
    for i in (0, rows - 1):
        dh = sum(d[i, a:a + 5000] @ w[a:a + 5000].double() for a in range(0, vocab, 5000))
        assert float((r.dh[i].double() - dh).norm()) <= 0.02 * float(dh.norm())


def test_largest_vocabulary():
    """2^24 tokens: more than 2^32 elements of d, 65,536 tiles across, a row's sum of 131,072 parts."""
    rows, features, vocab = 300, 16, 1 << 24
    g = gen(32)
    h = torch.randn(rows, features, generator=g, device="cuda").half()
    w = torch.randn(vocab, features, generator=g, device="cuda").half()
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    y[0], y[1] = vocab - 1, 0
    lse = torch.logsumexp(torch.stack([torch.logsumexp(h.double() @ w[a:a + (1 << 20)].double().t(), 1)
                                       for a in range(0, vocab, 1 << 20)]), 0)
    want = (h.double() * w[y].double()).sum(1) - lse
    r = mica.mica_linear_cross_entropy(h, w, y, grad_scale=2.0 ** 20)
    close(r.logps, want, (vocab / 1024 / 32 + 64) * U + 1e-5)  # a lane joins 4,096 of a row's parts, five joins follow
    for at in (0, vocab - 1, int(y[7])):
        p = torch.exp(h.double() @ w[at].double() - lse)
        d = (p - (y == at).double()) / rows * 2.0 ** 20
        dw = d @ h.double()
        assert float((r.dw[at].double() - dw).abs().max()) <= 2.0 ** -10 * float((d.abs() @ h.double().abs()).max())


@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_unlikely_targets(dtype):
    """Rows whose target is e^-30 to e^-400 likely, among ordinary ones: the sum of exp(z - z_target) leaves its range."""
    rows, features, vocab = 520, 512, 50021
    h, w, y = make(rows, features, vocab, dtype, seed=11, skip=0.1)
    g = gen(12)
    far = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    some = torch.arange(rows, device="cuda") % 7 == 3
    some &= torch.arange(rows, device="cuda") < 300  # the second tile of rows has a few, the third none
    row, at = w[far].float(), w[y.clamp(min=0)].float()
    size = 15.0 + 190.0 * torch.rand(rows, 1, generator=g, device="cuda")
    push = size * (row / row.square().sum(1, keepdim=True) - at / at.square().sum(1, keepdim=True))
    h = torch.where(some[:, None], (h.float() + push).to(dtype), h)
    want = Want(h, w, y)
    assert float(want.logps.min()) < -200 and int((want.logps < -45).sum()) > 20
    n = int(want.on.sum())
    r = mica.mica_linear_cross_entropy(h, w, y)
    close(r.logps, want.logps, 2 * want.err)
    alone = mica.mica_linear_cross_entropy(h, w, y, grad=False)
    assert torch.equal(alone.logps, r.logps) and torch.equal(alone.loss, r.loss)
    dh, dh_err, dw, dw_err = want.grads(torch.full((rows,), -1.0 / n, device="cuda"), dtype, once=True)
    rounded(r.dh, dh, dh_err)
    rounded(r.dw, dw, dw_err)


@pytest.mark.parametrize("rows,vocab", [(70, 200), (300, 70001)])
@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_what_does_not_count_is_not_read(dtype, rows, vocab):
    """Rows without a target may hold anything; their gradients are zeros, and the others' as if they were not there."""
    h, w, y = make(rows, 512, vocab, dtype, seed=3, skip=0.4)
    off = y < 0
    clean = mica.mica_linear_cross_entropy(h, w, y)
    dirty = torch.where(off[:, None], torch.full_like(h, math.nan), h)
    r = mica.mica_linear_cross_entropy(dirty, w, y)
    for a, b in zip(r, clean):
        assert torch.equal(a, b)
    assert not r.dh[off].any() and not r.logps[off].any()
    lp, lse = mica.mica_linear_logps(dirty, w, y, lse=True)
    assert not lp[off].any() and not lse[off].any() and lp.isfinite().all()
    c = torch.randn(rows, generator=gen(4), device="cuda")
    g1 = mica.mica_linear_logps_grad(h, w, y, lse, c)
    g2 = mica.mica_linear_logps_grad(dirty, w, y, torch.where(off, math.nan, lse), torch.where(off, math.nan, c))
    assert torch.equal(g1[0], g2[0]) and torch.equal(g1[1], g2[1])


@pytest.mark.parametrize("vocab", [300, 70001])
@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_targets_past_the_vocabulary(dtype, vocab):
    """NaN, in the row's log-probability and gradients and in all of dw; not where its coefficient is 0."""
    rows = 300
    h, w, y = make(rows, 512, vocab, dtype, seed=5, skip=0.2)
    y[7], y[11] = vocab, 1 << 40
    r = mica.mica_linear_cross_entropy(h, w, y)
    bad = (y >= vocab).nonzero()[:, 0]
    assert r.logps[bad].isnan().all() and r.loss.isnan() and r.dh[bad].isnan().all() and r.dw.isnan().all()
    rest = y < vocab
    assert r.logps[rest].isfinite().all() and r.dh[rest].isfinite().all()
    lp, lse = mica.mica_linear_logps(h, w, y, lse=True)
    assert lp[bad].isnan().all() and lp[rest].isfinite().all()
    c = torch.ones(rows, device="cuda")
    c[bad] = 0.0
    dh, dw = mica.mica_linear_logps_grad(h, w, y, lse, c)
    assert dh.isfinite().all() and dw.isfinite().all() and not dh[bad].any()
    c[7] = 1.0
    dh, dw = mica.mica_linear_logps_grad(h, w, y, lse, c)
    assert dh[7].isnan().all() and dw.isnan().all() and not dh[11].any()


@pytest.mark.parametrize("vocab", [300, 70001])
@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_infinities(dtype, vocab):
    """A row with an infinity in h or w: what the formula gives, infinities and NaNs, and the other rows as ever."""
    h, w, y = make(300, 512, vocab, dtype, seed=6, skip=0.0)
    h[5, 3] = math.inf
    h[9, 0] = math.nan
    want = torch.log_softmax(h.double() @ w.double().t(), 1).gather(1, y[:, None])[:, 0]
    r = mica.mica_linear_cross_entropy(h, w, y)
    ok = want.isfinite()
    assert int(ok.sum()) == 298
    close(r.logps[ok], want[ok], 2 * Want(h[ok], w, y[ok]).err)
    assert not r.logps[~ok].isfinite().any() and not r.loss.isfinite().any() and r.dh[~ok].isnan().any(1).all()
    assert r.dh[ok].isfinite().all()


@pytest.mark.parametrize("dtype", HALVES, ids=str)
@pytest.mark.parametrize("features,ld_h,ld_w,offset", [(64, 64, 64, 1), (63, 70, 65, 0), (72, 80, 96, 8), (72, 0, 72, 0), (40, 41, 48, 3),
                                                       (64, 64, 0, 0)])
def test_strides_and_offsets(features, ld_h, ld_w, offset, dtype):
    """Rows at every alignment, of h, w, the gradients and what these are added to; and matrices whose rows are all the same."""
    rows, vocab = 130, 517
    h, w, y = make(rows, features, vocab, dtype, seed=features, ld_h=ld_h or 1, ld_w=ld_w or 1, offset=offset)
    if ld_h == 0:
        h = h[:1].expand(rows, features)
    if ld_w == 0:
        w = w[:1].expand(vocab, features)
    want = Want(h, w, y)
    lp, lse = mica.mica_linear_logps(h, w, y, lse=True)
    close(lp, want.logps, 2 * want.err)
    c = torch.randn(rows, generator=gen(8), device="cuda")
    for first, extra, out in ((0, 0, dtype), (1, 3, dtype), (8, 8, torch.float32), (3, 1, torch.float32), (0, 16, torch.bfloat16)):
        g = gen(9)
        base_h = torch.full((first + rows * (features + extra) + 9,), 7.0, dtype=dtype, device="cuda")
        base_w = torch.full((first + vocab * (features + extra) + 9,), 7.0, dtype=out, device="cuda")
        dh = base_h[first:].as_strided((rows, features), (features + extra, 1))
        dw = base_w[first:].as_strided((vocab, features), (features + extra, 1))
        add = strided(g, vocab, features, features + 5, 1, out)
        exact = want.grads(c, dtype, add=add)
        a, b = mica.mica_linear_logps_grad(h, w, y, lse, c, dh=dh, dw=dw, add=add)
        assert a.data_ptr() == dh.data_ptr() and b.data_ptr() == dw.data_ptr()
        rounded(dh, exact[0], exact[1])
        rounded(dw, exact[2], exact[3])
        kept = dw.clone()
        mica.mica_linear_logps_grad(h, w, y, lse, c, want_dh=False, dw=dw, add=dw)
        exact = want.grads(c, dtype, add=kept)
        rounded(dw, exact[2], exact[3])
        for base, t in ((base_h, dh), (base_w, dw)):  # nothing beside the rows was written
            t.fill_(7.0)
            assert (base == 7.0).all()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=str)
def test_more_rows_than_a_piece(out):
    """A vocabulary so large that the rows are taken in pieces, whose sums wait for one another."""
    rows, features, vocab = 1500, 40, 600_007
    h, w, y = make(rows, features, vocab, torch.bfloat16, seed=2, skip=0.1)
    add = torch.randn(vocab, features, generator=gen(3), device="cuda").to(out)
    want = Want(h, w, y)
    n = int(want.on.sum())
    r = mica.mica_linear_cross_entropy(h, w, y, add=add)
    close(r.logps, want.logps, 2 * want.err)
    close(r.loss[0], -want.logps.sum() / n, 2 * want.err.sum() / n + 4 * U * want.logps.abs().sum() / n)
    dh, dh_err, dw, dw_err = want.grads(torch.full((rows,), -1.0 / n, device="cuda"), torch.bfloat16, add=add, once=True)
    rounded(r.dh, dh, dh_err)
    rounded(r.dw, dw, dw_err)
    lp, lse = mica.mica_linear_logps(h, w, y, lse=True)
    close(lp, want.logps, 2 * want.err)
    a, b = mica.mica_linear_logps_grad(h, w, y, lse, torch.where(want.on, -1.0 / n, 0.0).float(), add=add)
    rounded(a, dh, dh_err)
    rounded(b, dw, dw_err)


@pytest.mark.parametrize("rows,skip", [(1024, 0.5), (1025, 0.5), (2049, 0.5), (20_000, 0.1), (40_000, 0.9), (70_001, 0.02)])
def test_many_rows(rows, skip):
    """Rows that are looked through by a kernel of its own, more than a piece of the forward pass, and over the boundary."""
    h, w, y = make(rows, 40, 301, torch.float16, seed=rows, skip=skip)
    dirty = torch.where((y < 0)[:, None], torch.full_like(h, math.nan), h)
    want = Want(h, w, y)
    lp, lse = mica.mica_linear_logps(dirty, w, y, lse=True)
    close(lp, want.logps, 2 * want.err)
    close(lse, torch.where(want.on, want.lse, 0.0), want.err + U * want.lse.abs())
    c = torch.randn(rows, generator=gen(1), device="cuda")
    c[::5] = 0.0
    got = mica.mica_linear_logps_grad(dirty, w, y, lse, c)
    dh, dh_err, dw, dw_err = want.grads(c, torch.float16)
    rounded(got[0], dh, dh_err)
    rounded(got[1], dw, dw_err)
    assert not got[0][(y < 0) | (c == 0)].any()
    r = mica.mica_linear_cross_entropy(dirty, w, y, grad_scale=256.0)
    n = int(want.on.sum())
    close(r.loss[0], -want.logps.sum() / n, 2 * want.err.sum() / n + 4 * U * want.logps.abs().sum() / n)
    dh, dh_err, dw, dw_err = want.grads(torch.full((rows,), -256.0 / n, device="cuda"), torch.float16)
    rounded(r.dh, dh, dh_err)
    rounded(r.dw, dw, dw_err)


@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_no_rows(dtype):
    """Without rows, or with none that counts: the loss is 0, dw is add."""
    w = torch.randn(300, 72, generator=gen(1), device="cuda").to(dtype)
    add = torch.randn(300, 72, generator=gen(2), device="cuda")
    for rows in (0, 5, 700, 3000):
        h = torch.full((rows, 72), math.nan, dtype=dtype, device="cuda")
        y = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
        r = mica.mica_linear_cross_entropy(h, w, y, add=add)
        assert float(r.loss) == 0.0 and not r.logps.any() and not r.dh.any() and torch.equal(r.dw, add)
        r = mica.mica_linear_cross_entropy(h, w, y, denom=3.0)
        assert float(r.loss) == 0.0 and not r.dw.any()
        lp, lse = mica.mica_linear_logps(h, w, y, lse=True)
        assert not lp.any() and not lse.any()
        c = torch.ones(rows, device="cuda")
        a, b = mica.mica_linear_logps_grad(h, w, y, lse, c, add=add)
        assert not a.any() and torch.equal(b, add)
        a, b = mica.mica_linear_logps_grad(h, w, y, lse, c)
        assert not b.any() and b.dtype == dtype


@pytest.mark.parametrize("rows,features,vocab", [(200, 128, 3001), (400, 512, 60007)])
def test_one_gradient_alone(rows, features, vocab):
    h, w, y = make(rows, features, vocab, torch.bfloat16, seed=4)
    r = mica.mica_linear_cross_entropy(h, w, y)
    a = mica.mica_linear_cross_entropy(h, w, y, want_dw=False)
    b = mica.mica_linear_cross_entropy(h, w, y, want_dh=False)
    assert a.dw is None and b.dh is None and torch.equal(a.dh, r.dh) and torch.equal(b.dw, r.dw)
    assert torch.equal(a.loss, r.loss)
    none = mica.mica_linear_cross_entropy(h, w, y, grad=False)
    assert none.dh is None and none.dw is None and torch.equal(none.loss, r.loss) and torch.equal(none.logps, r.logps)


@pytest.mark.parametrize("rows,features,vocab", [(40, 100, 1000), (400, 512, 60007)])
def test_streams_graphs_and_repeats(rows, features, vocab):
    """The same bits on another stream, twice at once on two, and captured into a graph and replayed on new inputs."""
    h, w, y = make(rows, features, vocab, torch.bfloat16, seed=9)
    first = mica.mica_linear_cross_entropy(h, w, y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [mica.mica_linear_cross_entropy(h, w, y, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for r in both:
        assert all(torch.equal(a, b) for a, b in zip(r, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = mica.mica_linear_cross_entropy(h, w, y)
        lp, lse = mica.mica_linear_logps(h, w, y, lse=True)
        g = mica.mica_linear_logps_grad(h, w, y, lse, lp)
    for seed in (10, 11):
        h2, w2, y2 = make(rows, features, vocab, torch.bfloat16, seed=seed, skip=0.1 * (seed - 9))
        for a, b in ((h, h2), (w, w2), (y, y2)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = mica.mica_linear_cross_entropy(h2, w2, y2)
        assert all(torch.equal(a, b) for a, b in zip(r, want))
        lp2, lse2 = mica.mica_linear_logps(h2, w2, y2, lse=True)
        g2 = mica.mica_linear_logps_grad(h2, w2, y2, lse2, lp2)
        assert torch.equal(lp, lp2) and torch.equal(g[0], g2[0]) and torch.equal(g[1], g2[1])


def test_gradients_against_differences():
    """The loss's change along a direction of h, and of w, against the gradients: the loss is exact to 1e-6 or so, the step is
    small and the second difference is taken off by going both ways."""
    h, w, y = make(64, 128, 900, torch.float16, seed=21, skip=0.2)
    r = mica.mica_linear_cross_entropy(h, w, y, dw_dtype=torch.float32)
    g = gen(22)
    for x, d in ((h, r.dh), (w, r.dw)):
        step = (0.02 * torch.randn(x.shape, generator=g, device="cuda")).half()
        up, down = (x + step), (x - step)
        a = mica.mica_linear_cross_entropy(up if x is h else h, up if x is w else w, y, grad=False).loss.double()
        b = mica.mica_linear_cross_entropy(down if x is h else h, down if x is w else w, y, grad=False).loss.double()
        change = ((up.double() - down.double()) * d.double()).sum()
        # third differences: (|step| |row|)^3 / 6 or so of 0.2^3; and the gradients' own rounding
        assert abs(float(a - b - change)) <= 2e-3 * float(((up.double() - down.double()).abs() * d.double().abs()).sum()) + 1e-5


def test_refusals():
    h, w, y = make(8, 64, 100, torch.bfloat16)
    lse, c = torch.zeros(8, device="cuda"), torch.ones(8, device="cuda")
    with pytest.raises(mica.MicaError, match="OVERLAP"):
        mica.mica_linear_cross_entropy(h, w, y, dh=h)
    with pytest.raises(mica.MicaError, match="OVERLAP"):
        mica.mica_linear_logps_grad(h, w, y, lse, c, dw=w)
    with pytest.raises(mica.MicaError, match="HYPER"):
        mica.mica_linear_logps(h, w, y, temperature=0.0)
    with pytest.raises(mica.MicaError, match="HYPER"):
        mica.mica_linear_cross_entropy(h, w, y, grad_scale=math.inf)
    with pytest.raises(mica.MicaError, match="ADDRESS"):
        mica.mica_linear_logps(h.cpu(), w, y)
    with pytest.raises(mica.MicaError, match="ADDRESS"):
        mica.mica_linear_logps(h, w, y.cpu())
    dw = torch.zeros(100, 64, device="cuda")
    with pytest.raises(mica.MicaError, match="OVERLAP"):  # what is added to overlaps the result at another place
        both = torch.zeros(101, 64, device="cuda")
        mica.mica_linear_logps_grad(h, w, y, lse, c, dw=both[1:], add=both[:-1])
    mica.mica_linear_logps_grad(h, w, y, lse, c, dw=dw, add=dw)


@pytest.mark.parametrize("denom,scale", [(1e30, 1.0), (1.0, 1e-30), (1e20, 1e-10), (1e-20, 1.0)])
def test_small_and_large_coefficients(denom, scale):
    """A coefficient far from 1 with targets from ordinary to e^-70 likely: what multiplies d's rows, the coefficient over the
    sum of exp(z - z_target), is smaller than any normal float32, the gradients are not."""
    rows, features, vocab = 300, 512, 5003
    h, w, y = make(rows, features, vocab, torch.bfloat16, seed=41, skip=0.1)
    g = gen(42)
    far = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    row, at = w[far].float(), w[y.clamp(min=0)].float()
    size = torch.arange(rows, device="cuda")[:, None] % 4 * 6.0 * (1.0 + torch.rand(rows, 1, generator=g, device="cuda"))
    push = size * (row / row.square().sum(1, keepdim=True) - at / at.square().sum(1, keepdim=True))
    h = (h.float() + push).bfloat16()
    want = Want(h, w, y)
    assert int(((want.logps < -18) & (want.logps > -44)).sum()) > 50 and float(want.logps.min()) < -50
    c = torch.full((rows,), -scale / denom, device="cuda")
    dh, dh_err, dw, dw_err = want.grads(c, torch.bfloat16, once=True)
    # The factor of a row makes up for the rounding of its target's element, and shifts the others by that rounding: in dw, where
    # h's rows are rounded too, theirs is a third, e(d), which counts where one other token has nearly all of a row's probability.
    d = c[:, None].double() * (want.p - torch.zeros_like(want.p).scatter_(1, y.clamp(min=0)[:, None], 1.0)) * want.on[:, None]
    dw_err = dw_err + ROUND[torch.bfloat16] * (d.abs().t() @ want.h.abs())
    for out in (torch.float32, torch.bfloat16):
        r = mica.mica_linear_cross_entropy(h, w, y, denom=denom, grad_scale=scale, dw_dtype=out)
        rounded(r.dh, dh, dh_err)
        rounded(r.dw, dw, dw_err)


@pytest.mark.parametrize("vocab", [300, 70001])
@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_no_coefficient(dtype, vocab):
    """With a gradient scale of 0 every row's coefficient is 0: zeros, whatever the targets are, and the loss as ever."""
    rows = 300
    h, w, y = make(rows, 512, vocab, dtype, seed=43, skip=0.2)
    row, at = w[torch.arange(rows, device="cuda") % vocab].float(), w[y.clamp(min=0)].float()
    push = 100.0 * (row / row.square().sum(1, keepdim=True) - at / at.square().sum(1, keepdim=True))
    h[40:60] = (h.float() + push).to(dtype)[40:60]  # targets less likely than e^-100
    add = torch.randn(vocab, 512, generator=gen(44), device="cuda")
    r = mica.mica_linear_cross_entropy(h, w, y, grad_scale=0.0, add=add)
    assert not r.dh.any() and torch.equal(r.dw, add) and r.loss.isfinite()
    y[7], y[11] = vocab, 1 << 40
    r = mica.mica_linear_cross_entropy(h, w, y, grad_scale=0.0, add=add)
    assert r.logps[7].isnan() and r.logps[11].isnan() and r.loss.isnan()
    assert not r.dh.any() and torch.equal(r.dw, add)


@pytest.mark.parametrize("rows", [300, 1500])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan, 3e38])
def test_one_coefficient_that_is_no_number(bad, rows):
    """An infinity or a NaN among small coefficients: its row's gradient and dw show it, the other rows' have the bits that they
    have without it. 3e38 leaves float32 when it is divided by the temperature."""
    h, w, y = make(rows, 200, 900, torch.float16, seed=45, skip=0.2)
    y[3] = 5
    lp, lse = mica.mica_linear_logps(h, w, y, temperature=0.5, lse=True)
    c = 1e-7 * torch.randn(rows, generator=gen(46), device="cuda")
    c[3] = 1e-9
    dh, _ = mica.mica_linear_logps_grad(h, w, y, lse, c, temperature=0.5, dw_dtype=torch.float32)
    exact = Want(h, w, y, 0.5).grads(c, torch.float16)
    rounded(dh, exact[0], exact[1])
    c[3] = bad
    got, dw = mica.mica_linear_logps_grad(h, w, y, lse, c, temperature=0.5, dw_dtype=torch.float32)
    assert not got[3].isfinite().any() and not dw.isfinite().all()
    rest = torch.arange(rows, device="cuda") != 3
    assert torch.equal(got[rest], dh[rest])


@pytest.mark.parametrize("vocab", [129, 200, 257, 70017])
@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_banned_target(dtype, vocab):
    """A token whose embedding makes every logit minus infinity, the last of the vocabulary, as a target and not: a
    log-probability of minus infinity, and the gradients of a probability of 0."""
    rows, features = 70, 72
    h, w, y = make(rows, features, vocab, dtype, seed=vocab, skip=0.2)
    h[:, 0] = h[:, 0].abs() + 1.0
    y[y == vocab - 1] = 0
    y[5], y[64] = vocab - 1, vocab - 1
    w[-1, 0] = -2000.0
    want = Want(h, w, y)  # (a probability of exp(-2000): 0 in float64 too)
    want.err = Want(h, w[:-1], y.clamp(max=vocab - 2)).err
    w[-1, 0] = -math.inf
    last = y == vocab - 1
    lp, lse = mica.mica_linear_logps(h, w, y, lse=True)
    close(lse, torch.where(want.on, want.lse, 0.0), want.err + U * want.lse.abs())
    n = int(want.on.sum())
    r = mica.mica_linear_cross_entropy(h, w, y, dw_dtype=torch.float32)
    for got in (lp, r.logps):
        assert (got[last] == -math.inf).all()
        close(got[~last], want.logps[~last], 2 * want.err[~last])
    assert float(r.loss) == math.inf
    c = torch.full((rows,), -1.0 / n, device="cuda")
    dh, dh_err, dw, dw_err = want.grads(c, dtype, once=True)
    two = mica.mica_linear_logps_grad(h, w, y, want.lse.float(), c, dw_dtype=torch.float32)
    for got_h, got_w in (r[2:], two):
        rounded(got_h[:, 1:], dh[:, 1:], dh_err[:, 1:])  # (the first feature's is 0 times an infinity)
        rounded(got_w, dw, dw_err)


@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_only_banned_tokens(dtype):
    """A row with nothing but minus infinities gives NaN, as 0 / 0 does; the others are as they were."""
    h, w, y = make(40, 64, 100, dtype, seed=47, skip=0.0)
    h[:, 0], w[:, 0] = 0.0, -1.0
    lp = mica.mica_linear_logps(h, w, y)
    h[3, 0] = math.inf
    got, lse = mica.mica_linear_logps(h, w, y, lse=True)
    r = mica.mica_linear_cross_entropy(h, w, y)
    assert got[3].isnan() and lse[3] == -math.inf and r.logps[3].isnan() and r.dh[3].isnan().all()
    rest = torch.arange(40, device="cuda") != 3
    assert torch.equal(got[rest], lp[rest]) and r.dh[rest].isfinite().all()


@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_one_gradient_of_no_rows(dtype):
    """Without rows there is nothing in dh, whose pointer is null, and the call is none the worse for it."""
    h, w = torch.empty(0, 72, dtype=dtype, device="cuda"), torch.ones(300, 72, dtype=dtype, device="cuda")
    y, none = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    r = mica.mica_linear_cross_entropy(h, w, y, want_dw=False)
    assert float(r.loss) == 0.0 and r.dh.shape == (0, 72) and r.dw is None
    dh, dw = mica.mica_linear_logps_grad(h, w, y, none, none, want_dw=False)
    assert dh.shape == (0, 72) and dw is None
    r = mica.mica_linear_cross_entropy(h, w, y, want_dh=False)
    assert r.dh is None and not r.dw.any()


def test_workspace_sizes():
    """The documented sum, of which the matrix of d is the largest part: up to 1 GB of it, and never fewer than 256 rows."""
    L = mica.train._train()

    def size(rows, features, vocab, sums, dw_dtype=0, ld_w=None):
        l = mica.train._Linear(None, 0x1000, None, rows, features, vocab, features, ld_w or features, 1.0, 4, 8)
        g = mica.train._LinearGrads(0x1000, 0x1000, None, features, features, 0, dw_dtype, 0)
        return L.mica_linear_cross_entropy_workspace(l, g) if sums else L.mica_linear_grad_workspace(l, g)

    def documented(rows, features, vocab, sums, dw_dtype=0, copied=False):
        up = lambda n: (n + 255) // 256 * 256  # noqa: E731
        piece = max(256, (1 << 30) // (2 * vocab) // 256 * 256)
        if sums:
            piece = min(piece, 16384, max(256, (256 << 20) // (vocab // 16) // 256 * 256))
        piece = min(up(rows), piece)
        total = 2 * piece * vocab + 2 * piece * features + (80 << 20) + 4 * rows
        if sums:
            total += piece * vocab // 16 + 2 * piece * features
        if copied:
            total += 2 * vocab * features
        if piece < rows and dw_dtype:
            total += 4 * vocab * features
        return total

    for args in ((8192, 768, 50257), (100, 64, 1000), (4096, 1600, 131072), (1500, 40, 600_007), (300, 16, 1 << 24), (40, 40_000, 60_000)):
        for sums in (False, True):
            for dt in (0, 4):
                got, want = size(*args, sums, dt), documented(*args, sums, dt)
                assert 0.9 * want <= got <= 1.1 * want + (1 << 20), (args, sums, dt, got, want)
    assert size(300, 16, 1 << 24, True) > 8 << 30  # 256 rows of 2^24
    got, want = size(512, 1001, 30_000, False, ld_w=1001), documented(512, 1001, 30_000, False, copied=True)
    assert 0.9 * want <= got <= 1.1 * want + (1 << 20)


@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_coefficients_at_the_end_of_float32(dtype):
    """Coefficients of up to 2.8e38, whose gradients float32 still holds: small hidden states, one row to a token."""
    rows, features, vocab = 120, 64, 900
    h, w, y = make(rows, features, vocab, dtype, seed=48, skip=0.1)
    h = (h.float() * 2.0 ** -6).to(dtype)
    y = torch.where(y < 0, y, torch.arange(rows, device="cuda"))
    lp, lse = mica.mica_linear_logps(h, w, y, lse=True)
    c = 2.8e38 * (2.0 * torch.rand(rows, generator=gen(49), device="cuda") - 1.0)
    c[1], c[2] = 2.8e38, -2.8e38
    want = Want(h, w, y)
    _, _, dw, dw_err = want.grads(c, dtype)
    assert float(dw.abs().max()) < 3e38
    got = mica.mica_linear_logps_grad(h, w, y, lse, c, want_dh=False, dw_dtype=torch.float32)[1]
    rounded(got, dw, dw_err)
    n = int(want.on.sum())
    for scale in (1e38, 2.8e38):
        r = mica.mica_linear_cross_entropy(h, w, y, denom=1.0, grad_scale=scale, want_dh=False, dw_dtype=torch.float32)
        _, _, dw, dw_err = want.grads(torch.full((rows,), -scale, device="cuda"), dtype, once=True)
        assert float(dw.abs().max()) < 3e38
        rounded(r.dw, dw, dw_err)


def test_cross_entropy_is_as_exact_as_its_roundings():
    """In the norm: dh is off by its own rounding, a float32 dw by one rounding of its rows. A rounding to bfloat16 is off by
    2^-8 / 3^1/2 (2^-2 <= u < 2^-1 in size: a root mean square of 2^-9 3^-1/2 / u, between 1.1e-3 and 2.3e-3, 1.66e-3 over all),
    and two of them by 2^1/2 as much: 2.35e-3. 2.0e-3 lies between one and two."""
    h, w, y = make(700, 256, 5000, torch.bfloat16, seed=50, skip=0.1)
    want = Want(h, w, y)
    n = int(want.on.sum())
    dh, _, dw, _ = want.grads(torch.full((700,), -1.0 / n, device="cuda"), torch.bfloat16)
    r = mica.mica_linear_cross_entropy(h, w, y, dw_dtype=torch.float32)
    for got, exact in ((r.dh, dh), (r.dw, dw)):
        assert float((got.double() - exact).norm()) <= 2.0e-3 * float(exact.norm())


@pytest.mark.parametrize("dtype", HALVES, ids=str)
def test_cross_entropy_rounds_what_it_says(dtype):
    """A float32 dw against a model in float64: binary16 rounds 2^14 (1[target] - p) and nothing else, whatever the number of
    rows; bfloat16 h's rows times a factor, and p where the target is not. Half as much again is allowed for p's own error (a few
    2^-22 against 2^-11) and for which way the roundings fall."""
    h, w, y = make(601, 256, 5000, dtype, seed=51, skip=0.1)
    want = Want(h, w, y)
    n = int(want.on.sum())
    c = torch.full((601,), -1.0 / n, device="cuda")
    _, _, dw, _ = want.grads(c, dtype)
    one = torch.zeros_like(want.p).scatter_(1, y.clamp(min=0)[:, None], 1.0)
    f = -want.on.double()[:, None] / n
    if dtype is torch.float16:
        model = ((one - want.p) * 2.0 ** 14).half().double().t() @ (want.h * f * 2.0 ** -14)
    else:
        p = torch.where(one > 0, want.p, want.p.bfloat16().double())
        model = (one - p).t() @ (want.h * f).bfloat16().double()
    r = mica.mica_linear_cross_entropy(h, w, y, dw_dtype=torch.float32)
    off = float((r.dw.double() - dw).norm())
    assert off <= 1.5 * float((model - dw).norm()), (off, float((model - dw).norm()), float(dw.norm()))
