"""The losses over logits against their definitions in float64: log-probabilities and their gradient, the preference loss
and the policy loss, over element types, odd sizes, strides, masks and the values that end in infinities and NaNs.

Tolerances, with u = 2^-24 (half a unit in the last place of float32). A row's sum of exponentials adds positive terms,
each off by a few u and by |x| u for its exponent x; a thread adds at most vocab / 128 of them in a row and a few dozen
joins follow, so log(sum) is off by at most (vocab / 128 + 64) u, and a log-probability by that and some u of its own size.
The gradient's rows inherit the same relative error, and round once to their type.
"""
import math

import pytest
import torch

import clip_tensor_adamw_gb300 as mica

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def rel(vocab):
    return (vocab / 128 + 64) * U


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make(rows, vocab, dtype, seed=0, ld=None, offset=0, index=torch.int64, skip=0.3):
    """Logits in a buffer of their own (row stride ld, first element at `offset`), and targets of which a share is
    skipped."""
    g = gen(seed)
    ld = vocab if ld is None else ld
    flat = torch.randn(offset + max(rows, 1) * max(ld, vocab), generator=g, device="cuda") * 3
    z = flat.to(dtype)[offset:].as_strided((rows, vocab), (ld, 1))
    y = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    y[torch.rand(rows, generator=g, device="cuda") < skip] = -100
    return z, y.to(index)


def reference(z, y, temperature=1.0):
    """(log-probabilities, entropies, softmax) in float64."""
    x = z.double() / temperature
    p = torch.softmax(x, 1)
    lp = torch.log_softmax(x, 1).gather(1, y.long().clamp(min=0)[:, None])[:, 0]
    h = torch.special.entr(p).sum(1)
    on = y >= 0
    return torch.where(on, lp, 0.0), torch.where(on, h, 0.0), p


def close(a, b, tol):
    a = a.double()
    bad = ~((a - b).abs() <= tol) & ~(a.isnan() & b.isnan()) & ~(a == b)
    assert not bad.any(), (int(bad.sum()), a[bad][:4], b[bad][:4])


def close_grad(d, want, p, c, vocab, c_tol=None):
    """d against want, rows of c * (onehot - p); c_tol: how far the coefficients themselves may be off."""
    c_tol = c.abs() * 8 * U if c_tol is None else c_tol
    share = (want / torch.where(c == 0, 1.0, c)[:, None]).abs()
    tol = c.abs()[:, None] * (p * rel(vocab) * 1.5 + 4 * U * share) + c_tol[:, None] * share
    close(d, want, tol + (want.abs() + tol) * ROUND[d.dtype] + TINY[d.dtype])


def grad_of(p, y, c):
    on = y >= 0
    want = -p * c[:, None]
    want.scatter_add_(1, y.long().clamp(min=0)[:, None], c[:, None])
    return torch.where(on[:, None], want, 0.0)


SHAPES = [(1, 1), (3, 7), (5, 33), (2, 257), (17, 1000), (9, 4099), (1, 50257), (40, 50257), (3, 65536), (2, 131079),
          (700, 130), (2, 300001)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_token_logps(rows, vocab, dtype):
    z, y = make(rows, vocab, dtype, seed=rows + vocab, skip=0.0 if rows == 1 else 0.3)
    for t in (1.0, 0.7):
        lp, h = mica.mica_token_logps(z, y, temperature=t, entropy=True)
        want, want_h, _ = reference(z, y, t)
        close(lp, want, rel(vocab) + 6 * U * want.abs() + 64 * U)
        close(h, want_h, 30 * rel(vocab))
        assert torch.equal(lp, mica.mica_token_logps(z, y, temperature=t))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_token_logps_grad(rows, vocab, dtype):
    z, y = make(rows, vocab, dtype, seed=2 * rows + vocab, index=torch.int32)
    c = torch.randn(rows, generator=gen(5), device="cuda")
    c[::3] = 0.0
    d = mica.mica_token_logps_grad(z, y, c, temperature=0.9)
    k = torch.where(y >= 0, c.double() / 0.9, 0.0)
    p = reference(z, y, 0.9)[2]
    close_grad(d, grad_of(p, y, k), p, k, vocab)
    assert not d[(y < 0) | (c == 0)].any()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("vocab,ld,offset", [(1003, 1003, 1), (1003, 1003, 3), (1003, 1024, 0), (1000, 1009, 5),
                                             (9001, 9004, 2), (513, 0, 0), (513, 0, 1), (50257, 50304, 7)])
def test_strides_and_offsets(vocab, ld, offset, dtype):
    """Rows at every alignment, and a matrix whose rows are all the same memory; the gradient written elsewhere, at
    another alignment, and in place."""
    rows = 11
    z, y = make(rows, vocab, dtype, seed=vocab + ld, ld=ld, offset=offset)
    c = torch.randn(rows, generator=gen(6), device="cuda")
    k = torch.where(y >= 0, c.double(), 0.0)
    want, _, p = reference(z, y)
    close(mica.mica_token_logps(z, y), want, rel(vocab) + 6 * U * want.abs() + 64 * U)
    base = torch.full((rows * (vocab + 5) + 16,), 7.0, dtype=dtype, device="cuda")
    for first, stride in ((offset, max(ld, vocab)), (0, vocab), (1, vocab + 2), (3, vocab + 5), (8, vocab + 3)):
        if first + (rows - 1) * stride + vocab > base.numel():
            continue
        base.fill_(7.0)
        out = base[first:].as_strided((rows, vocab), (stride, 1))
        d = mica.mica_token_logps_grad(z, y, c, out=out)
        assert d.data_ptr() == out.data_ptr()
        close_grad(d, grad_of(p, y, k), p, k, vocab)
        out.fill_(7.0)
        assert (base == 7.0).all()  # nothing outside the rows was written
    if ld:
        apart = mica.mica_token_logps_grad(z, y, c)
        d = mica.mica_token_logps_grad(z, y, c, out=z)
        close_grad(d, grad_of(p, y, k), p, k, vocab)
        assert torch.equal(d, apart)  # (the same bits for the same alignment of the rows)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("vocab", [9, 1500, 50257])
def test_masks_and_values(vocab, dtype):
    """Banned tokens, rows with nothing left, the type's lowest value, infinities and NaNs: the formula's values."""
    z, y = make(12, vocab, dtype, seed=vocab, skip=0.0)
    low, inf = torch.finfo(dtype).min, math.inf
    z[1, : vocab // 2] = -inf
    z[2, vocab // 3:] = low
    z[3] = -inf                      # nothing left: NaN
    z[4] = low                       # uniform
    z[5] = -inf
    z[5, vocab - 1] = -3.0           # one token left
    z[6, vocab // 2] = math.nan
    z[7, vocab // 2] = inf
    y[0], y[5] = 0, vocab - 1
    y[8] = -1                        # a row that does not count, whatever it holds
    z[8] = math.nan
    y[9] = -2 ** 40
    y[10] = vocab                    # past the vocabulary
    y[11] = 2 ** 40
    z[1, y[1]] = -inf                # a banned target
    lp, h = mica.mica_token_logps(z, y, entropy=True)
    inside = y.clamp(max=vocab - 1)
    want, want_h, p = reference(z, inside)
    want[10:] = math.nan
    close(lp, want, rel(vocab) + 6 * U * want.abs().nan_to_num(0, 0, 0) + 64 * U)
    close(h, want_h, 30 * rel(vocab))
    assert lp[1] == -inf and lp[3].isnan() and lp[5] == 0 and lp[6].isnan() and lp[7].isnan()
    assert abs(lp[4].item() + math.log(vocab)) < 1e-5 and lp[8] == 0 and lp[9] == 0
    c = torch.ones(12, device="cuda")
    d = mica.mica_token_logps_grad(z, y, c)
    k = torch.where(y >= 0, 1.0, 0.0).double()
    want_d = grad_of(p, inside, k)
    want_d[10:] = math.nan
    want_d[y < 0] = 0
    fine = [0, 1, 2, 4, 5, 8, 9]
    close_grad(d[fine], want_d[fine], p[fine].nan_to_num(0), k[fine], vocab)
    for r in (3, 6, 7, 10, 11):
        assert d[r].isnan().any(), r
    assert d[10].isnan().all()


def test_empty_and_refusals():
    z, y = make(4, 100, torch.float32)
    assert mica.mica_token_logps(z[:0], y[:0]).shape == (0,)
    assert mica.mica_token_logps_grad(z[:0], y[:0], torch.zeros(0, device="cuda")).shape == (0, 100)
    c = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        mica.mica_token_logps(z.double(), y)
    with pytest.raises(TypeError):
        mica.mica_token_logps(z, y.float())
    with pytest.raises(ValueError):
        mica.mica_token_logps(z, y[:3])
    with pytest.raises(ValueError):
        mica.mica_token_logps(z.t(), y)
    with pytest.raises(TypeError):
        mica.mica_token_logps_grad(z, y, c.double())
    for t in (0.0, -1.0, math.inf, math.nan, 1e-45, 1e45):
        with pytest.raises(mica.MicaError, match="HYPER"):
            mica.mica_token_logps(z, y, temperature=t)
    with pytest.raises(mica.MicaError, match="OVERLAP"):
        flat = torch.zeros(1000, device="cuda")
        mica.mica_token_logps_grad(flat[:400].view(4, 100), y, c, out=flat[1:401].view(4, 100))
    with pytest.raises(mica.MicaError, match="ADDRESS"):
        mica.mica_token_logps_grad(z, y, c, out=torch.empty(4, 100))
    with pytest.raises(ValueError):
        mica.mica_preference_loss(z, y, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        mica.mica_preference_loss(z, y, torch.zeros(3, device="cuda"))
    ends = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    for bad in (dict(beta=0.0), dict(beta=math.nan), dict(label_smoothing=1.0), dict(label_smoothing=-0.1),
                dict(kind="ipo", label_smoothing=0.1), dict(grad_scale=math.inf)):
        with pytest.raises(mica.MicaError, match="HYPER"):
            mica.mica_preference_loss(z, y, ends, **bad)
    with pytest.raises(ValueError):
        mica.mica_preference_loss(z, y, ends, kind="other")
    for bad in (dict(denom=0.0), dict(denom=math.inf), dict(clip_low=1.5), dict(clip_low=-0.1), dict(clip_high=-0.1),
                dict(kl_coef=-1.0), dict(kl_coef=math.nan), dict(grad_scale=math.nan)):
        with pytest.raises(mica.MicaError, match="HYPER"):
            mica.mica_policy_loss(z, y, c, c, **{"denom": 1.0, **bad})
    for T, V in ((0, 5), (0, 0)):
        s = mica.mica_policy_loss(torch.zeros(T, max(V, 1), device="cuda"), y[:T], c[:T], c[:T], denom=1.0)
        assert not s.stats.any()


# ----------------------------------------------------------------------------------------------------------------------
# preference loss
# ----------------------------------------------------------------------------------------------------------------------

def preference_reference(lp, on, ends, ref, beta, kind, smoothing, length_norm):
    """(loss, rewards, d loss / d lp) in float64, by autograd."""
    lp = lp.detach().clone().requires_grad_()
    d = []
    for a, b in zip(ends[:-1], ends[1:]):
        n = max(1, int(on[a:b].sum())) if length_norm else 1
        d.append(torch.where(on[a:b], lp[a:b] - ref[a:b], 0.0).sum() / n)
    d = torch.stack(d)
    gap = d[0::2] - d[1::2]
    f = torch.nn.functional
    if kind == "sigmoid":
        loss = -(1 - smoothing) * f.logsigmoid(beta * gap) - smoothing * f.logsigmoid(-beta * gap)
    elif kind == "hinge":
        loss = torch.relu(1 - beta * gap)
    else:
        loss = (gap - 1 / (2 * beta)) ** 2
    loss = loss.mean()
    return loss.detach(), beta * d.detach(), torch.autograd.grad(loss, lp)[0]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("lens,vocab", [([1, 1], 5), ([3, 0], 40), ([0, 0, 2, 9], 333), ([17, 40, 64, 33, 1, 5], 4099),
                                        ([130, 61], 50257), ([5] * 200, 130)])
@pytest.mark.parametrize("kind,smoothing,length_norm", [("sigmoid", 0.0, False), ("sigmoid", 0.2, True),
                                                        ("hinge", 0.0, False), ("ipo", 0.0, True)])
def test_preference_loss(lens, vocab, kind, smoothing, length_norm, dtype):
    lead, tail = 3, 2  # rows before the first sequence and after the last, which count for nothing
    ends = [lead]
    for n in lens:
        ends.append(ends[-1] + n)
    rows = ends[-1] + tail
    z, y = make(rows, vocab, dtype, seed=rows + vocab)
    on = y >= 0
    ref = reference(z, y)[0].float() + 0.3 * torch.randn(rows, generator=gen(3), device="cuda")
    beta, scale, t = 0.15, 3.0, 1.2
    cu = torch.tensor(ends, dtype=torch.int32, device="cuda")
    r = mica.mica_preference_loss(z, y, cu, ref, beta=beta, kind=kind, label_smoothing=smoothing, length_norm=length_norm,
                                  temperature=t, grad_scale=scale)
    lp, _, p = reference(z, y, t)
    loss, rewards, dlp = preference_reference(lp, on, ends, ref.double(), beta, kind, smoothing, length_norm)
    lp_tol = rel(vocab) + 6 * U * lp.abs() + 64 * U
    close(r.logps, lp, lp_tol)
    longest = max(max(lens), 1)
    d_tol = longest * float(lp_tol.max()) + 1e-30     # of a sequence's sum
    close(r.rewards, rewards, beta * d_tol + 2 * U * rewards.abs())
    gap = (rewards[0::2] - rewards[1::2]) / beta
    slope = 2 * (gap - 0.5 / beta).abs().max().item() if kind == "ipo" else beta
    close(r.loss, loss.reshape(1), 2 * d_tol * (slope + d_tol) + 4 * U * loss.abs())
    k = dlp * scale / t
    bend = 2.0 if kind == "ipo" else beta * beta / 4
    if kind == "hinge":
        assert ((1 - beta * gap).abs() > 10 * d_tol).all()  # no pair at the corner
        bend = 0.0
    c_tol = torch.full_like(k, 2 * d_tol * bend * scale / t / (len(lens) // 2)) + 8 * U * k.abs()
    close_grad(r.dlogits, grad_of(p, y, k), p, k, vocab, torch.where(on, c_tol, 0.0))
    assert not r.dlogits[:lead].any() and not r.dlogits[rows - tail:].any()
    alone = mica.mica_preference_loss(z, y, cu, ref, beta=beta, kind=kind, label_smoothing=smoothing,
                                      length_norm=length_norm, temperature=t, grad=False)
    assert alone.dlogits is None and torch.equal(alone.loss, r.loss) and torch.equal(alone.logps, r.logps)
    again = mica.mica_preference_loss(z, y.to(torch.int32), cu, ref, beta=beta, kind=kind, label_smoothing=smoothing,
                                      length_norm=length_norm, temperature=t, grad_scale=scale, out=z)
    assert again.dlogits.data_ptr() == z.data_ptr()
    for a, b in zip(r, again):  # in place, and the same bits
        assert torch.equal(a, b)


def test_preference_edges():
    z, y = make(8, 50, torch.float32, skip=0.0)
    none = mica.mica_preference_loss(z, y, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert none.loss.item() == 0 and none.rewards.numel() == 0 and not none.dlogits.any()
    # bounds past the rows are clamped, a sequence that ends before it starts is empty
    cu = torch.tensor([-5, 4, 900], dtype=torch.int32, device="cuda")
    fine = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    a, b = mica.mica_preference_loss(z, y, cu), mica.mica_preference_loss(z, y, fine)
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    back = mica.mica_preference_loss(z, y, torch.tensor([6, 2, 8], dtype=torch.int32, device="cuda"))
    assert back.rewards[0] == 0
    # a chosen sequence with a banned token, then a rejected one: infinite loss, zero loss
    z[1, y[1]] = -math.inf
    r = mica.mica_preference_loss(z, y, fine)
    assert r.loss.item() == math.inf and r.rewards[0] == -math.inf and r.dlogits.isfinite().all()
    r = mica.mica_preference_loss(z, y, torch.tensor([4, 8, 8], dtype=torch.int32, device="cuda"))
    assert r.loss.isfinite().all()
    swapped = mica.mica_preference_loss(z.flip(0).contiguous(), y.flip(0).contiguous(), fine)
    assert swapped.loss.item() == 0 and not swapped.dlogits.any()


# ----------------------------------------------------------------------------------------------------------------------
# policy loss
# ----------------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,vocab", [(1, 3), (5, 33), (64, 1000), (33, 9001), (20, 50257), (3, 131079), (1500, 130),
                                        (2, 300001)])
@pytest.mark.parametrize("ref,weighted", [(False, False), (True, True)])
def test_policy_loss(rows, vocab, ref, weighted, dtype):
    z, y = make(rows, vocab, dtype, seed=3 * rows + vocab, skip=0.0 if rows == 1 else 0.25)
    on = y >= 0
    lp, _, p = reference(z, y, 0.8)
    noise = lambda s: torch.randn(rows, generator=gen(s), device="cuda").double()  # noqa: E731
    lo, hi, kl, denom, scale = 0.2, 0.3, 0.1, 7.0, 2.5
    shift = 0.25 * noise(1)
    r = torch.exp(shift)
    shift = torch.where(((r - 0.8).abs() < 1e-3) | ((r - 1.3).abs() < 1e-3), 0.0, shift)  # not on the clip's edges
    old = (lp - shift).float()
    adv, w = noise(2).float(), (0.5 + noise(3).abs()).float()
    other = (lp + 0.2 * noise(4)).float()
    other[~on] = math.nan  # what is not scored is not read
    adv[~on] = math.nan
    got = mica.mica_policy_loss(z, y, old, adv, denom=denom, ref_logps=other if ref else None,
                                weights=w if weighted else None, clip_low=lo, clip_high=hi, kl_coef=kl, temperature=0.8,
                                grad_scale=scale)
    x = lp.clone().requires_grad_()
    a = torch.where(on, adv.double(), 0.0)
    r = torch.exp(x - old.double())
    held = torch.clamp(r, 1 - lo, 1 + hi) * a
    each = -torch.minimum(r * a, held)
    q = torch.where(on, other.double(), 0.0) - x
    k3 = torch.exp(q) - q - 1 if ref else torch.zeros_like(x)
    wt = torch.where(on, w.double() if weighted else 1.0, 0.0) / denom
    loss = (wt * (each + kl * k3)).sum()
    k = torch.autograd.grad(loss, x)[0] * scale / 0.8
    lp_tol = rel(vocab) + 6 * U * lp.abs() + 64 * U
    close(got.logps, lp, lp_tol)
    size = wt * ((r * a).abs() + (kl * (torch.exp(q) + 1) if ref else 0.0)).detach()
    each_tol = size * 2 * (lp_tol + 8 * U * (1 + old.abs()))
    parts = torch.stack([loss, (wt * each).sum(), (wt * k3).sum(), (wt * (held < r * a)).sum()]).detach()
    kl_tol = (wt * ((torch.exp(q) - 1).abs() * lp_tol + 8 * U * (torch.exp(q) + q.abs() + 1))).sum().item()
    s_tol = torch.tensor([each_tol.sum().item() + kl_tol, each_tol.sum().item(), kl_tol, 4 * U * parts[3].item()],
                         device="cuda", dtype=torch.float64)
    close(got.stats, parts, s_tol + 4 * U * parts.abs())
    close_grad(got.dlogits, grad_of(p, y, k), p, k, vocab, each_tol * scale / 0.8 + 8 * U * k.abs())
    assert not got.dlogits[~on].any()
    alone = mica.mica_policy_loss(z, y, old, adv, denom=denom, ref_logps=other if ref else None,
                                  weights=w if weighted else None, clip_low=lo, clip_high=hi, kl_coef=kl,
                                  temperature=0.8, grad=False)
    close(alone.stats, parts, s_tol + 4 * U * parts.abs())
    again = mica.mica_policy_loss(z, y.to(torch.int32), old, adv, denom=denom, ref_logps=other if ref else None,
                                  weights=w if weighted else None, clip_low=lo, clip_high=hi, kl_coef=kl,
                                  temperature=0.8, grad_scale=scale, out=z)
    assert again.dlogits.data_ptr() == z.data_ptr()
    for s, t in zip(got, again):
        assert torch.equal(s, t)


def test_policy_gradient_by_differences():
    """The gradient against central differences of the loss itself, in float64 (the loss taken from the definition and
    the gradient from the kernel)."""
    z, y = make(6, 40, torch.float32, seed=9, skip=0.2)
    lp = reference(z, y)[0]
    old = (lp - 0.1).float()
    adv = torch.randn(6, generator=gen(1), device="cuda")
    other = (lp + 0.2).float()
    d = mica.mica_policy_loss(z, y, old, adv, denom=3.0, ref_logps=other, kl_coef=0.2).dlogits

    def loss(x):
        on = y >= 0
        l = torch.log_softmax(x, 1).gather(1, y.clamp(min=0)[:, None])[:, 0]
        r = torch.exp(l - old.double())
        q = other.double() - l
        each = -torch.minimum(r * adv, torch.clamp(r, 0.8, 1.2) * adv) + 0.2 * (torch.exp(q) - q - 1)
        return torch.where(on, each, 0.0).sum() / 3.0

    x, step = z.double(), 1e-5
    for i in range(6):
        for j in (0, 13, int(y[i].clamp(min=0))):
            up, down = x.clone(), x.clone()
            up[i, j] += step
            down[i, j] -= step
            num = ((loss(up) - loss(down)) / (2 * step)).item()
            # the difference's own error is step^2 and 2^-52 / step, both under 1e-9
            assert abs(d[i, j].item() - num) < 1e-6, (i, j)


def test_streams_graphs_and_repeats():
    """On a side stream, and replayed from a graph on new logits in the same buffers: the same bits as a plain call."""
    z, y = make(48, 5003, torch.bfloat16, seed=1)
    cu = torch.tensor([0, 10, 20, 40, 48], dtype=torch.int32, device="cuda")
    old = mica.mica_token_logps(z, y) + 0.1
    adv = torch.randn(48, generator=gen(2), device="cuda")
    side = torch.cuda.Stream()

    def both(stream=None):
        a = mica.mica_preference_loss(z, y, cu, old, stream=stream)
        b = mica.mica_policy_loss(z, y, old, adv, denom=5.0, ref_logps=old, kl_coef=0.1, stream=stream)
        return [t for r in (a, b) for t in r]

    want = both()
    torch.cuda.synchronize()
    got = both(side)
    side.synchronize()
    raw = both(side.cuda_stream)
    side.synchronize()
    for a, b, c in zip(want, got, raw):
        assert torch.equal(a, b) and torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    z.copy_(torch.randn(48, 5003, generator=gen(8), device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(both(), held):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,vocab,ld,offset", [(700, 20011, 20011, 1), (640, 32768, 32768, 0), (1300, 16411, 16416, 3)])
def test_many_long_rows(rows, vocab, ld, offset, dtype):
    """Every operator over more long rows than there are CTAs, at every alignment: runs of rows that do not count,
    masked values, the gradient in place and elsewhere."""
    z, y = make(rows, vocab, dtype, seed=rows, ld=ld, offset=offset)
    y[100:300] = -1
    y[5] = vocab + 3
    z[7, 10:] = -math.inf
    y[7] = 4
    z[8] = torch.finfo(dtype).min
    inside = y.clamp(max=vocab - 1)
    want, want_h, p = reference(z, inside, 0.9)
    lp, h = mica.mica_token_logps(z, y, temperature=0.9, entropy=True)
    fine = torch.arange(rows, device="cuda") != 5
    tol = rel(vocab) + 6 * U * want.abs() + 64 * U
    close(lp[fine], want[fine], tol[fine])
    close(h[fine], want_h[fine], 30 * rel(vocab))
    assert lp[5].isnan()
    assert torch.equal(lp[fine], mica.mica_token_logps(z, y, temperature=0.9)[fine])
    y[5] = 3
    want, _, p = reference(z, y, 0.9)
    c = torch.randn(rows, generator=gen(5), device="cuda")
    c[::5] = 0.0
    k = torch.where(y >= 0, c.double() / 0.9, 0.0)
    d = mica.mica_token_logps_grad(z, y, c, temperature=0.9)
    close_grad(d, grad_of(p, y, k), p, k, vocab)
    elsewhere = torch.full((rows * (vocab + 3) + 9,), 7.0, dtype=dtype, device="cuda")
    out = elsewhere[2:].as_strided((rows, vocab), (vocab + 3, 1))
    mica.mica_token_logps_grad(z, y, c, temperature=0.9, out=out)
    assert torch.equal(out, d)
    out.fill_(7.0)
    assert (elsewhere == 7.0).all()
    # preference: pairs of 40 rows, one sequence empty
    cu = torch.arange(0, rows + 1, 20, dtype=torch.int32, device="cuda")[:31].clone()
    cu[4] = cu[5]
    ref = (reference(z, y)[0] + 0.1 * c).float()
    r = mica.mica_preference_loss(z, y, cu, ref, beta=0.1)
    lp64, _, p1 = reference(z, y)
    loss, rewards, dlp = preference_reference(lp64, y >= 0, cu.tolist(), ref.double(), 0.1, "sigmoid", 0.0, False)
    lp_tol = float((rel(vocab) + 6 * U * lp64.abs() + 64 * U).max())
    close(r.rewards, rewards, 0.1 * 40 * lp_tol + 2 * U * rewards.abs())
    close(r.loss, loss.reshape(1), 80 * 0.1 * lp_tol + 4 * U * loss)
    c_tol = torch.where(y >= 0, 80 * lp_tol * 0.0025 / 15 + 8 * U * dlp.abs(), 0.0)
    close_grad(r.dlogits, grad_of(p1, y, dlp), p1, dlp, vocab, c_tol)
    # policy, then both gradients in place: the same bits
    old = (lp64 + 0.05 * c).float()
    adv = torch.randn(rows, generator=gen(9), device="cuda")
    q = mica.mica_policy_loss(z, y, old, adv, denom=100.0, ref_logps=ref, kl_coef=0.1, clip_low=1.0, clip_high=math.inf)
    x = lp64.clone().requires_grad_()
    ratio, kq = torch.exp(x - old.double()), ref.double() - x
    each = torch.where(y >= 0, -ratio * adv + 0.1 * (torch.exp(kq) - kq - 1), 0.0)
    k = torch.autograd.grad(each.sum() / 100, x)[0]
    size = (torch.where(y >= 0, (ratio * adv).abs() + 0.1 * (torch.exp(kq) + 1), 0.0) / 100).detach()
    each_tol = size * 2 * (lp_tol + 8 * U * (1 + old.abs()))
    close(q.stats[0], (each.sum() / 100).detach(), float(each_tol.sum()) + 1e-6 * float(size.sum()))
    close_grad(q.dlogits, grad_of(p1, y, k), p1, k, vocab, each_tol + 8 * U * k.abs())
    copy = z.clone() if ld == vocab else None
    again = mica.mica_policy_loss(z, y, old, adv, denom=100.0, ref_logps=ref, kl_coef=0.1, clip_low=1.0,
                                  clip_high=math.inf, out=z)
    assert torch.equal(again.dlogits, q.dlogits) and torch.equal(again.stats, q.stats)
    if copy is not None:
        z.copy_(copy)
        again = mica.mica_preference_loss(z, y, cu, ref, beta=0.1, out=z)
        assert torch.equal(again.dlogits, r.dlogits)
    mica.mica_sync()


def test_many_long_rows_in_a_graph_and_on_two_streams():
    """Rows handed out by the hardware: replayed from a graph on new logits, and by two launches at once."""
    rows, vocab = 900, 18001
    z, y = make(rows, vocab, torch.bfloat16, seed=4)
    c = torch.randn(rows, generator=gen(2), device="cuda")
    graph = torch.cuda.CUDAGraph()
    mica.mica_token_logps_grad(z, y, c)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = [mica.mica_token_logps(z, y), mica.mica_token_logps_grad(z, y, c)]
    for seed in (5, 6):
        z.copy_(make(rows, vocab, torch.bfloat16, seed=seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[0], mica.mica_token_logps(z, y))
        assert torch.equal(held[1], mica.mica_token_logps_grad(z, y, c))
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a = [mica.mica_token_logps_grad(z, y, c, stream=s) for s in (one, two, one, two)]
    torch.cuda.synchronize()
    for d in a:
        assert torch.equal(d, held[1])
    mica.mica_sync()


def peaked(rows, vocab, gap, dtype, seed=0):
    """Rows with one likely token, a target `gap` below it, and the others so far below that they add nothing: (logits,
    targets, entropies in float64)."""
    g = gen(seed)
    z = -150.0 - torch.rand((rows, vocab), generator=g, device="cuda")
    likely = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    y = (likely + torch.randint(1, vocab, (rows,), generator=g, device="cuda")) % vocab
    at = torch.arange(rows, device="cuda")
    z[at, likely] = 20.0
    z[at, y] = 20.0 - gap
    z = z.to(dtype)
    return z, y, reference(z, y)[1]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,vocab", [(12, 1009), (9, 50257), (320, 16411)])  # the row kernel, clusters of it, the ring
def test_entropy_of_confident_rows(rows, vocab, dtype):
    """An unlikely target leaves the entropy its digits, and above 0. The row's sum is 1 + w, w = e^-gap (the other tokens'
    weights are under e^-150): one rounding, u, and log of it another. The moment is w gap: the exponent of w is off by
    gap / ln 2 of some u, the power of two by 4 u, the products and joins by 12 u more."""
    for gap in (1.0, 8.0, 15.0, 20.5, 25.0, 30.0, 41.0, 60.0):
        z, y, want = peaked(rows, vocab, gap, dtype, seed=int(gap))
        lp, h = mica.mica_token_logps(z, y, entropy=True)
        assert (h >= 0).all(), (gap, float(h.min()))
        close(h, want, 2 * U + (2 * gap + 16) * U * want)
        close(lp, reference(z, y)[0], (2 * gap + 16) * U * (1 + gap))
        other = (y + 1) % vocab  # (an even less likely target)
        close(mica.mica_token_logps(z, other, entropy=True)[1], want, 2 * U + (2 * gap + 16) * U * want)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,vocab", [(40, 1000), (11, 50257), (330, 20011)])
def test_entropy_does_not_depend_on_the_target(rows, vocab, dtype):
    """The same rows with likely and unlikely targets. An entropy is log(sum) plus the mean of -x: the sum is off by
    rel(vocab), and both sides of the mean by as much again and by some 8 u, so by rel(vocab) * (1 + 2 h) + 8 u h."""
    z, y = make(rows, vocab, dtype, seed=vocab, skip=0.0)
    want = reference(z, y)[1]
    for target in (y, z.float().argmin(1), z.float().argmax(1)):
        h = mica.mica_token_logps(z, target, entropy=True)[1]
        close(h, want, rel(vocab) * (1 + 2 * want) + 8 * U * want)


@pytest.mark.parametrize("length_norm", [False, True])
def test_long_sequences_that_nearly_cancel(length_norm):
    """Two long sequences alike but for one row, and no reference policy: the sums are some -3e4, of which float32 has 2e-3,
    and their difference that of one row. The rows alike cancel exactly, so what may be off is the one row's two
    log-probabilities, and 2^-40 of the sums."""
    n, vocab, beta = 1500, 64, 0.5
    g = gen(11)
    z = torch.randn((n, vocab), generator=g, device="cuda")
    y = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    z[torch.arange(n, device="cuda"), y] -= 15.0
    z, y = torch.cat([z, z]), torch.cat([y, y])
    z[n + 700, y[700]] += 0.37
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    r = mica.mica_preference_loss(z, y, cu, beta=beta, kind="ipo", length_norm=length_norm)
    lp, _, p = reference(z, y)
    share = 1.0 / n if length_norm else 1.0
    gap = ((lp[700] - lp[n + 700]) * share - 0.5 / beta).item()
    lp_tol = 2 * (rel(vocab) + 6 * U * 25 + 64 * U) * share + 2.0 ** -40 * 3e4 * share
    assert abs(lp[:n].sum().item()) > 2e4
    close(r.loss, torch.tensor([gap * gap], dtype=torch.float64, device="cuda"), 2 * abs(gap) * lp_tol + 4 * U * gap * gap)
    k = torch.cat([torch.full((n,), 2 * gap * share), torch.full((n,), -2 * gap * share)]).double().cuda()
    close_grad(r.dlogits, grad_of(p, y, k), p, k, vocab, torch.full_like(k, 2 * lp_tol * share) + 8 * U * k.abs())
    # the difference of the gradient's two coefficients of a row alike in both is exactly twice the one
    assert torch.equal(r.dlogits[:700], -r.dlogits[n:n + 700])


@pytest.mark.parametrize("rows,vocab", [(9, 50), (9, 50257), (310, 33001)])  # few short rows, few long ones, many
def test_targets_past_the_vocabulary_in_no_sequence(rows, vocab):
    """A row in no sequence gets zeros, whatever its target; one in a sequence makes its pair's loss and gradient NaN."""
    z, y = make(rows, vocab, torch.bfloat16, seed=vocab, skip=0.0)
    y[rows - 1] = vocab
    cu = torch.tensor([1, 3, 4, 6, 8], dtype=torch.int32, device="cuda")
    r = mica.mica_preference_loss(z, y, cu)
    assert r.logps[rows - 1].isnan() and r.loss.isfinite().all()
    assert not r.dlogits[0].any() and not r.dlogits[8:].any() and r.dlogits[1:8].any(1).all()
    y[2] = vocab + 7
    r = mica.mica_preference_loss(z, y, cu)
    assert r.loss.isnan().all() and r.dlogits[1:4].isnan().any(1).all() and r.dlogits[2].isnan().all()
    assert r.dlogits[4:8].isfinite().all() and not r.dlogits[0].any() and not r.dlogits[8:].any()


@pytest.mark.parametrize("rows,vocab", [(12, 1009), (9, 50257), (320, 16411), (310, 41003)])
def test_float32_gradient_of_confident_rows(rows, vocab):
    """The softmax of a row's likeliest token is its weight's share of the sum that has that weight in it, so it is off by a
    few u however far the target is: the sum's rounding, the reciprocal's and three products'. (The row kernel, clusters of
    it, and both rings.)"""
    for t in (1.0, 0.7):
        for gap in (3.0, 11.0, 20.0, 26.5):
            z, y, _ = peaked(rows, vocab, gap, torch.float32, seed=int(gap))
            p = reference(z, y, t)[2]
            c = torch.ones(rows, device="cuda")
            d = mica.mica_token_logps_grad(z, y, c, temperature=t)
            close(d, grad_of(p, y, c.double() / t), (8 * U * p + 8 * U) / t + 1e-30)
            likely = z.argmax(1, keepdim=True)
            top = d.gather(1, likely).double() * t
            close(top, -p.gather(1, likely), 8 * U * torch.ones_like(top))
            n = rows // 2
            cu = torch.tensor([0, n, rows], dtype=torch.int32, device="cuda")
            r = mica.mica_preference_loss(z, y, cu, beta=0.1, kind="ipo", temperature=t)
            k = r.dlogits.double().gather(1, y[:, None]) / (1.0 - p.gather(1, y[:, None]))  # the rows' coefficients
            close(r.dlogits.gather(1, likely).double() / k, -p.gather(1, likely), 16 * U * torch.ones_like(top))


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_banned_tokens_at_extreme_temperatures(dtype):
    """log2(e) / temperature in two floats, the second of which may be below float32's least: a banned token's weight is 0
    at any temperature."""
    near = []
    a = torch.tensor(1.5e-30, dtype=torch.float32)
    while len(near) < 3:  # temperatures whose quotient is a little above a float32
        a = torch.nextafter(a, torch.tensor(1.0))
        t = 1.4426950408889634074 / a.item()
        for _ in range(4):
            rest = 1.4426950408889634074 / t - a.item()
            if 0 < rest < 2.0 ** -150 and t <= 1e30:
                near.append(t)
                break
            t = math.nextafter(t, 0.0)
    vocab = 101
    for t in near + [1e30, 1e-30, 1e20, 1e-20]:
        z, y = make(7, vocab, dtype, seed=3, skip=0.0)
        z[:, 60:] = -math.inf
        y %= 60
        z[torch.arange(7), y] = 40.0  # (the likeliest by far where the temperature is low)
        lp, h = mica.mica_token_logps(z, y, temperature=t, entropy=True)
        want, want_h, p = reference(z, y, t)
        close(lp, want, rel(vocab) + 6 * U * want.abs() + 64 * U)
        close(h, want_h, 30 * rel(vocab))
        d = mica.mica_token_logps_grad(z, y, torch.full((7,), min(t, 1.0), device="cuda"), temperature=t)
        assert not d.isnan().any() and not d[:, 60:].any()


def test_sync_reads_no_status_of_kernels_that_never_ran():
    """mica_sync copies back the status words of kernels with bounded waits: those of the operators before the step only
    in a process that has launched them."""
    import os
    import subprocess
    import sys
    code = """
import torch
from torch.profiler import ProfilerActivity, profile
import clip_tensor_adamw_gb300 as mica
g = mica.TensorList([torch.ones(5000, device="cuda")])
z = torch.randn(400, 20000, device="cuda")
y = torch.zeros(400, dtype=torch.int64, device="cuda")
mica.mica_clip_grad_norms(g, 1.0)
mica.mica_sync()
def copies():
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CPU, ProfilerActivity.CUDA]) as p:
        mica.mica_sync()
        torch.cuda.synchronize()
    return sum("memcpy" in e.name.lower() and "dtoh" in e.name.lower().replace(" ", "") for e in p.events())
copies()
before = copies()
mica.mica_token_logps(z, y)
print("copies", before, copies())
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stderr
    before, after = map(int, out.stdout.split("copies")[1].split())
    if after == 0:
        pytest.skip("no record of copies on this machine")
    assert (before, after) == (2, 3)


@pytest.mark.parametrize("dtype,rows,vocab,ld,offset", [
    (torch.bfloat16, 320, 50257, 50257, 0), (torch.float16, 310, 50257, 50260, 3),      # unaligned 16-bit rows over 64 KB
    (torch.bfloat16, 305, 90001, 90001, 1), (torch.float16, 304, 98304, 98304, 0),      # rows over 160 KB
    (torch.float32, 303, 41003, 41003, 0), (torch.float32, 304, 45056, 45060, 2)], ids=str)
def test_gradients_of_many_longer_rows(dtype, rows, vocab, ld, offset):
    """What test_many_long_rows has no rows long enough for: the gradient's ring over long rows and over unaligned ones."""
    z, y = make(rows, vocab, dtype, seed=vocab, ld=ld, offset=offset)
    y[50:90] = -1
    z[7, 10:] = -math.inf
    y[7] = 4
    c = torch.randn(rows, generator=gen(5), device="cuda")
    c[::5] = 0.0
    k = torch.where(y >= 0, c.double() / 0.9, 0.0)
    p = reference(z, y, 0.9)[2]
    d = mica.mica_token_logps_grad(z, y, c, temperature=0.9)
    close_grad(d, grad_of(p, y, k), p, k, vocab)
    apart = torch.full((rows * (vocab + 1) + 8,), 7.0, dtype=dtype, device="cuda")
    out = apart[1:].as_strided((rows, vocab), (vocab + 1, 1))
    mica.mica_token_logps_grad(z, y, c, temperature=0.9, out=out)
    assert torch.equal(out, d)
    out.fill_(7.0)
    assert (apart == 7.0).all()
    del apart, out
    lp64, _, p = reference(z, y)
    lp_tol = float((rel(vocab) + 6 * U * lp64.abs() + 64 * U).max())
    old = (lp64 + 0.05 * c).float()
    adv = torch.randn(rows, generator=gen(9), device="cuda")
    q = mica.mica_policy_loss(z, y, old, adv, denom=100.0, clip_low=1.0, clip_high=math.inf)
    k = torch.where(y >= 0, -torch.exp(lp64 - old.double()) * adv / 100, 0.0)
    c_tol = k.abs() * (2 * lp_tol + 16 * U * (1 + old.abs()))
    close_grad(q.dlogits, grad_of(p, y, k), p, k, vocab, c_tol)
    cu = torch.arange(0, rows + 1, 60, dtype=torch.int32, device="cuda")[:5].clone()
    r = mica.mica_preference_loss(z, y, cu, old, beta=0.1)
    loss, rewards, dlp = preference_reference(lp64, y >= 0, cu.tolist(), old.double(), 0.1, "sigmoid", 0.0, False)
    close(r.rewards, rewards, 0.1 * 60 * lp_tol + 2 * U * rewards.abs())
    c_tol = torch.where(y >= 0, 120 * lp_tol * 0.0025 / 2 + 8 * U * dlp.abs(), 0.0)
    close_grad(r.dlogits, grad_of(p, y, dlp), p, dlp, vocab, c_tol)
    again = z.clone(memory_format=torch.preserve_format) if ld == vocab else None
    assert torch.equal(mica.mica_policy_loss(z, y, old, adv, denom=100.0, clip_low=1.0, clip_high=math.inf,
                                             out=z).dlogits, q.dlogits)
    if again is not None and offset == 0:
        assert torch.equal(mica.mica_preference_loss(again, y, cu, old, beta=0.1, out=again).dlogits, r.dlogits)
    mica.mica_sync()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("vocab", [1000, 16411])  # the row kernel, the ring
def test_log_probabilities_err_to_both_sides(vocab, dtype):
    """A preference loss adds up a sequence's log-probabilities, so what counts is their error's mean. Rounding one, under 16 in
    size, is off by 0.29 * 2^-20 on average either way, the mean of 4,000 by 4.4e-9: 5 of those, and 2e-8 for the rest."""
    rows = 4000
    z, y = make(rows, vocab, dtype, seed=vocab, skip=0.0)
    z.mul_(torch.linspace(0.2, 1.0, rows, device="cuda").to(dtype)[:, None])
    near = z.float().topk(30, 1).indices[torch.arange(rows, device="cuda"), torch.randint(0, 30, (rows,), generator=gen(1),
                                                                                         device="cuda")]
    for target in (near, y):
        want = reference(z, target)[0]
        fine = want > -16
        assert fine.sum() > 3000
        e = (mica.mica_token_logps(z, target).double() - want)[fine]
        assert abs(e.mean().item()) < 4.2e-8 * math.sqrt(4000 / len(e)), e.mean().item()


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,vocab,ld,offset", [(4100, 1537, 1537, 1), (4500, 2048, 2048, 0), (4096, 4099, 4104, 3),
                                                  (4097, 12301, 12301, 0)])
def test_very_many_short_rows(rows, vocab, ld, offset, dtype):
    """Log-probabilities and entropies of short rows in such number that they take the ring: part of a stage, or one and a
    part; runs of rows that do not count, masked values."""
    z, y = make(rows, vocab, dtype, seed=rows, ld=ld, offset=offset)
    y[1000:2500] = -1
    y[5] = vocab + 3
    z[7, 10:] = -math.inf
    y[7] = 4
    z[8] = torch.finfo(dtype).min
    z[9] = -math.inf
    z[10, vocab // 2] = math.nan
    z[11, vocab - 1] = math.inf
    z[12, y[12]] = -math.inf
    y[[8, 9, 10, 11]] = 1
    want, want_h, _ = reference(z, y.clamp(max=vocab - 1), 0.9)
    want[5] = math.nan
    lp, h = mica.mica_token_logps(z, y, temperature=0.9, entropy=True)
    close(lp, want, rel(vocab) + 6 * U * want.abs().nan_to_num(0, 0, 0) + 64 * U)
    close(h, want_h, rel(vocab) * (1 + 2 * want_h.nan_to_num(0)) + 8 * U * want_h.nan_to_num(0))
    assert lp[[5, 9, 10, 11]].isnan().all() and lp[12] in (0, -math.inf) and not lp[y < 0].any() and not h[y < 0].any()
    alone = mica.mica_token_logps(z, y, temperature=0.9)
    assert torch.equal(lp.view(torch.int32), alone.view(torch.int32))
    mica.mica_sync()
