"""The losses from hidden states and the orthogonalised step without a GPU: bad arguments are refused on the host, before
anything reaches a device, with the documented status; workspace sizes; and the binding's own checks."""
import ctypes
import math
import random

import pytest
import torch

import clip_tensor_adamw_gb300 as mica
from clip_tensor_adamw_gb300 import muon, train

OK, NULL, COUNT, DTYPE, HYPER = 0, 1, 2, 3, 4
F32, F16, BF16X2, BF16 = 0, 1, 2, 4


def linear(**kw):
    d = dict(h=0x1000, w=0x2000, targets=0x3000, rows=4, features=64, vocab=100, ld_h=64, ld_w=64, temperature=1.0, dtype=BF16,
             target_bytes=8)
    d.update(kw)
    return train._Linear(*(d[k] for k, _ in train._Linear._fields_))


def grads(**kw):
    d = dict(dh=0x4000, dw=0x5000, add=None, ld_dh=64, ld_dw=64, ld_add=64, dw_dtype=F32, reserved=0)
    d.update(kw)
    return train._LinearGrads(*(d[k] for k, _ in train._LinearGrads._fields_))


def hp(denom=0.0, grad_scale=1.0):
    return train._CrossEntropyHP(denom, grad_scale)


BAD = [(dict(dtype=F32), DTYPE), (dict(dtype=BF16X2), DTYPE), (dict(target_bytes=2), DTYPE), (dict(temperature=0.0), HYPER),
       (dict(temperature=math.nan), HYPER), (dict(temperature=math.inf), HYPER), (dict(temperature=-1.0), HYPER),
       (dict(temperature=2.0 ** 21), HYPER), (dict(rows=-1), COUNT), (dict(rows=(1 << 30) + 1), COUNT), (dict(vocab=0), COUNT),
       (dict(vocab=(1 << 24) + 1), COUNT), (dict(features=0), COUNT), (dict(features=(1 << 16) + 1), COUNT), (dict(ld_h=-1), COUNT),
       (dict(ld_w=-1), COUNT), (dict(ld_w=1 << 41), COUNT), (dict(rows=1 << 30, ld_h=1 << 40), COUNT)]


@pytest.mark.parametrize("bad,want", BAD)
def test_hidden_states_are_checked_by_every_call(bad, want):
    L = train._train()
    l = linear(**bad)
    assert L.mica_linear_logps(l, 0x6000, None, 0x7000, 1 << 40, None) == want
    assert L.mica_linear_logps_grad(l, 0x6000, 0x6100, grads(), 0x7000, 1 << 40, None) == want
    assert L.mica_linear_cross_entropy(l, hp(), 0x6000, 0x6100, grads(), 0x7000, 1 << 40, None) == want
    assert L.mica_linear_logps_workspace(l) == 0
    assert L.mica_linear_grad_workspace(l, grads()) == 0 and L.mica_linear_cross_entropy_workspace(l, None) == 0


def test_linear_host_validation():
    L = train._train()
    assert L.mica_linear_logps(None, 0x6000, None, 0x7000, 1 << 40, None) == NULL
    assert L.mica_linear_logps(linear(rows=0), None, None, None, 0, None) == OK
    assert L.mica_linear_logps_workspace(linear(rows=0)) == 0 and L.mica_linear_logps_workspace(linear()) > 0

    def g(**kw):
        return L.mica_linear_logps_grad(linear(), 0x6000, 0x6100, grads(**kw), 0x7000, 1 << 40, None)

    assert L.mica_linear_logps_grad(linear(), 0x6000, 0x6100, None, 0x7000, 1 << 40, None) == NULL
    assert g(dh=None, dw=None) == NULL and g(dw=None, add=0x8000) == NULL
    assert g(dw_dtype=BF16X2) == DTYPE and g(dw_dtype=9) == DTYPE
    assert g(ld_dh=63) == COUNT and g(ld_dw=63) == COUNT and g(add=0x8000, ld_add=-1) == COUNT

    def c(h, **kw):
        return L.mica_linear_cross_entropy(linear(**kw), h, 0x6000, 0x6100, grads(), 0x7000, 1 << 40, None)

    assert c(None) == NULL
    for bad in (hp(denom=-1.0), hp(denom=math.inf), hp(denom=math.nan), hp(denom=1e31), hp(denom=1e-31), hp(grad_scale=math.nan),
                hp(grad_scale=math.inf)):
        assert c(bad) == HYPER


def test_linear_binding_checks():
    h, w, y = torch.zeros(4, 64).bfloat16(), torch.zeros(100, 64).bfloat16(), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        mica.mica_linear_logps(h.float(), w.float(), y)
    with pytest.raises(TypeError):
        mica.mica_linear_logps(h, w.half(), y)
    with pytest.raises(ValueError):
        mica.mica_linear_logps(h, w[:, :63], y)
    with pytest.raises(ValueError):
        mica.mica_linear_logps(h, w.t().contiguous().t(), y)
    with pytest.raises(TypeError):
        mica.mica_linear_logps(h, w, y.float())
    with pytest.raises(ValueError):
        mica.mica_linear_logps(h, w, y[:3])
    with pytest.raises(TypeError):
        mica.mica_linear_logps_grad(h, w, y, torch.zeros(4).double(), torch.zeros(4))
    with pytest.raises(ValueError):
        mica.mica_linear_cross_entropy(h, w, y, denom=0.0)


def sizes(*shapes):
    T = len(shapes)
    arr = ctypes.c_int64 * max(T, 1)
    return arr(*(s[0] for s in shapes)), arr(*(s[1] for s in shapes)), T


def iteration(coefficients=(3.4445, -4.775, 2.0315) * 5, eps=1e-7, steps=5, flags=0):
    return muon._NewtonSchulz((ctypes.c_double * max(1, len(coefficients)))(*coefficients), eps, steps, flags)


def step(**kw):
    d = dict(lr=0.1, momentum=0.9, weight_decay=0.0, nesterov=1, adjust=0, zero_grad=0, flags=0)
    d.update(kw)
    return muon._MuonHP(*(d[k] for k, _ in muon._MuonHP._fields_))


def orthogonalize(shapes=((8, 8),), x=F32, out=F16, ns=None, work=None, size=0):
    rows, cols, T = sizes(*shapes)
    p = (ctypes.c_void_p * max(T, 1))(*([0x1000] * T))
    return muon._muon().mica_orthogonalize(p, p, rows, cols, T, x, out, ns if ns is not None else iteration(), work, size, None)


def steps(hp=None, shapes=((8, 8),), g=F32, ns=None):
    rows, cols, T = sizes(*shapes)
    p = (ctypes.c_void_p * max(T, 1))(*([0x1000] * T))
    return muon._muon().mica_muon_steps(p, p, p, rows, cols, T, g, hp, ns if ns is not None else iteration(), None, None, 0, None)


def test_muon_host_validation():
    M = muon._muon()
    assert orthogonalize(shapes=()) == OK and steps(step(), shapes=()) == OK and orthogonalize(shapes=((0, 5), (5, 0))) == OK
    for shape in ((-1, 4), (4, -1), ((1 << 17) + 1, 1), (1, (1 << 17) + 1)):
        assert orthogonalize(shapes=(shape,)) == COUNT and steps(step(), shapes=(shape,)) == COUNT
    assert M.mica_orthogonalize(None, None, None, None, 1, F32, F16, iteration(), None, 0, None) == NULL
    assert M.mica_orthogonalize(None, None, None, None, -1, F32, F16, iteration(), None, 0, None) == COUNT
    assert M.mica_orthogonalize(None, None, None, None, (1 << 20) + 1, F32, F16, iteration(), None, 0, None) == COUNT
    assert orthogonalize(x=BF16X2) == DTYPE and orthogonalize(out=F32) == DTYPE and orthogonalize(out=BF16X2) == DTYPE
    assert steps(step(), g=BF16) == DTYPE and steps(step(), g=BF16X2) == DTYPE
    assert steps(None) == NULL
    for bad in (dict(lr=-1.0), dict(lr=math.nan), dict(lr=math.inf), dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=math.nan),
                dict(weight_decay=-1.0), dict(weight_decay=math.inf), dict(adjust=3), dict(adjust=-1), dict(flags=2)):
        assert steps(step(**bad)) == HYPER, bad
    for bad in (dict(eps=0.0), dict(eps=1e-31), dict(eps=1.5), dict(eps=math.nan), dict(steps=0), dict(steps=17), dict(flags=2),
                dict(coefficients=(math.nan, 0.0, 0.0) * 5), dict(coefficients=(math.inf, 0.0, 0.0) * 5),
                dict(coefficients=(6.0, 0.0, 0.0) * 5), dict(coefficients=(33.0, 0.0, 0.0), steps=1)):
        assert orthogonalize(ns=iteration(**bad)) == HYPER and steps(step(), ns=iteration(**bad)) == HYPER, bad
    null = muon._NewtonSchulz(None, 1e-7, 5, 0)
    assert orthogonalize(ns=null) == NULL
    assert M.mica_orthogonalize(None, None, *sizes((8, 8)), F32, F16, None, None, 0, None) == NULL


def test_muon_workspace():
    M = muon._muon()

    def size(*shapes, flags=0):
        return M.mica_newton_schulz_workspace(*sizes(*shapes), flags)

    assert size((-1, 4)) == 0 and size() == 0 and size((0, 9)) == 0
    large = size((1600, 6400))
    assert large >= 1600 * 6400 * 4 + 1600 * 1600 * 4
    assert size((1600, 6400), flags=1) >= 2 * large - (40 << 20)
    # a list is taken in batches: its workspace is the largest one's
    many = size(*[(4096, 4096)] * 40)
    assert many < 128 * 2 ** 20 * 9
    assert size((1600, 6400), (6400, 1600)) == size((6400, 1600), (1600, 6400))


def test_muon_binding_checks():
    x = torch.zeros(4, 5)
    for f in (lambda: mica.mica_orthogonalize([torch.zeros(4)]), lambda: mica.mica_orthogonalize([x], coefficients=(1.0, 2.0)),
              lambda: mica.mica_orthogonalize([x], steps=3, coefficients=[(1.0, 0.0, 0.0)] * 2),
              lambda: mica.mica_muon_steps([x], [x.t().contiguous()], [x], lr=0.1),
              lambda: mica.mica_muon_steps([x], [x], [x, x], lr=0.1),
              lambda: mica.mica_muon_steps([x], [x], [x], lr=0.1, adjust="other"),
              lambda: mica.mica_muon_steps([x], [x], [x], lr=0.1, factor=torch.ones(1).half()),
              lambda: mica.mica_muon_steps([x], [x], [x], lr=0.1, factor=torch.ones(2))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        mica.mica_orthogonalize([x.double()])
    with pytest.raises(TypeError):
        mica.mica_muon_steps([x.half()], [x], [x], lr=0.1)
    with pytest.raises(TypeError):
        mica.mica_muon_steps([x], [x], [x.half()], lr=0.1)


def test_no_rows_and_no_gradients():
    """Without rows dh has no elements and its pointer may be null; with rows a gradient has to go somewhere."""
    L = train._train()
    none = grads(dh=None, dw=None)
    assert L.mica_linear_logps_grad(linear(rows=0), None, None, none, None, 0, None) == OK
    assert L.mica_linear_grad_workspace(linear(rows=0), none) == 0
    assert L.mica_linear_logps_grad(linear(rows=0), None, None, grads(dh=None, dw=None, add=0x8000), None, 0, None) == NULL
    assert L.mica_linear_cross_entropy(linear(), hp(), 0x6000, 0x6100, none, 0x7000, 1 << 40, None) == NULL


def test_dropped_arguments():
    """What cannot be filled is refused, not dropped: a gradient's buffer, or what is added to it, where none is wanted."""
    h, w, y = torch.zeros(4, 64).bfloat16(), torch.zeros(100, 64).bfloat16(), torch.zeros(4, dtype=torch.int64)
    z, dw, dh = torch.zeros(4), torch.zeros(100, 64), torch.zeros(4, 64).bfloat16()
    for kw in (dict(grad=False, dw=dw), dict(grad=False, add=dw), dict(grad=False, dh=dh), dict(want_dw=False, dw=dw),
               dict(want_dw=False, add=dw), dict(want_dh=False, dh=dh), dict(want_dh=False, want_dw=False, dw=dw)):
        with pytest.raises(ValueError, match="given"):
            mica.mica_linear_cross_entropy(h, w, y, **kw)
        if "grad" not in kw:
            with pytest.raises(ValueError, match="given"):
                mica.mica_linear_logps_grad(h, w, y, z, z, **kw)


def test_output_of_another_type():
    """out_dtype beside out has to be out's."""
    x = torch.zeros(4, 5)
    with pytest.raises(TypeError, match="out_dtype"):
        mica.mica_orthogonalize([x], [x.half()], out_dtype=torch.bfloat16)


def test_polynomials_are_bounded_between_samples_too():
    """The second step's factor 32 + e - c (t^2 - u)^2 passes 32 at t^2 = u alone, by less than its curvature takes off within a
    four-thousandth of the range of t; and one that touches 32 from below is taken (and fails for want of a device)."""
    u, c = (0.1 * 2048.5 / 4096) ** 2, 1e6

    def rows(e):
        return (0.1, 0.0, 0.0, 32.0 + e - c * u * u, 2.0 * c * u, -c)

    assert orthogonalize(ns=iteration(rows(7e-7), steps=2)) == HYPER
    assert orthogonalize(ns=iteration(rows(-7e-7), steps=2)) not in (OK, HYPER)
    # t (a + b t^2 + c t^4) at its own peak, where neither end nor the factor's peak is: 1.5 t - 0.5 t^3 ... scaled to pass sqrt(32)
    top = 32.0 ** 0.5
    for scale, want in ((1.0 + 1e-9, True), (1.0 - 1e-9, False)):
        a = top * scale * 1.5 * 3.0 ** 0.5  # a t (1 - t^2) peaks at t = 3^-1/2 with a 2 / (3 3^1/2) a
        got = orthogonalize(ns=iteration((a, -a, 0.0), steps=1))
        assert (got == HYPER) == want
    # a step after one that leaves nothing takes whatever is finite
    assert orthogonalize(ns=iteration((0.0, 0.0, 0.0, 1.0, -0.5, 0.0), steps=2)) not in (OK, HYPER)
    # what float32 does not hold is refused, also where it would be multiplied by 0
    assert orthogonalize(ns=iteration((0.0, 0.0, 0.0, 1.0, 1e39, 0.0), steps=2)) == HYPER


def test_polynomials_at_their_limits():
    """Random polynomials scaled to where they reach the limits, by 20,001 samples (off by less than 1e-5 of the peak)."""
    r = random.Random(5)
    for _ in range(60):
        a, b, c = (r.uniform(-1, 1) * 4.0 ** r.uniform(-1, 2) for _ in range(3))
        t = [i / 20000 for i in range(20001)]
        q = [abs(a + x * x * (b + x * x * c)) for x in t]
        s = min(32.0 / max(q), 32.0 ** 0.5 / max(x * y for x, y in zip(t, q)))
        for e, refused in ((1e-4, True), (-1e-4, False)):
            got = orthogonalize(ns=iteration([v * s * (1 + e) for v in (a, b, c)], steps=1))
            assert (got == HYPER) == refused, (a, b, c, e)


def test_small_lists_take_small_workspaces():
    """Room for parts of sums only where the list has sums that are split."""
    M = muon._muon()

    def size(*shapes):
        return M.mica_newton_schulz_workspace(*sizes(*shapes), 0)

    assert size((1, 1)) < 1 << 16 and size((64, 64)) < 1 << 18
    exact = 4 * 384 * 1536 + 4 * 384 * 384
    assert exact <= size((384, 1536)) < exact + (1 << 14)
    part = 256 * 256 * 4
    assert 2 * part < size((16, 1600)) < 24 << 20  # a sum of 75 stages in pairs
