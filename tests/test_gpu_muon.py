"""The orthogonalised step against its definition in float64, over shapes, types, options and the values that end in
infinities and NaNs.

Tolerances. x, G = x x^T and B = a I + b G + c G^2 are rounded to binary16 in each step, or (where the smaller side is at most
256, and with `precise`) to a pair of binary16. What a rounding does to the end depends on the polynomial's condition at this
very input, and worst-case bounds grow by some 30 a step without saying anything. So it is measured in a model: the same
iteration in float64 with every stored matrix so rounded (`stored`), whose distance D from the definition is what these
roundings do. The kernels round the same things; their float32 sums differ and flip some of those roundings, so theirs is
another draw of the same error: twice the model's is allowed. In pairs the sums themselves count: over K terms they truncate at
most (K / 16 + 4) 2^-23 of their size, where one binary16 rounds 2^-12, and errors this small act in proportion: D of single
binary16 times (K / 16 + 4) 2^-11. Then the output's own rounding (2^-8 or 2^-11 relative per element, less in the norm).
"""
import math

import pytest
import torch

import clip_tensor_adamw_gb300 as mica

pytestmark = pytest.mark.gpu

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
U = 2.0 ** -24


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def iterate(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7, keep=lambda x: x):
    x = u.double()
    x = keep(x / (x.norm() + eps))
    wide = x.shape[0] <= x.shape[1]
    eye = torch.eye(min(x.shape), dtype=x.dtype, device=x.device)
    rows = [coefficients] * steps if not hasattr(coefficients[0], "__len__") else coefficients
    for i, (a, b, c) in enumerate(rows):
        g = keep(x @ x.t() if wide else x.t() @ x)
        p = keep(a * eye + b * g + c * (g @ g))
        x = p @ x if wide else x @ p
        if i + 1 < len(rows):
            x = keep(x)
    return x


def half(x):
    return (x * 1024.0).half().double() / 1024.0


def pair(x):
    return half(x) + half(x - half(x))


def distance(a, b):
    return float((a.double() - b).norm())


def off(u, want, precise=False, **kw):
    """How far a result may be from the definition's before its own rounding."""
    single = distance(iterate(u, keep=half, **kw), want)
    if not precise and min(u.shape) > 256:
        return 2.0 * single
    return 2.0 * distance(iterate(u, keep=pair, **kw), want) + single * (max(u.shape) / 16 + 4) * 2.0 ** -11


def check(got, u, precise=False, **kw):
    want = iterate(u, **kw)
    most = off(u, want, precise, **kw) + HALF[got.dtype] * float(want.norm()) + 1e-6
    assert distance(got, want) <= most, (tuple(u.shape), distance(got, want), most)


SHAPES = [(1, 1), (1, 57), (57, 1), (2, 3), (7, 64), (64, 7), (64, 64), (33, 129), (129, 33), (100, 333), (333, 100), (256, 256),
          (257, 300), (300, 257), (384, 1536), (777, 1201), (1201, 777), (16, 4096), (600, 600)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_one_matrix(shape, dtype):
    x = (1e-2 * torch.randn(shape, generator=gen(sum(shape)), device="cuda")).to(dtype)
    for out in (torch.float16, torch.bfloat16):
        r = mica.mica_orthogonalize([x], out_dtype=out)
        assert r.tensors[0].dtype == out
        check(r.tensors[0], x)


@pytest.mark.parametrize("shape", [(300, 257), (257, 300), (1201, 777), (777, 1201), (600, 600)], ids=str)
def test_precise(shape):
    """Pairs of binary16 for larger matrices: what is left of a tiny singular value's direction shows the difference."""
    g = gen(7)
    x = torch.randn(shape, generator=g, device="cuda")
    u, s, v = torch.linalg.svd(x, full_matrices=False)
    x = (u * torch.logspace(0, -3, len(s), device="cuda")) @ v
    r = mica.mica_orthogonalize([x], out_dtype=torch.float16, precise=True).tensors[0]
    check(r, x, precise=True)
    check(mica.mica_orthogonalize([x], out_dtype=torch.float16).tensors[0], x)


def test_singular_values_end_near_one():
    x = torch.randn(500, 900, generator=gen(1), device="cuda")
    s = torch.linalg.svdvals(mica.mica_orthogonalize([x], out_dtype=torch.float16).tensors[0].double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.25


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_a_list_is_its_matrices(dtype):
    """Each of a list's matrices comes out as it would alone, bit for bit; more shapes and matrices than a batch holds."""
    g = gen(2)
    shapes = [(40 + 8 * (i % 11), 24 + 16 * (i % 5)) for i in range(70)] + [(5, 5)] * 300 + [(0, 7), (7, 0), (300, 20)]
    x = [torch.randn(s, generator=g, device="cuda").to(dtype) for s in shapes]
    r = mica.mica_orthogonalize(x)
    assert [t.shape for t in r.tensors] == [t.shape for t in x]
    for i in list(range(0, 70, 7)) + [70, 369, 372]:
        assert torch.equal(r.tensors[i], mica.mica_orthogonalize([x[i]]).tensors[0]), i
        check(r.tensors[i], x[i])


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("gdt", [torch.float32, torch.float16], ids=str)
@pytest.mark.parametrize("adjust,precise", [("none", False), ("original", True), ("match_rms_adamw", False)])
def test_steps(adjust, precise, gdt, nesterov):
    g = gen(3)
    shapes = [(100, 333), (333, 100), (64, 64), (1, 57), (257, 300)]
    scale = 1024.0 if gdt is torch.float16 else 1.0
    w = [0.02 * torch.randn(s, generator=g, device="cuda") for s in shapes]
    m = [torch.zeros_like(t) for t in w]
    factor = torch.full((1,), 0.5 / scale, device="cuda")
    lr, mu, wd = 3e-2, 0.9, 0.1
    for step in range(3):
        grads = [(1e-2 * scale * torch.randn(s, generator=g, device="cuda")).to(gdt) for s in shapes]
        before_w, before_m, kept = [t.clone() for t in w], [t.clone() for t in m], [t.clone() for t in grads]
        zero = step == 1
        mica.mica_muon_steps(w, grads, m, lr=lr, momentum=mu, weight_decay=wd, nesterov=nesterov, adjust=adjust, factor=factor,
                             zero_grad=zero, precise=precise)
        for k, (r, c) in enumerate(shapes):
            gh = kept[k].double() * factor.double()
            want_m = before_m[k].double() + (1 - mu) * (gh - before_m[k].double())
            assert ((m[k].double() - want_m).abs() <= 8 * U * (before_m[k].abs() + gh.abs())).all()
            u = gh + mu * (want_m - gh) if nesterov else want_m
            rate = lr * (math.sqrt(max(1.0, r / c)) if adjust == "original" else
                         0.2 * math.sqrt(max(r, c)) if adjust == "match_rms_adamw" else 1.0)
            o = iterate(u)
            want = before_w[k].double() * (1 - lr * wd) - rate * o
            most = rate * off(u, o, precise) + 8 * U * float(before_w[k].double().norm() + rate * o.norm()) + 1e-6 * rate
            assert distance(w[k], want) <= most, (k, distance(w[k], want), most)
            assert not grads[k].any() if zero else torch.equal(grads[k], kept[k])
