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


def test_zeros_infinities_and_nans():
    """A zero matrix gives zeros, one with an infinity or a NaN gives NaNs; the others of the list are as they would be alone."""
    g = gen(11)
    x = [torch.randn(s, generator=g, device="cuda") for s in [(300, 400), (300, 400), (300, 400), (40, 20), (40, 20), (40, 20)]]
    x[0].zero_()
    x[3].zero_()
    x[1][17, 5] = math.inf
    x[4][3, 3] = math.nan
    r = mica.mica_orthogonalize(x).tensors
    assert not r[0].any() and not r[3].any() and r[1].isnan().all() and r[4].isnan().all()
    for i in (2, 5):
        assert torch.equal(r[i], mica.mica_orthogonalize([x[i]]).tensors[0])
        check(r[i], x[i])


@pytest.mark.parametrize("scale", [1e-25, 1e-18, 1e15, 1e34])
@pytest.mark.parametrize("shape", [(60, 90), (300, 280)], ids=str)
def test_any_scale(shape, scale):
    """Squares that float32 cannot hold: the result does not depend on the matrix's size (eps apart)."""
    x = torch.randn(shape, generator=gen(12), device="cuda") * scale
    check(mica.mica_orthogonalize([x], eps=1e-30).tensors[0], x, eps=1e-30)
    one = torch.zeros_like(x)  # a single element: the square sum is one square
    one[7, 3] = scale
    r = mica.mica_orthogonalize([one], eps=1e-30, out_dtype=torch.float16).tensors[0]
    want = 1.0
    for _ in range(5):
        a, b, c = COEFFICIENTS
        want = a * want + b * want ** 3 + c * want ** 5
    assert abs(float(r[7, 3]) - want) <= 0.01 and int((r != 0).sum()) == 1


def test_eps_counts():
    x = torch.randn(50, 70, generator=gen(13), device="cuda") * 1e-3
    for eps in (1e-7, 0.05, 1.0):
        check(mica.mica_orthogonalize([x], eps=eps).tensors[0], x, eps=eps)


def test_in_place_and_alignment():
    """Results over the inputs; matrices that begin at any element."""
    g = gen(14)
    for dtype in (torch.float16, torch.bfloat16):
        for offset in (0, 1, 3, 4):
            flat = torch.randn(offset + 130 * 77 + 300 * 8, generator=g, device="cuda").to(dtype)
            views = [flat[offset:offset + 130 * 77].view(130, 77), flat[offset + 130 * 77:offset + 130 * 77 + 2400].view(300, 8)]
            want = mica.mica_orthogonalize([v.clone() for v in views])
            tail = flat[offset + 130 * 77 + 2400:].clone()
            mica.mica_orthogonalize(views, views)
            for a, b in zip(views, want.tensors):
                assert torch.equal(a, b)
            assert torch.equal(flat[offset + 130 * 77 + 2400:], tail)
    w = torch.randn(1 + 65 * 33, generator=g, device="cuda")[1:].view(65, 33)
    grad = torch.randn(3 + 65 * 33, generator=g, device="cuda")[3:].view(65, 33)
    m = torch.randn(2 + 65 * 33, generator=g, device="cuda")[2:].view(65, 33)
    copies = [t.clone() for t in (w, grad, m)]
    mica.mica_muon_steps([w], [grad], [m], lr=0.1)
    mica.mica_muon_steps(*[[t] for t in copies], lr=0.1)
    assert torch.equal(w, copies[0]) and torch.equal(m, copies[2])


@pytest.mark.parametrize("coefficients,steps", [((1.5, -0.5, 0.0), 10), ((1.875, -1.25, 0.375), 7), ((2.0, -1.5, 0.5), 1)])
def test_other_polynomials(coefficients, steps):
    x = torch.randn(90, 300, generator=gen(15), device="cuda")
    check(mica.mica_orthogonalize([x], coefficients=coefficients, steps=steps).tensors[0], x, coefficients=coefficients, steps=steps)
    rows = [coefficients] * (steps - 1) + [(3.0, -3.2, 1.2)]
    check(mica.mica_orthogonalize([x], coefficients=rows, steps=steps).tensors[0], x, coefficients=rows)


def test_long_sides():
    g = gen(16)
    for shape in [(3, 100_003), (70_001, 5), (260, 20_000), (20_000, 260)]:
        x = torch.randn(shape, generator=g, device="cuda")
        check(mica.mica_orthogonalize([x], out_dtype=torch.float16).tensors[0], x)


def test_offsets_past_32_bits():
    """A matrix of more than 2^31 elements, one step: its last rows against the formula in float32 (whose own error, 1e-5 or
    so, counts for nothing beside binary16's 2^-11 per rounding)."""
    rows, cols = 131_072, 16_392
    assert rows * cols > 2 ** 31
    x = torch.empty(rows, cols, dtype=torch.float16, device="cuda").normal_(generator=gen(19))
    r = mica.mica_orthogonalize([x], steps=1, out_dtype=torch.float16).tensors[0]
    norm = math.sqrt(sum(float(x[a:a + 8192].float().square().sum(dtype=torch.float64)) for a in range(0, rows, 8192)))
    gram = torch.zeros(cols, cols, device="cuda")
    for a in range(0, rows, 8192):
        part = x[a:a + 8192].float() / norm
        gram += part.t() @ part
    a, b, c = COEFFICIENTS
    for at in (slice(0, 4), slice(rows - 4, rows)):
        u = x[at].float() / norm
        ug = u @ gram
        want = a * u + b * ug + c * (ug @ gram)
        assert float((r[at].float() - want).norm()) <= 4 * 2.0 ** -11 * float(want.norm())


@pytest.mark.parametrize("gdt", [torch.float32, torch.float16], ids=str)
@pytest.mark.parametrize("factor", [0.0, math.nan, math.inf, -1.0])
def test_skip_nonfinite(factor, gdt):
    """A factor that is not > 0 leaves w and m as they are, and still zeroes g when asked; without the flag it counts."""
    g = gen(17)
    shapes = [(40, 30), (300, 310)]
    w, m = ([torch.randn(s, generator=g, device="cuda") for s in shapes] for _ in range(2))
    grads = [torch.randn(s, generator=g, device="cuda").to(gdt) for s in shapes]
    f = torch.full((1,), factor, device="cuda")
    kept = [[t.clone() for t in x] for x in (w, m)]
    mica.mica_muon_steps(w, grads, m, lr=0.1, factor=f, skip_nonfinite=True, zero_grad=True)
    went = factor == math.inf  # > 0
    for a, b in zip((w, m), kept):
        for s, t in zip(a, b):
            assert torch.equal(s, t) != went
    assert not any(t.any() for t in grads)
    if factor == 0.0:
        mica.mica_muon_steps(w, grads, m, lr=0.1, factor=f)
        assert not torch.equal(w[0], kept[0][0])


def test_lists_without_elements():
    assert mica.mica_orthogonalize([]).T == 0
    e = torch.empty(0, 5, device="cuda")
    r = mica.mica_orthogonalize([e, e.t().contiguous()])
    assert [tuple(t.shape) for t in r.tensors] == [(0, 5), (5, 0)]
    mica.mica_muon_steps([], [], [], lr=0.1)
    mica.mica_muon_steps([e], [e.clone()], [e.clone()], lr=0.1)


def test_streams_graphs_and_repeats():
    g = gen(18)
    shapes = [(384, 384), (384, 1536), (16, 1600), (513, 2048)]
    x = mica.TensorList([torch.randn(s, generator=g, device="cuda") for s in shapes])
    first = mica.mica_orthogonalize(x)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    both = [mica.mica_orthogonalize(x, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for r in both:
        assert all(torch.equal(a, b) for a, b in zip(r.tensors, first.tensors))
    w, m = ([torch.randn(s, generator=g, device="cuda") for s in shapes] for _ in range(2))
    copies = [[t.clone() for t in y] for y in (w, m)]
    factor = torch.full((1,), 0.5, device="cuda")
    graph = torch.cuda.CUDAGraph()
    mica.mica_muon_steps(*[[t.clone() for t in y] for y in (w, x.tensors, m)], lr=0.01, factor=factor)  # loads the library
    with torch.cuda.graph(graph):
        mica.mica_muon_steps(w, x, m, lr=0.01, factor=factor)
    for step in range(3):
        for t in x.tensors:
            t.normal_(generator=g)
        factor.fill_(0.3 + step)
        graph.replay()
        mica.mica_muon_steps(copies[0], x, copies[1], lr=0.01, factor=factor)
        for a, b in zip((w, m), copies):
            assert all(torch.equal(s, t) for s, t in zip(a, b)), step


def test_refusals():
    x = torch.randn(64, 64, device="cuda")
    with pytest.raises(mica.MicaError, match="OVERLAP"):
        mica.mica_muon_steps([x], [x], [torch.zeros_like(x)], lr=0.1)
    with pytest.raises(mica.MicaError, match="OVERLAP"):
        mica.mica_muon_steps([x, x], [x.clone(), x.clone()], [x.clone(), x.clone()], lr=0.1)
    with pytest.raises(mica.MicaError, match="OVERLAP"):
        half = torch.randn(65, 64, device="cuda").half()
        mica.mica_orthogonalize([half[:64]], [half[1:]])
    y = torch.randn(64, 64, device="cuda").half()
    with pytest.raises(mica.MicaError, match="OVERLAP"):
        mica.mica_orthogonalize([y, y], [y, torch.empty_like(y)])
    with pytest.raises(mica.MicaError, match="ADDRESS"):
        mica.mica_orthogonalize([x.cpu()], [torch.empty(64, 64, dtype=torch.float16, device="cuda")])
    for bad in (dict(coefficients=(3.4445, 4.775, 2.0315)), dict(coefficients=(7.0, 0.0, 0.0)), dict(eps=0.0), dict(eps=2.0)):
        with pytest.raises(mica.MicaError, match="HYPER"):
            mica.mica_orthogonalize([x], **bad)
    with pytest.raises(ValueError):
        mica.mica_orthogonalize([x], steps=0, coefficients=[])
    mica.mica_orthogonalize([x, x])  # one matrix read twice is fine


@pytest.mark.parametrize("shape", [(16, 1600), (260, 20_000), (1600, 16)], ids=str)
def test_split_sums(shape):
    """A sum that is split where the list leaves pairs of CTAs idle and is not beside larger matrices: other bits perhaps, the
    same error; and the same bits whenever the list is the same."""
    g = gen(20)
    x = torch.randn(shape, generator=g, device="cuda")
    others = [torch.randn(s, generator=g, device="cuda") for s in [(1600, 1600), (1201, 777)] + [shape] * 20]
    alone = [mica.mica_orthogonalize([x], out_dtype=torch.float16).tensors[0] for _ in range(3)]
    beside = [mica.mica_orthogonalize([x] + others, out_dtype=torch.float16).tensors[0] for _ in range(3)]
    for r in (alone, beside):
        check(r[0], x)
        assert torch.equal(r[0], r[1]) and torch.equal(r[0], r[2])
    w, m = torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    mica.mica_muon_steps([w], [x], [m], lr=1.0, momentum=0.0, adjust="none")
    want = iterate(x)
    assert distance(-w, want) <= off(x, want) + 8 * U * float(want.norm()) + 1e-6
