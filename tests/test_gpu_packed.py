"""8-bit activation checkpoints against their definition in float64: the format, the activation functions' values and
backward passes, and the weight gradient, over types, odd sizes, strides and extreme values.

Tolerances. The format is exact: codes, steps and values are compared for equality. The activation functions are computed in
float32 (some 2^-22 of their terms' sizes) and rounded once. The weight gradient sums exact products in float32: with a
chunk of at most 512 tokens summed by the tensor cores, 16 at a time (which may truncate each addition: 2^-23 of the
running size), and the chunks (here at most 9) added to nearest, |error| <= 2^-23 * (32 + 64) * sum |x dy| for any order,
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
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make(rows, cols, dtype, seed=0, ld=None, offset=0, spread=4.0):
    """A matrix whose blocks have sizes from 2^-spread to 2^spread."""
    g = gen(seed)
    ld = cols if ld is None else ld
    n = offset + max(rows, 1) * max(ld, cols)
    flat = torch.randn(n, generator=g, device="cuda")
    flat *= torch.exp2(spread * (2 * torch.rand((n + 31) // 32, generator=g, device="cuda") - 1)).repeat_interleave(32)[:n]
    return flat.to(dtype)[offset:].as_strided((rows, cols), (ld, 1))


def format_of(x):
    """(codes, e + 127, values) of the definition, in float64."""
    rows, cols = x.shape
    half = x.dtype == torch.float16
    xp = torch.nn.functional.pad(x.double(), (0, -cols % 32)).reshape(rows, -1, 32)
    most = xp.abs().amax(2)
    e = torch.full(most.shape, -24.0 if half else -126.0, device=x.device, dtype=torch.float64)
    for k in range(-126, 123):  # the smallest e with most / 2^e < 127.5
        e = torch.where((most >= 127.5 * 2.0 ** (k - 1)) & (k > e), float(k), e)
    bad = ~torch.isfinite(most)
    step = torch.exp2(e)[..., None]
    q = torch.round(xp / step)
    top = torch.floor(torch.finfo(x.dtype).max / step)  # a value is finite in its source's type
    q = torch.minimum(torch.maximum(q, -top), top)
    q = torch.where(bad[..., None], 0.0, q)
    v = torch.where(bad[..., None], math.nan, q * step)
    return (q.reshape(rows, -1), torch.where(bad, 255.0, e + 127.0), v.reshape(rows, -1)[:, :cols])


SIZES = [(1, 1), (1, 32), (3, 31), (5, 33), (2, 64), (7, 100), (13, 1601), (64, 768), (300, 96), (2, 6400), (1, 70001)]


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_format(rows, cols, dtype):
    x = make(rows, cols, dtype, seed=rows + cols, spread=12.0 if dtype == torch.float16 else 40.0)
    p = mica.mica_act_pack(x)
    codes, steps, values = format_of(x)
    blocks = (cols + 31) // 32
    assert torch.equal(p.codes.double(), codes) and torch.equal(p.steps[:, :blocks].double(), steps)
    y = mica.mica_act_unpack(p)
    assert y.dtype == dtype and torch.equal(y.double(), values)
    top = torch.nn.functional.pad(x.double(), (0, -cols % 32)).reshape(rows, -1, 32).abs().amax(2)
    assert ((y.double() - x.double()).abs() <= (top / 127).repeat_interleave(32, 1)[:, :cols] + TINY[dtype]).all()
    # a second pass over the values changes nothing
    again = mica.mica_act_unpack(mica.mica_act_pack(y))
    assert torch.equal(again, y)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_format_extremes(dtype):
    info = torch.finfo(dtype)
    rows = [[0.0] * 32, [info.max] * 32, [-info.max] + [0.0] * 31, [info.tiny] * 32, [info.smallest_normal * 127] * 32,
            [127.0] * 32, [127.49] * 32, [127.5] * 32, [127.25, 0.5, 1.5, 2.5, -0.5, -1.5] + [0.0] * 26,
            [math.inf] + [1.0] * 31, [1.0] * 31 + [math.nan], [-math.inf] * 32, [1.9921875] * 32, [1.984375] * 32,
            [65504.0] * 32, [65024.0] * 32, [2.0 ** -24] * 32, [2.0 ** -149] * 32, [2.0 ** -130, 2.0 ** -126] * 16]
    x = torch.tensor(rows, device="cuda", dtype=torch.float64).to(dtype)
    p = mica.mica_act_pack(x)
    codes, steps, values = format_of(x)
    assert torch.equal(p.codes.double(), codes) and torch.equal(p.steps[:, :1].double(), steps)
    y = mica.mica_act_unpack(p).double()
    assert torch.equal(y.isnan(), values.isnan()) and torch.equal(y.nan_to_num(0), values.nan_to_num(0))


def act64(x, act):
    f = torch.nn.functional
    return {"gelu_tanh": lambda: f.gelu(x, approximate="tanh"), "gelu": lambda: f.gelu(x), "silu": lambda: f.silu(x),
            "relu": lambda: f.relu(x)}[act]()


def close(a, b, tol):
    a = a.double()
    bad = ~((a - b).abs() <= tol) & ~(a.isnan() & b.isnan()) & ~(a == b)
    assert not bad.any(), (int(bad.sum()), a[bad][:4], b[bad][:4])


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("act", ["gelu_tanh", "gelu", "silu", "relu"])
@pytest.mark.parametrize("rows,cols,gated", [(1, 1, False), (5, 33, False), (40, 1601, False), (16, 768, False),
                                             (3, 64, True), (17, 1344, True), (200, 128, True)])
def test_act_and_grad(rows, cols, gated, act, dtype):
    x = make(rows, cols, dtype, seed=rows * cols, spread=3.0)
    p, y = mica.mica_act_pack(x, act, gated=gated)
    assert torch.equal(p.codes, mica.mica_act_pack(x).codes)
    F = cols // 2 if gated else cols
    xd = x.double()
    want = act64(xd[:, :F], act) * (xd[:, F:] if gated else 1.0)
    size = xd[:, :F].abs() * (xd[:, F:].abs() if gated else 1.0)
    close(y, want, 32 * U * size + ROUND[dtype] * want.abs() + TINY[dtype])
    dy = make(rows, F, dtype, seed=3, spread=2.0)
    v = mica.mica_act_unpack(p).double().requires_grad_()
    out = act64(v[:, :F], act) * (v[:, F:] if gated else 1.0)
    want, = torch.autograd.grad(out, v, dy.double())
    dx = mica.mica_act_grad(p, dy, act, gated=gated)
    v = v.detach()
    g = dy.double().abs()
    size = g * (1 + v[:, :F].abs()) * (v[:, F:].abs() if gated else 1.0)
    if gated:
        size = torch.cat([size, g * v[:, :F].abs()], 1)
    close(dx, want, 64 * U * size + ROUND[dtype] * want.abs() + TINY[dtype])
    assert dx.dtype == dtype
    if not gated:
        own = dy.clone()
        assert mica.mica_act_grad(p, own, act, out=own).data_ptr() == own.data_ptr() and torch.equal(own, dx)
    for other in DTYPES:  # dy of another type than the checkpoint's source
        dx2 = mica.mica_act_grad(p, dy.to(other), act, gated=gated)
        assert dx2.dtype == other


@pytest.mark.parametrize("act", ["gelu_tanh", "gelu", "silu", "relu"])
def test_act_extremes(act):
    """Far tails and non-finite blocks: no NaN from an overflow on the way."""
    x = torch.tensor([[-3e38, -1e30, -1e19, -1e10, -200.0, -90.0, -20.0, 0.0, 20.0, 90.0, 200.0, 1e10, 1e19, 1e30, 3e38]],
                     device="cuda")
    for i in range(x.shape[1]):
        one = x[:, i:i + 1]
        p, y = mica.mica_act_pack(one, act)
        v = mica.mica_act_unpack(p)
        assert y.isfinite().all() and abs(y.item() - max(one.item(), 0)) <= 1e-6 * abs(one.item()) + 1e-6
        dx = mica.mica_act_grad(p, torch.ones_like(one), act)
        want = 0.5 if v.item() == 0 and act != "relu" else float(v.item() > 0)
        assert abs(dx.item() - want) < 1e-5, (one.item(), dx.item())
    bad = torch.tensor([[1.0, math.inf]], device="cuda")
    p, y = mica.mica_act_pack(bad, act)
    assert mica.mica_act_unpack(p).isnan().all() and y[0, 0].isfinite()
    assert mica.mica_act_grad(p, torch.ones_like(bad), act).isnan().all()


def test_grad_by_differences():
    x = make(4, 64, torch.float32, seed=2, spread=1.0)
    for act in ("gelu_tanh", "gelu", "silu"):
        p = mica.mica_act_pack(x)
        v = mica.mica_act_unpack(p).double()
        h = 1e-5
        num = (act64(v + h, act) - act64(v - h, act)) / (2 * h)
        got = mica.mica_act_grad(p, torch.ones_like(x), act)
        close(got, num, 1e-6 * (1 + v.abs()))


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_float32_slopes_of_large_inputs(act):
    """From x = 3 on the slope is h, off by a rounding of 1 + e, two of the reciprocal and one of the sum, plus a term that
    has 1 - h in it: 0.013 for GELU and 0.15 for SiLU at x = 3, less beyond, off by at most 20 u of itself."""
    x = torch.linspace(3.0, 12.0, 32 * 40, device="cuda").reshape(40, 32)
    p = mica.mica_act_pack(x)
    v = mica.mica_act_unpack(p).double().requires_grad_()
    want, = torch.autograd.grad(act64(v, act).sum(), v)
    close(mica.mica_act_grad(p, torch.ones_like(x), act), want, 5 * U + {"gelu_tanh": 0.013, "silu": 0.15}[act] * 20 * U)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("cols,ld,offset", [(100, 100, 1), (100, 128, 0), (96, 97, 3), (1601, 1608, 8), (64, 0, 0)])
def test_strides(cols, ld, offset, dtype):
    rows = 9
    x = make(rows, cols, dtype, seed=cols + ld, ld=ld, offset=offset)
    same = x.clone()
    p, y = mica.mica_act_pack(x, "silu")
    q, want = mica.mica_act_pack(same, "silu")
    blocks = (cols + 31) // 32
    assert torch.equal(p.codes, q.codes) and torch.equal(p.steps[:, :blocks], q.steps[:, :blocks])
    assert torch.equal(y, want)
    base = torch.full((rows * (cols + 7) + 16,), 5.0, dtype=dtype, device="cuda")
    dy = make(rows, cols, dtype, seed=1, ld=cols + 5, offset=1)
    for first, stride in ((0, cols), (1, cols + 3), (8, cols + 7)):
        for fill in (lambda o: mica.mica_act_unpack(p, out=o), lambda o: mica.mica_act_grad(p, dy, "silu", out=o),
                     lambda o: mica.mica_act_pack(x, "silu", out=o)):
            base.fill_(5.0)
            out = base[first:].as_strided((rows, cols), (stride, 1))
            fill(out)
            plain = torch.empty((rows, cols), dtype=dtype, device="cuda")
            fill(plain)
            assert torch.equal(out, plain)
            out.fill_(5.0)
            assert (base == 5.0).all()
    # a checkpoint inside larger buffers, whose other cells stay as they are
    codes = torch.full((rows, 2048), 99, dtype=torch.int8, device="cuda")
    steps = torch.full((rows, 72), 9, dtype=torch.uint8, device="cuda")
    inside = mica.PackedActivation(codes[:, 32:32 + blocks * 32], steps[:, 4:4 + blocks], cols, dtype)
    mica.mica_act_pack(x, packed=inside)
    assert torch.equal(inside.codes, p.codes) and torch.equal(inside.steps[:, :blocks], p.steps[:, :blocks])
    assert torch.equal(mica.mica_act_unpack(inside), mica.mica_act_unpack(p))
    inside.codes.fill_(99)
    inside.steps.fill_(9)
    assert (codes == 99).all() and (steps == 9).all()


# ----------------------------------------------------------------------------------------------------------------------
# weight gradient
# ----------------------------------------------------------------------------------------------------------------------

def wgrad_check(p, dy, got, add=None):
    x, g = mica.mica_act_unpack(p).double(), dy.double()
    want, size = x.t() @ g, x.abs().t() @ g.abs()
    tol = 2 * U * 96 * size
    if add is not None:
        want = want + add.double()
        tol = tol + 2 * U * (want.abs() + size)
    close(got, want, tol + ROUND[got.dtype] * (want.abs() + tol) + TINY[got.dtype])


WG = [(0, 40, 40), (1, 1, 1), (1, 128, 256), (3, 33, 7), (15, 64, 64), (17, 100, 130), (64, 128, 256), (65, 129, 257),
      (509, 768, 96), (300, 1601, 333), (1000, 160, 1000), (4099, 96, 72), (128, 257, 2047), (2500, 384, 520)]


@pytest.mark.parametrize("tokens,features,n", WG)
@pytest.mark.parametrize("xt,gt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                   (torch.float32, torch.bfloat16), (torch.float16, torch.bfloat16)], ids=str)
def test_wgrad(tokens, features, n, xt, gt):
    x = make(tokens, features, xt, seed=tokens + features, spread=2.0)
    dy = make(tokens, n, gt, seed=n, spread=2.0)
    p = mica.mica_act_pack(x)
    dw = mica.mica_packed_wgrad(p, dy)
    assert dw.dtype == torch.float32 and dw.shape == (features, n)
    wgrad_check(p, dy, dw)
    for out in (torch.float16, torch.bfloat16):
        wgrad_check(p, dy, mica.mica_packed_wgrad(p, dy, out_dtype=out))
    for ot in DTYPES:
        add = make(features, n, ot, seed=5, spread=2.0)
        got = mica.mica_packed_wgrad(p, dy, add=add)
        wgrad_check(p, dy, got, add)
        own = add.clone()
        assert mica.mica_packed_wgrad(p, dy, add=own, out=own).data_ptr() == own.data_ptr()
        assert torch.equal(own, got)
    assert torch.equal(dw, mica.mica_packed_wgrad(p, dy))


@pytest.mark.parametrize("tokens,features,n", [(200, 2300, 2600), (1100, 2300, 4700), (1030, 5000, 2100)])
def test_wgrad_many_tiles(tokens, features, n):
    """More tiles than pairs of SMs: a pair takes tile after tile, whole ones and, of 1,024 tokens and more, parts of split
    ones, its rings going on from one to the next. The same bits each time, and added to a gradient in place."""
    x = make(tokens, features, torch.bfloat16, seed=tokens, spread=2.0)
    dy = make(tokens, n, torch.bfloat16, seed=n, spread=2.0)
    p = mica.mica_act_pack(x)
    dw = mica.mica_packed_wgrad(p, dy)
    wgrad_check(p, dy, dw)
    for _ in range(5):
        assert torch.equal(dw, mica.mica_packed_wgrad(p, dy))
    add = make(features, n, torch.float32, seed=5, spread=2.0)
    got = mica.mica_packed_wgrad(p, dy, add=add)
    wgrad_check(p, dy, got, add)
    assert torch.equal(got, mica.mica_packed_wgrad(p, dy, add=add, out=add))
    mica.mica_sync()


@pytest.mark.parametrize("n,ld,offset,ld_dw,off_dw", [(64, 64, 1, 64, 0), (64, 65, 0, 67, 1), (100, 104, 4, 100, 2),
                                                      (257, 257, 0, 260, 0), (256, 256, 8, 256, 4), (40, 0, 0, 41, 3)])
@pytest.mark.parametrize("ot", DTYPES, ids=str)
def test_wgrad_strides(n, ld, offset, ld_dw, off_dw, ot):
    tokens, features = 77, 200
    x = make(tokens, features, torch.bfloat16, seed=4, spread=1.0)
    p = mica.mica_act_pack(x)
    dy = make(tokens, n, torch.bfloat16, seed=n, ld=ld, offset=offset, spread=1.0)
    base = torch.full((features * (n + 8) + 16,), 5.0, dtype=ot, device="cuda")
    out = base[off_dw:].as_strided((features, n), (ld_dw, 1))
    wgrad_check(p, dy, mica.mica_packed_wgrad(p, dy, out=out))
    add = make(features, n, ot, seed=8, ld=n + 3, offset=1)
    wgrad_check(p, dy, mica.mica_packed_wgrad(p, dy, add=add, out=out), add)
    out.fill_(5.0)
    assert (base == 5.0).all()


def test_wgrad_nonfinite_and_extremes():
    x = make(100, 128, torch.bfloat16, seed=1)
    dy = make(100, 64, torch.bfloat16, seed=2)
    x[7, 40] = math.inf  # the token's block of 32 features stands for NaNs
    p = mica.mica_act_pack(x)
    dw = mica.mica_packed_wgrad(p, dy)
    assert dw[32:64].isnan().all() and dw[:32].isfinite().all() and dw[64:].isfinite().all()
    x[7, 40] = 1.0
    dy[3, 5] = math.nan
    dw = mica.mica_packed_wgrad(mica.mica_act_pack(x), dy)
    assert dw[:, 5].isnan().all() and dw[:, :5].isfinite().all() and dw[:, 6:].isfinite().all()
    for dtype, value in ((torch.float16, 65504.0), (torch.float16, 2.0 ** -24), (torch.bfloat16, 3e38),
                         (torch.bfloat16, 2.0 ** -120)):
        x = torch.full((2, 32), value, device="cuda", dtype=dtype)
        dy = torch.full((2, 8), 0.5, device="cuda", dtype=dtype)
        p = mica.mica_act_pack(x)
        wgrad_check(p, dy, mica.mica_packed_wgrad(p, dy))


def test_wgrad_streams_and_graph():
    x = make(700, 320, torch.bfloat16, seed=1)
    dy = make(700, 264, torch.bfloat16, seed=2)
    p = mica.mica_act_pack(x)
    want = mica.mica_packed_wgrad(p, dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mica.mica_packed_wgrad(p, dy, stream=side)
    q, y = mica.mica_act_pack(x, "silu", stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(q.codes, p.codes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = mica.mica_act_pack(x)
        held = mica.mica_packed_wgrad(q, dy)
    x.copy_(make(700, 320, torch.bfloat16, seed=9))
    dy.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, mica.mica_packed_wgrad(mica.mica_act_pack(x), dy))


def test_refusals():
    x = make(6, 96, torch.bfloat16)
    p = mica.mica_act_pack(x)
    dy = make(6, 40, torch.bfloat16)
    with pytest.raises(TypeError):
        mica.mica_act_pack(x.double())
    with pytest.raises(ValueError):
        mica.mica_act_pack(x, "tanh")
    with pytest.raises(mica.MicaError, match="COUNT"):
        mica.mica_act_pack(x, "silu", gated=True)  # 96 is not twice a multiple of 32
    with pytest.raises(mica.MicaError, match="HYPER"):
        mica.mica_act_pack(x, gated=True)
    with pytest.raises(mica.MicaError, match="HYPER"):
        mica.mica_act_grad(p, x, "none")
    with pytest.raises(mica.MicaError, match="HYPER"):
        mica.mica_act_pack(x, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        mica.mica_act_grad(p, dy, "silu")
    with pytest.raises(ValueError):
        mica.mica_packed_wgrad(p, dy[:5])
    with pytest.raises(mica.MicaError, match="DTYPE"):
        mica.mica_packed_wgrad(p, dy.float())
    with pytest.raises(mica.MicaError, match="DTYPE"):
        mica.mica_packed_wgrad(p, dy.half())
    with pytest.raises(ValueError):
        mica.mica_packed_wgrad(p, dy, add=torch.zeros(96, 41, device="cuda"))
    with pytest.raises(mica.MicaError, match="OVERLAP"):
        flat = torch.zeros(4096, dtype=torch.int8, device="cuda")
        inside = mica.PackedActivation(flat[:576].view(6, 96), p.steps, 96, torch.bfloat16)
        mica.mica_act_unpack(inside, out=flat[64:64 + 1152].view(torch.bfloat16).view(6, 96))
    with pytest.raises(TypeError):
        mica.PackedActivation(p.codes.float(), p.steps, 96, torch.bfloat16)
    with pytest.raises(ValueError):
        mica.PackedActivation(p.codes, p.steps, 97, torch.bfloat16)
    with pytest.raises(mica.MicaError, match="COUNT"):
        odd = torch.zeros(6, 100, dtype=torch.int8, device="cuda")
        mica.mica_act_unpack(mica.PackedActivation(odd, p.steps, 96, torch.bfloat16))
    with pytest.raises(mica.MicaError, match="ADDRESS"):
        flat = torch.zeros(6 * 128 + 8, dtype=torch.int8, device="cuda")[8:].view(6, 128)
        mica.mica_act_unpack(mica.PackedActivation(flat, p.steps, 96, torch.bfloat16))
    assert mica.mica_act_unpack(mica.mica_act_pack(x[:0])).shape == (0, 96)
    assert mica.mica_act_grad(mica.mica_act_pack(x[:0]), x[:0], "silu").shape == (0, 96)
