"""What the losses from hidden states and the orthogonalised optimizer step are measured on.

Five operators of one training step of a language model, on both sides of its backward pass:

* ``linear_logps``  log-probabilities of given tokens from hidden states and an output embedding, whose product (the
                    logits) is not kept: scoring by a reference or sampling policy, evaluation; forward only.
* ``linear_grad``   their gradient, for any loss over log-probabilities: of the hidden states and of the embedding.
* ``linear_ce``     softmax cross entropy over the vocabulary with both gradients, in one call.
* ``orthogonal``    a list of matrices, each taken by Newton-Schulz products to the nearest matrix with orthogonal rows
                    (or columns), roughly: singular values end between 0.7 and 1.2.
* ``muon``          an optimizer step over a list of weight matrices: momentum, the orthogonalised update, decay.

``run`` computes them in elementary torch operations, in 32 bits and rounded once, or, with ``own`` set, through this
package's entry points. ``exact`` computes the definitions in float64, by other means (autograd, another order of the
products). Rows without a target (negative: a prompt's tokens) do not count; their gradients are zeros.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
LAYER = "1600x4800,1600x1600,1600x6400,6400x1600"  # the matrices of a GPT-2 XL layer


# ----------------------------------------------------------------------------------------------------------------------
# the cases
# ----------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one new token scored, as a serving loop does after each step (GPT-2 small's width, GPT-2's vocabulary)
        dict(name="logps_one_token", op="linear_logps", tokens=1, features=768, vocab=50257, dtype="bf16", prompt=0.0,
             temperature=0.7),
        # a micro-batch scored by the reference policy at GPT-2 XL's width; a quarter of it are prompts
        dict(name="logps_batch", op="linear_logps", tokens=8192, features=1600, vocab=50257, dtype="bf16", prompt=0.25,
             temperature=1.0),
        # the gradient of one short sampled answer's loss, loss-scaled binary16, a small vocabulary of odd size
        dict(name="grad_answer", op="linear_grad", tokens=96, features=1000, vocab=32003, dtype="f16", prompt=0.25,
             temperature=0.8, scale=1024.0),
        # the gradient of a policy's loss over a micro-batch at GPT-2 small's width
        dict(name="grad_batch", op="linear_grad", tokens=4096, features=768, vocab=50257, dtype="bf16", prompt=0.25,
             temperature=1.0, scale=1.0),
        # cross entropy of one ragged sequence, narrow odd widths whose rows are unaligned, loss-scaled binary16
        dict(name="ce_sequence", op="linear_ce", tokens=333, features=387, vocab=5003, dtype="f16", prompt=0.4,
             temperature=1.0, scale=1024.0),
        # pre-training of GPT-2 small: a micro-batch of eight sequences of 1,024 tokens, all scored
        dict(name="ce_pretrain", op="linear_ce", tokens=8192, features=768, vocab=50257, dtype="bf16", prompt=0.0,
             temperature=1.0, scale=1.0),
        # fine-tuning at GPT-2 XL's width with a large vocabulary
        dict(name="ce_large_vocab", op="linear_ce", tokens=4096, features=1600, vocab=131072, dtype="bf16",
             prompt=0.125, temperature=1.0, scale=1.0),
        # one matrix of the smallest workload, where latency counts
        dict(name="orthogonal_one", op="orthogonal", shapes="384x1536", dtype="bf16", out="bf16"),
        # small matrices of odd shapes (heads, adapters, a router), binary16
        dict(name="orthogonal_ragged", op="orthogonal", shapes="100x333,64x64,1x57,2048x513,777x1201,16x1600",
             dtype="f16", out="f16"),
        # a layer of GPT-2 XL from float32 momentum
        dict(name="orthogonal_layer", op="orthogonal", shapes=LAYER, dtype="f32", out="bf16"),
        # the two matrices of the smallest workload
        dict(name="muon_tiny", op="muon", shapes="384x384,384x1536", dtype="f32", nesterov=True, adjust="original",
             lr=2e-3, scale=1.0),
        # four layers of GPT-2 XL
        dict(name="muon_layers", op="muon", shapes=",".join([LAYER] * 4), dtype="f32", nesterov=True,
             adjust="match_rms_adamw", lr=3e-4, scale=1.0),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["linear_logps", "linear_grad", "linear_ce", "orthogonal", "muon"])
    if op in ("linear_logps", "linear_grad", "linear_ce"):
        dtype = rng.choice(["bf16", "bf16", "f16"])
        features, vocab = _log_int(rng, 33, 2048), _log_int(rng, 500, 131072)
        if rng.random() < 0.7:
            features = (features + 7) // 8 * 8
        # the largest listed case's products, scored rows only
        most = {"linear_logps": 6144 * 1600 * 50257, "linear_grad": 4096 * 3 // 4 * 768 * 50257,
                "linear_ce": 3584 * 1600 * 131072}[op]
        tokens = _log_int(rng, 1, max(1, min(8192, most // (features * vocab))))
        return dict(op=op, tokens=tokens, features=features, vocab=vocab, dtype=dtype,
                    prompt=rng.choice([0.0, 0.25, 0.5]), temperature=rng.choice([1.0, 1.0, 0.8]),
                    scale=1024.0 if dtype == "f16" else 1.0)
    count = _log_int(rng, 1, 12)
    shapes, left = [], 8 * 3 * 1600 * 1600 * 6400  # under the largest listed case's products
    for _ in range(count):
        r, c = _log_int(rng, 8, 4096), _log_int(rng, 8, 4096)
        if rng.random() < 0.4:
            r, c = (r + 31) // 32 * 32, (c + 31) // 32 * 32
        if _products(r, c) <= left:
            left -= _products(r, c)
            shapes.append("%dx%d" % (r, c))
    shapes = ",".join(shapes or ["64x129"])
    dtype = rng.choice(["f32", "f32", "f16"])
    if op == "orthogonal":
        return dict(op=op, shapes=shapes, dtype=rng.choice(["f32", "f16", "bf16"]), out=rng.choice(["bf16", "f16"]))
    adjust = rng.choice(["original", "match_rms_adamw"])
    return dict(op=op, shapes=shapes, dtype=dtype, nesterov=rng.random() < 0.7, adjust=adjust,
                lr=2e-3 if adjust == "original" else 3e-4, scale=65536.0 if dtype == "f16" else 1.0)


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _active(case):
    """Which rows count: runs of at most 512 tokens, each beginning with its prompt, whose tokens are not scored."""
    on = []
    for a in range(0, case["tokens"], 512):
        n = min(512, case["tokens"] - a)
        p = int(n * case["prompt"])
        on += [False] * p + [True] * (n - p)
    return on


def _shapes(case):
    return [tuple(int(v) for v in s.split("x")) for s in case["shapes"].split(",")]


def _products(r, c):
    """Multiplications of one Newton-Schulz step: the Gram matrix and its square (both symmetric), and the product."""
    s, n = min(r, c), max(r, c)
    return s * s * n // 2 + s * s * s // 2 + s * s * n


def _spread(g, r, c):
    """A gradient's shape of spectrum: most of its energy in a few directions over a broad rest."""
    x = torch.randn(r, c, generator=g, device="cuda")
    x *= (0.5 + torch.rand(1, c, generator=g, device="cuda")) * (0.5 + torch.rand(r, 1, generator=g, device="cuda"))
    k = max(1, min(8, r // 4, c // 4))
    top = torch.randn(r, k, generator=g, device="cuda") @ torch.randn(k, c, generator=g, device="cuda")
    return x + top * (x.norm() / top.norm().clamp(min=1e-6)) * 1.5


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] in ("linear_logps", "linear_grad", "linear_ce"):
        dt = DTYPES[case["dtype"]]
        t, d, v = case["tokens"], case["features"], case["vocab"]
        on = torch.tensor(_active(case), device="cuda")
        w = (torch.randn(v, d, generator=g, device="cuda") * (1.2 / math.sqrt(d))).to(dt)
        h = torch.randn(t, d, generator=g, device="cuda") * (0.5 + torch.rand(1, d, generator=g, device="cuda"))
        targets = torch.randint(0, v, (t,), generator=g, device="cuda")
        # the scored token is among the likely ones
        row = w[targets].float()
        h += row * (8.0 * torch.rand(t, 1, generator=g, device="cuda") / row.square().sum(1, keepdim=True))
        h = h.to(dt)
        s.update(h=h, w=w, targets=torch.where(on, targets, torch.full_like(targets, -100)))
        if case["op"] == "linear_grad":
            lse = [torch.logsumexp(h[a:a + 2048].float() @ w.float().t() / case["temperature"], 1)
                   for a in range(0, t, 2048)]
            s["lse"] = torch.where(on, torch.cat(lse), torch.zeros(t, device="cuda"))
            s["dlogps"] = torch.randn(t, generator=g, device="cuda") * (case["scale"] / max(1, int(on.sum())))
        return s
    shapes, dt = _shapes(case), DTYPES[case["dtype"]]
    if case["op"] == "orthogonal":
        s["x"] = [(1e-2 * _spread(g, r, c)).to(dt) for r, c in shapes]
        s["out"] = [torch.empty(r, c, dtype=DTYPES[case["out"]], device="cuda") for r, c in shapes]
        names = ("x", "out")
    else:
        s["w"] = [0.02 * torch.randn(r, c, generator=g, device="cuda") for r, c in shapes]
        s["g"] = [(1e-3 * case["scale"] * _spread(g, r, c)).to(dt) for r, c in shapes]
        s["m"] = [1e-3 * _spread(g, r, c) for r, c in shapes]
        # what ClipGradNorms leaves on the device: the clip, with the loss scale taken out
        s["factor"] = torch.full((1,), 0.37 / case["scale"], device="cuda")
        names = ("w", "g", "m")
    if own:  # a program builds its lists once
        import clip_tensor_adamw_gb300 as mica
        s["lists"] = [mica.TensorList(s[n]) for n in names]
    return s


# ----------------------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------------------

def _logits(s):
    return (s["h"].float() @ s["w"].float().t()) * (1.0 / s["case"]["temperature"])


def _gather(x, targets):
    return x.gather(1, targets.clamp(min=0)[:, None])[:, 0]


def _grads(s, p, coef):
    """The gradients, coef * (1[target] - p) / temperature being that of the logits; p is overwritten."""
    on = s["targets"] >= 0
    coef = torch.where(on, coef, torch.zeros_like(coef)) * (1.0 / s["case"]["temperature"])
    p[torch.arange(p.shape[0], device=p.device), s["targets"].clamp(min=0)] -= 1.0
    p *= -coef[:, None]
    return (p @ s["w"].float()).to(s["h"].dtype), (p.t() @ s["h"].float()).to(s["w"].dtype)


def _orthogonal(x):
    x = x.float()
    x = x / (torch.sqrt((x * x).sum()) + EPS)
    wide = x.shape[0] <= x.shape[1]
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = x @ x.t() if wide else x.t() @ x
        poly = b * gram + c * (gram @ gram)
        x = a * x + (poly @ x if wide else x @ poly)
    return x


def _rate(case, r, c):
    return case["lr"] * (math.sqrt(max(1.0, r / c)) if case["adjust"] == "original" else 0.2 * math.sqrt(max(r, c)))


MOMENTUM, DECAY = 0.95, 0.1


def _plain(s):
    c = s["case"]
    if c["op"] == "linear_logps":
        z = _logits(s)
        top = z.amax(1)
        lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
        zero = torch.zeros((), device=z.device)
        on = s["targets"] >= 0
        return dict(logps=torch.where(on, _gather(z, s["targets"]) - lse, zero), lse=torch.where(on, lse, zero))
    if c["op"] == "linear_grad":
        dh, dw = _grads(s, torch.exp(_logits(s) - s["lse"][:, None]), s["dlogps"])
        return dict(dh=dh, dw=dw)
    if c["op"] == "linear_ce":
        z = _logits(s)
        z -= z.amax(1, keepdim=True)
        at = _gather(z, s["targets"])
        p = z.exp_()
        total = p.sum(1)
        on = s["targets"] >= 0
        lp = torch.where(on, at - torch.log(total), torch.zeros_like(at))
        n = on.sum().clamp(min=1).float()
        p /= total[:, None]
        dh, dw = _grads(s, p, (-c["scale"] / n).expand(lp.shape))
        return dict(loss=(-lp.sum() / n)[None], logps=lp, dh=dh, dw=dw)
    if c["op"] == "orthogonal":
        for x, out in zip(s["x"], s["out"]):
            out.copy_(_orthogonal(x))
        return s["out"]
    for w, g, m in zip(s["w"], s["g"], s["m"]):
        gh = g.float() * s["factor"]
        m += (1.0 - MOMENTUM) * (gh - m)
        u = gh + MOMENTUM * (m - gh) if c["nesterov"] else m
        rate = _rate(c, *w.shape)
        w *= 1.0 - c["lr"] * DECAY
        w -= rate * _orthogonal(u)
    return dict(w=s["w"], m=s["m"])


def _own(s):
    import clip_tensor_adamw_gb300 as mica
    c = s["case"]
    if c["op"] == "linear_logps":
        logps, lse = mica.mica_linear_logps(s["h"], s["w"], s["targets"], temperature=c["temperature"], lse=True)
        return dict(logps=logps, lse=lse)
    if c["op"] == "linear_grad":
        dh, dw = mica.mica_linear_logps_grad(s["h"], s["w"], s["targets"], s["lse"], s["dlogps"],
                                             temperature=c["temperature"])
        return dict(dh=dh, dw=dw)
    if c["op"] == "linear_ce":
        r = mica.mica_linear_cross_entropy(s["h"], s["w"], s["targets"], temperature=c["temperature"],
                                           grad_scale=c["scale"])
        return dict(loss=r.loss, logps=r.logps, dh=r.dh, dw=r.dw)
    if c["op"] == "orthogonal":
        mica.mica_orthogonalize(*s["lists"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        return s["out"]
    mica.mica_muon_steps(*s["lists"], lr=c["lr"], momentum=MOMENTUM, weight_decay=DECAY, nesterov=c["nesterov"],
                         adjust=c["adjust"], factor=s["factor"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
    return dict(w=s["w"], m=s["m"])


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------------------------------------------

def work(case):
    if case["op"] in ("linear_logps", "linear_grad", "linear_ce"):
        t, d, v = case["tokens"], case["features"], case["vocab"]
        rows, e = sum(_active(case)), BYTES[case["dtype"]]
        read = (rows + v) * d * e + t * 8
        if case["op"] == "linear_logps":
            return dict(bytes=read + t * 8, flops=2 * rows * d * v)
        # the gradient takes the logits again and two more products of their size
        return dict(bytes=read + (t + v) * d * e + t * (8 if case["op"] == "linear_grad" else 4),
                    flops=6 * rows * d * v)
    n = sum(r * c for r, c in _shapes(case))
    flops = 2 * STEPS * sum(_products(r, c) for r, c in _shapes(case))
    if case["op"] == "orthogonal":
        return dict(bytes=n * (BYTES[case["dtype"]] + BYTES[case["out"]]), flops=flops)
    return dict(bytes=n * (BYTES[case["dtype"]] + 16), flops=flops)


# ----------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------------------------------------

def _exact_orthogonal(x):
    x = x.double()
    x = x / (torch.linalg.matrix_norm(x) + EPS)
    if x.shape[0] > x.shape[1]:
        return _exact_orthogonal_rows(x.t().contiguous()).t()
    return _exact_orthogonal_rows(x)


def _exact_orthogonal_rows(x):
    """x (a I + G (b I + c G)) with the Gram matrix on the left, by Horner's rule."""
    a, b, c = COEFFICIENTS
    eye = torch.eye(x.shape[0], dtype=x.dtype, device=x.device)
    for _ in range(STEPS):
        gram = torch.mm(x, x.t())
        x = torch.mm(torch.addmm(eye, gram, eye.mul(b).add_(gram, alpha=c), beta=a), x)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonal":
        return [_exact_orthogonal(x) for x in s["x"]]
    if case["op"] == "muon":
        f = s["factor"].double()
        ws, ms = [], []
        for w, g, m in zip(s["w"], s["g"], s["m"]):
            gh = g.double() * f
            m = torch.lerp(m.double(), gh, 1.0 - MOMENTUM)
            u = torch.lerp(gh, m, MOMENTUM) if case["nesterov"] else m
            ws.append(w.double() * (1.0 - case["lr"] * DECAY) - _rate(case, *w.shape) * _exact_orthogonal(u))
            ms.append(m)
        return dict(w=ws, m=ms)
    on = s["targets"] >= 0
    y = s["targets"].clamp(min=0)
    grads = case["op"] != "linear_logps"
    h, w = (s[k].double().requires_grad_(grads) for k in ("h", "w"))
    with torch.enable_grad():
        z = torch.nn.functional.linear(h, w).div(case["temperature"])
        lse = torch.logsumexp(z, 1)
        lp = torch.where(on, z.gather(1, y[:, None]).squeeze(1) - lse, 0.0)
        if case["op"] == "linear_logps":
            return dict(logps=lp, lse=torch.where(on, lse, 0.0))
        if case["op"] == "linear_grad":
            dh, dw = torch.autograd.grad((lp * s["dlogps"].double()).sum(), (h, w))
            return dict(dh=dh, dw=dw)
        loss = -lp.sum() / on.sum().clamp(min=1)
        dh, dw = torch.autograd.grad(loss * case["scale"], (h, w))
    return dict(loss=loss.detach()[None], logps=lp.detach(), dh=dh, dw=dw)
