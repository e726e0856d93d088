"""What the loss operators and the 8-bit activation checkpoints are measured on.

Six operators of one fine-tuning step around the optimizer step of this package:

* ``logps``       log-probabilities (and entropies) of given tokens from a matrix of logits: the reference policy's and
                  the sampling policy's scoring pass, forward only.
* ``preference``  a preference loss over pairs of packed sequences, from the logits, with the gradient of the logits.
* ``policy``      a clipped policy loss with a KL term, from the logits, with the gradient of the logits.
* ``save``        an activation's checkpoint in 8 bits (and the activation function's output, for the forward pass),
                  and the values that it stands for.
* ``act_grad``    the backward pass of an activation function from its 8-bit checkpoint.
* ``wgrad``       the weight gradient of a linear layer from its input's 8-bit checkpoint.

``run`` computes them in elementary torch operations, in 32 bits and rounded once, or, with ``own`` set, through this
package's entry points. ``exact`` computes the definitions in float64, by other means (autograd, logsumexp).

The checkpoint's format: a row's columns in blocks of 32; a block holds one exponent e and 32 signed codes q, and
stands for q * 2^e. e is the smallest integer with max|x| / 2^e < 127.5 (at least -126, or -24 for binary16 sources,
whose values are all multiples of 2^-24), q = x / 2^e to the nearest integer, ties to even (in binary16 at most
65504 / 2^e, so that every value is a binary16 one). The exponent is stored as e + 127; 255 marks a block with an
infinity or a NaN in it, which stands for NaNs.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.05
BETA = 0.1


# ----------------------------------------------------------------------------------------------------------------------
# the cases
# ----------------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # one new token scored from one row of logits, as a serving loop does after each step (the vocabulary of the
        # GPT-2 workloads, whose odd size leaves rows unaligned)
        dict(name="logps_one_token", op="logps", tokens=1, vocab=50257, ld=50257, dtype="bf16", prompt=0.0, banned=0,
             temperature=0.7),
        # a micro-batch scored by the reference policy: whole rows, packed without padding
        dict(name="logps_batch", op="logps", tokens=8192, vocab=50257, ld=50257, dtype="bf16", prompt=0.25, banned=0,
             temperature=1.0),
        # two short pairs in the loss-scaled binary16 recipe, with a small vocabulary, one of whose sequences is empty
        dict(name="preference_two_pairs", op="preference", pairs=2, length=48, empty=1, vocab=32003, ld=32003,
             dtype="f16", prompt=0.4, banned=3, kind="sigmoid", smoothing=0.1, length_norm=False, grad_scale=1024.0),
        # a micro-batch of sixteen pairs of ragged lengths; logits with their rows padded to a multiple of 64 columns
        dict(name="preference_batch", op="preference", pairs=16, length=256, empty=0, vocab=50257, ld=50304,
             dtype="bf16", prompt=0.25, banned=0, kind="sigmoid", smoothing=0.0, length_norm=False, grad_scale=1.0),
        # one short sampled answer in float32, with a few tokens of the vocabulary banned (-inf)
        dict(name="policy_one_answer", op="policy", tokens=96, vocab=50257, ld=50257, dtype="f32", prompt=0.25,
             banned=5, ref=True, weights=False, temperature=1.0, grad_scale=1.0),
        # a micro-batch of sampled answers over a large vocabulary, weighted token by token
        dict(name="policy_batch", op="policy", tokens=6144, vocab=131072, ld=131072, dtype="bf16", prompt=0.125,
             banned=0, ref=True, weights=True, temperature=0.8, grad_scale=1.0),
        # a short ragged sequence of a narrow odd layer's inputs, saved for the backward pass
        dict(name="save_short", op="save", rows=333, cols=1601, act="none", gated=False, dtype="f16"),
        # the MLP activations of a GPT-2 XL layer over a long micro-batch: function and checkpoint in one pass
        dict(name="save_mlp", op="save", rows=16384, cols=6400, act="gelu_tanh", gated=False, dtype="bf16"),
        # the backward pass of the same function, one short sequence of the smallest workload's MLP in float32
        dict(name="act_grad_short", op="act_grad", rows=257, cols=1536, act="gelu_tanh", gated=False, dtype="f32"),
        # the backward pass of a gated unit over a long micro-batch
        dict(name="act_grad_gated", op="act_grad", rows=16384, cols=4096, act="silu", gated=True, dtype="bf16"),
        # the attention input projection of GPT-2 small for one ragged sequence, binary16 gradients (loss scaling)
        dict(name="wgrad_short", op="wgrad", tokens=509, rows=768, cols=2304, dtype="f16", out="f16", accumulate=False),
        # the MLP's first weight in GPT-2 XL over a long micro-batch, added to the float32 gradient
        dict(name="wgrad_mlp", op="wgrad", tokens=16384, rows=1600, cols=6400, dtype="bf16", out="f32",
             accumulate=True),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, min(hi, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["logps", "preference", "policy", "save", "act_grad", "wgrad"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("logps", "policy", "preference"):
        vocab = _log_int(rng, 500, 131072)
        ld = vocab if rng.random() < 0.6 else (vocab + 63) // 64 * 64
        ld += 64 if ld == 3072 else 0
        banned = rng.choice([0, 0, rng.randrange(1, 9)])
        prompt = rng.choice([0.0, 0.25, 0.5])
        # the listed cases' bytes, whose prompts are not scored
        most = {"logps": 6144 * 50257 * 2, "policy": 5632 * 131072 * 2, "preference": 6016 * 50257 * 2}[op]
        rows = max(1, min(8192, most // (vocab * BYTES[dtype])))
        if op == "logps":
            return dict(op=op, tokens=_log_int(rng, 1, rows), vocab=vocab, ld=ld, dtype=dtype, prompt=prompt,
                        banned=banned, temperature=rng.choice([1.0, 0.7]))
        if op == "policy":
            return dict(op=op, tokens=_log_int(rng, 1, rows), vocab=vocab, ld=ld, dtype=dtype, prompt=prompt,
                        banned=banned, ref=rng.random() < 0.7, weights=rng.random() < 0.5,
                        temperature=rng.choice([1.0, 0.8]), grad_scale=256.0 if dtype == "f16" else 1.0)
        pairs = _log_int(rng, 1, 16)
        length = _log_int(rng, 2, max(2, min(1024, rows // (2 * pairs))))
        return dict(op=op, pairs=pairs, length=length, empty=rng.choice([0, 0, 1]), vocab=vocab, ld=ld, dtype=dtype,
                    prompt=prompt, banned=banned, kind=rng.choice(["sigmoid", "sigmoid", "ipo"]),
                    smoothing=rng.choice([0.0, 0.1]), length_norm=rng.random() < 0.3,
                    grad_scale=1024.0 if dtype == "f16" else 1.0)
    if op in ("save", "act_grad"):
        act = rng.choice(["gelu_tanh", "silu"] if op == "act_grad" else ["none", "gelu_tanh", "silu"])
        gated = act != "none" and rng.random() < 0.5
        cols = _log_int(rng, 33, 6400)
        if gated:
            cols = max(32, cols // 2 // 32 * 32)
            cols += 32 if cols in (1536, 3072) else 0
        rows = _log_int(rng, 1, 16384)
        most = 16384 * 4096 if op == "act_grad" else 16384 * 6400
        rows = max(1, min(rows, most * 2 // (cols * BYTES[dtype] * (2 if gated else 1))))
        return dict(op=op, rows=rows, cols=cols, act=act, gated=gated, dtype=dtype)
    dtype = rng.choice(["bf16", "f16"])
    rows, cols, tokens = _log_int(rng, 64, 6400), _log_int(rng, 64, 6400), _log_int(rng, 1, 16384)
    if rng.random() < 0.7:
        cols = (cols + 7) // 8 * 8
    if cols == 3072:
        cols += 8
    tokens = max(1, min(tokens, 16384 * 1600 * 6400 // (rows * cols)))
    return dict(op=op, tokens=tokens, rows=rows, cols=cols, dtype=dtype, out=rng.choice(["f32", "f32", "f16"]),
                accumulate=rng.random() < 0.5)


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------

def _lengths(case):
    """The sequences' lengths: ragged around case["length"] for pairs (a fixed pattern), runs of at most 512 tokens
    otherwise."""
    if case["op"] == "preference":
        n = 2 * case["pairs"]
        lens = [max(1, case["length"] - (37 * i + 11) % max(1, case["length"] // 3)) for i in range(n)]
        for i in range(case["empty"]):
            lens[(3 + 2 * i) % n] = 0
        return lens
    t = case["tokens"]
    return [min(512, t - a) for a in range(0, t, 512)]


def _active(case):
    """Which rows count: each sequence starts with its prompt, whose tokens are not scored."""
    on = []
    for n in _lengths(case):
        p = int(n * case["prompt"])
        on += [False] * p + [True] * (n - p)
    return on


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _logits(case, seed):
    """Logits as a language model's: a spread that differs from row to row, the scored token among the likely ones,
    some tokens of the vocabulary banned (half of them -inf, half the type's lowest value)."""
    g = _gen(seed)
    on = torch.tensor(_active(case), device="cuda")
    t, v = len(on), case["vocab"]
    dt = DTYPES[case["dtype"]]
    z = torch.randn(t, case["ld"], generator=g, device="cuda", dtype=torch.float32)
    z *= 1.0 + 2.0 * torch.rand(t, 1, generator=g, device="cuda")
    banned = case["banned"]
    targets = torch.randint(0, v - banned, (t,), generator=g, device="cuda")
    z[torch.arange(t, device="cuda"), targets] += 8.0 * torch.rand(t, generator=g, device="cuda")
    if banned:
        z[:, v - banned:v] = float("-inf")
        z[:, v - banned:v - banned // 2] = torch.finfo(dt).min
    z = z.to(dt)[:, :v]
    targets = torch.where(on, targets, torch.full_like(targets, -100))
    return z, targets, on, g


def _rough_logps(z, targets, temperature):
    """The scored tokens' log-probabilities, from which the other policies' are made."""
    out = []
    for a in range(0, z.shape[0], 2048):
        x = z[a:a + 2048].float() / temperature
        out.append(x.gather(1, targets[a:a + 2048].clamp(min=0)[:, None])[:, 0] - torch.logsumexp(x, 1))
    return torch.cat(out) if out else torch.zeros(0, device="cuda")


def _quantise(x, dt):
    """Codes (int8, rows padded to a multiple of 32 columns) and exponents (uint8, e + 127; rows padded to a multiple
    of 4 blocks) of a checkpoint, in torch operations."""
    t, m = x.shape
    blocks = (m + BLOCK - 1) // BLOCK
    xp = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - m)).view(t, blocks, BLOCK)
    bits = xp.abs().amax(2).view(torch.int32)
    biased = (((bits + 0x10000) >> 23) - 6).clamp(min=103 if dt == torch.float16 else 1)
    inverse = ((254 - biased) << 23).view(torch.float32)
    q = torch.round(xp * inverse[..., None])
    if dt == torch.float16:
        most = torch.floor(65504.0 * inverse)[..., None]
        q = torch.minimum(torch.maximum(q, -most), most)
    bad = bits >= 0x7F800000
    q = torch.where(bad[..., None], torch.zeros_like(q), q)
    biased = torch.where(bad, torch.full_like(biased, 255), biased)
    lds = (blocks + 3) // 4 * 4
    return q.to(torch.int8).view(t, blocks * BLOCK), torch.nn.functional.pad(biased, (0, lds - blocks)).to(torch.uint8)


def _activations(g, t, m, dt):
    """Activations: most of a row near one size, a few columns much larger, as a transformer's residual stream has."""
    x = torch.randn(t, m, generator=g, device="cuda", dtype=torch.float32)
    x *= 0.5 + torch.rand(1, m, generator=g, device="cuda")
    loud = torch.randint(0, m, (max(1, m // 200),), generator=g, device="cuda")
    x[:, loud] *= 12.0
    return x.to(dt)


def prepare(case, seed):
    op = case["op"]
    s = dict(case=case)
    if op in ("logps", "preference", "policy"):
        z, targets, on, g = _logits(case, seed)
        s.update(logits=z, targets=targets)
        t = z.shape[0]
        noise = lambda: torch.randn(t, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
        if op == "preference":
            lp = _rough_logps(z, targets, 1.0)
            s["ref"] = torch.where(on, lp + 0.2 * noise(), torch.zeros_like(lp))
            ends = [0]
            for n in _lengths(case):
                ends.append(ends[-1] + n)
            s["cu_seqlens"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        if op == "policy":
            lp = _rough_logps(z, targets, case["temperature"])
            d = 0.2 * noise()
            r = torch.exp(d)  # nothing sits on the clip's edges, where either side is right
            edge = ((r - (1 - CLIP_LOW)).abs() < 1e-3) | ((r - (1 + CLIP_HIGH)).abs() < 1e-3)
            s["old"] = lp - torch.where(edge, torch.zeros_like(d), d)
            s["ref"] = lp + 0.1 * noise() if case["ref"] else None
            s["advantages"] = noise()
            s["weights"] = 0.5 + torch.rand(t, generator=g, device="cuda") if case["weights"] else None
            s["denom"] = float(max(1, int(on.sum())))
        return s
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    if op == "save":
        s["x"] = _activations(g, case["rows"], case["cols"] * (2 if case["gated"] else 1), dt)
        return s
    if op == "act_grad":
        x = _activations(g, case["rows"], case["cols"] * (2 if case["gated"] else 1), dt)
        s["codes"], s["scales"] = _quantise(x, dt)
        s["dy"] = (1e-2 * torch.randn(case["rows"], case["cols"], generator=g, device="cuda")).to(dt)
        return s
    x = _activations(g, case["tokens"], case["rows"], dt)
    s["codes"], s["scales"] = _quantise(x, dt)
    size = 1.0 if case["dtype"] == "f16" else 1e-3  # binary16 gradients come scaled
    s["dy"] = (size * torch.randn(case["tokens"], case["cols"], generator=g, device="cuda")).to(dt)
    if case["accumulate"]:
        s["dw"] = (size * torch.randn(case["rows"], case["cols"], generator=g, device="cuda")).to(DTYPES[case["out"]])
    return s


# ----------------------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------------------

def _values(codes, scales, cols):
    """What a checkpoint stands for, in float32."""
    t, padded = codes.shape
    blocks = padded // BLOCK
    e = scales[:, :blocks].int()
    step = torch.where(e == 255, torch.full_like(e, 0x7FC00000), e << 23).view(torch.float32)
    return (codes.float().view(t, blocks, BLOCK) * step[..., None]).reshape(t, padded)[:, :cols]


def _act(x, kind):
    """The activation function and its derivative, in float32."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return x * s, s * (1.0 + x * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    u = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1.0 + u), 0.5 * (1.0 + u) + 0.5 * x * (1.0 - u * u) * c * (1.0 + 3 * 0.044715 * x * x)


def _softmax(z, temperature):
    """Row softmax in float32: x minus its row's maximum, exp of it, the sums, and their logarithms."""
    x = z.float() * (1.0 / temperature)
    x = x - x.amax(1, keepdim=True)
    p = torch.exp(x)
    s = p.sum(1, keepdim=True)
    return x, p, s, torch.log(s)


def _gather(x, targets):
    return x.gather(1, targets.clamp(min=0)[:, None])[:, 0]


def _dlogits(z, p, s, targets, coef):
    """coef * (1[target] - p) row by row, rounded once."""
    d = p * (-coef[:, None] / s)
    rows = torch.arange(z.shape[0], device=z.device)
    t = targets.clamp(min=0)
    d[rows, t] = coef * (1.0 - _gather(p, targets) / s[:, 0])
    return d.to(z.dtype)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "logps":
        x, p, t, l = _softmax(s["logits"], c["temperature"])
        on = s["targets"] >= 0
        zero = torch.zeros((), device=x.device)
        h = l[:, 0] - (p * torch.where(p > 0, x, zero)).sum(1) / t[:, 0]
        return dict(logps=torch.where(on, _gather(x, s["targets"]) - l[:, 0], zero), entropy=torch.where(on, h, zero))
    if op == "preference":
        x, p, t, l = _softmax(s["logits"], 1.0)
        on = s["targets"] >= 0
        zero = torch.zeros((), device=x.device)
        lp = torch.where(on, _gather(x, s["targets"]) - l[:, 0], zero)
        ends = s["cu_seqlens"].long()
        rows = torch.arange(lp.shape[0], device=lp.device)
        member = ((rows[None] >= ends[:-1, None]) & (rows[None] < ends[1:, None]) & on[None]).float()
        d = member @ (lp - torch.where(on, s["ref"], zero))
        share = torch.ones_like(d)
        if c["length_norm"]:
            share = 1.0 / member.sum(1).clamp(min=1.0)
        d = d * share
        h = BETA * (d[0::2] - d[1::2])
        eps, pairs = c["smoothing"], c["pairs"]
        if c["kind"] == "sigmoid":
            soft = lambda v: torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))  # noqa: E731
            loss = (1 - eps) * soft(-h) + eps * soft(h)
            slope = -(1 - eps) / (1 + torch.exp(h)) + eps / (1 + torch.exp(-h))
            slope = slope * BETA
        else:
            gap = d[0::2] - d[1::2] - 1.0 / (2.0 * BETA)
            loss, slope = gap * gap, 2.0 * gap
        both = torch.stack([slope, -slope], 1).reshape(-1) * share * (c["grad_scale"] / pairs)
        coef = both @ member
        return dict(loss=loss.mean().reshape(1), rewards=BETA * d, logps=lp,
                    dlogits=_dlogits(s["logits"], p, t, s["targets"], coef))
    if op == "policy":
        x, p, t, l = _softmax(s["logits"], c["temperature"])
        on = s["targets"] >= 0
        zero = torch.zeros((), device=x.device)
        lp = _gather(x, s["targets"]) - l[:, 0]
        w = on.float() if s["weights"] is None else torch.where(on, s["weights"], zero)
        w = w / s["denom"]
        a = s["advantages"]
        r = torch.exp(lp - s["old"])
        free, held = r * a, torch.clamp(r, 1 - CLIP_LOW, 1 + CLIP_HIGH) * a
        clipped = held < free
        surrogate = -torch.minimum(free, held)
        slope = torch.where(clipped, zero, -free)
        kl = torch.zeros_like(lp)
        if s["ref"] is not None:
            q = s["ref"] - lp
            kl = torch.exp(q) - q - 1.0
            slope = slope + KL_COEF * (1.0 - torch.exp(q))
        coef = torch.where(on, slope * w, zero) * (c["grad_scale"] / c["temperature"])
        total = lambda v: torch.where(on, v * w, zero).sum()  # noqa: E731
        parts = [total(surrogate + KL_COEF * kl), total(surrogate), total(kl), total(clipped.float())]
        return dict(stats=torch.stack(parts), logps=torch.where(on, lp, zero),
                    dlogits=_dlogits(s["logits"], p, t, s["targets"], coef))
    if op == "save":
        x = s["x"]
        codes, scales = _quantise(x, x.dtype)
        out = dict(values=_values(codes, scales, x.shape[1]).to(x.dtype))
        if c["act"] != "none":
            f = c["cols"]
            y = _act(x[:, :f].float(), c["act"])[0]
            out["y"] = (y * x[:, f:].float() if c["gated"] else y).to(x.dtype)
        return out
    if op == "act_grad":
        f = c["cols"]
        x = _values(s["codes"], s["scales"], f * (2 if c["gated"] else 1))
        y, slope = _act(x[:, :f], c["act"])
        dy = s["dy"].float()
        if not c["gated"]:
            return (dy * slope).to(s["dy"].dtype)
        return torch.cat([dy * x[:, f:] * slope, dy * y], 1).to(s["dy"].dtype)
    x = _values(s["codes"], s["scales"], c["rows"])
    dw = x.t() @ s["dy"].float()
    if c["accumulate"]:
        dw = dw + s["dw"].float()
    return dw.to(DTYPES[c["out"]])


def _own(s):
    import clip_tensor_adamw_gb300 as mica
    c = s["case"]
    op = c["op"]
    if op == "logps":
        lp, h = mica.mica_token_logps(s["logits"], s["targets"], temperature=c["temperature"], entropy=True)
        return dict(logps=lp, entropy=h)
    if op == "preference":
        r = mica.mica_preference_loss(s["logits"], s["targets"], s["cu_seqlens"], s["ref"], beta=BETA, kind=c["kind"],
                                      label_smoothing=c["smoothing"], length_norm=c["length_norm"],
                                      grad_scale=c["grad_scale"])
        return dict(loss=r.loss, rewards=r.rewards, logps=r.logps, dlogits=r.dlogits)
    if op == "policy":
        r = mica.mica_policy_loss(s["logits"], s["targets"], s["old"], s["advantages"], denom=s["denom"],
                                  ref_logps=s["ref"], weights=s["weights"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                                  kl_coef=KL_COEF, temperature=c["temperature"], grad_scale=c["grad_scale"])
        return dict(stats=r.stats, logps=r.logps, dlogits=r.dlogits)
    if op == "save":
        if c["act"] == "none":
            return dict(values=mica.mica_act_unpack(mica.mica_act_pack(s["x"])))
        packed, y = mica.mica_act_pack(s["x"], act=c["act"], gated=c["gated"])
        return dict(values=mica.mica_act_unpack(packed), y=y)
    cols = c["rows"] if op == "wgrad" else c["cols"] * (2 if c["gated"] else 1)
    packed = mica.PackedActivation(s["codes"], s["scales"], cols, DTYPES[c["dtype"]])
    if op == "act_grad":
        return mica.mica_act_grad(packed, s["dy"], act=c["act"], gated=c["gated"])
    return mica.mica_packed_wgrad(packed, s["dy"], add=s["dw"] if c["accumulate"] else None, out_dtype=DTYPES[c["out"]])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    if op in ("logps", "preference", "policy"):
        on = _active(case)
        t, v, live = len(on), case["vocab"], sum(on)
        vectors = {"logps": 8 + 4 + 4, "preference": 8 + 4 + 4, "policy": 8 + 4 * 3 + 4 * case.get("ref", 0) +
                   4 * case.get("weights", 0)}[op]
        # rows that do not count are not read, but their gradient is written
        return dict(bytes=live * v * b + (0 if op == "logps" else t * v * b) + t * vectors,
                    flops=live * v * (5 if op == "logps" else 6))
    if op == "save":
        m = case["cols"] * (2 if case["gated"] else 1)
        held = case["rows"] * (m + (m + BLOCK - 1) // BLOCK)  # a checkpoint is written, and read again
        y = case["rows"] * case["cols"] * b if case["act"] != "none" else 0
        return dict(bytes=2 * case["rows"] * m * b + 2 * held + y, flops=4 * case["rows"] * m)
    if op == "act_grad":
        m = case["cols"] * (2 if case["gated"] else 1)
        return dict(bytes=case["rows"] * (m + (m + BLOCK - 1) // BLOCK + case["cols"] * b + m * b),
                    flops=20 * case["rows"] * case["cols"])
    t, m, n = case["tokens"], case["rows"], case["cols"]
    return dict(bytes=t * (m + (m + BLOCK - 1) // BLOCK) + t * n * b +
                m * n * BYTES[case["out"]] * (2 if case["accumulate"] else 1), flops=2 * t * m * n)


# ----------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------------------------------------------

def _exact_values(codes, scales, cols):
    e = scales.to(torch.float64)[:, :codes.shape[1] // BLOCK]
    step = torch.where(e == 255, torch.full_like(e, float("nan")), torch.exp2(e - 127.0))
    return (codes.to(torch.float64) * step.repeat_interleave(BLOCK, 1))[:, :cols]


def _exact_act(x, kind):
    if kind == "silu":
        return x * torch.sigmoid(x)
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)))


def _exact_logps(z, targets, temperature, coef=None):
    """(log-probabilities, entropies, gradient of sum(coef * log-probabilities)) in float64, some rows at a time."""
    lps, hs, grads = [], [], []
    for a in range(0, z.shape[0], 1024):
        x = (z[a:a + 1024].double() / temperature)
        lse = torch.logsumexp(x, 1, keepdim=True)
        t = targets[a:a + 1024]
        lp = x.gather(1, t.clamp(min=0)[:, None]) - lse
        p = torch.exp(x - lse)
        lps.append(torch.where(t >= 0, lp[:, 0], 0.0))
        if coef is None:
            hs.append(torch.where(t >= 0, torch.special.entr(p).sum(1), 0.0))
        else:
            k = (torch.where(t >= 0, coef[a:a + 1024], 0.0) / temperature)[:, None]
            p = -k * p
            p.scatter_add_(1, t.clamp(min=0)[:, None], k)
            grads.append(p)
    return torch.cat(lps), torch.cat(hs) if hs else None, torch.cat(grads) if grads else None


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "logps":
        lp, h, _ = _exact_logps(s["logits"], s["targets"], case["temperature"])
        return dict(logps=lp, entropy=h)
    if op in ("preference", "policy"):
        temperature = case.get("temperature", 1.0)
        lp = _exact_logps(s["logits"], s["targets"], temperature)[0].requires_grad_()
        on = s["targets"] >= 0
        if op == "preference":
            ends = s["cu_seqlens"].tolist()
            ref = torch.where(on, s["ref"].double(), 0.0)
            d = []
            for a, b in zip(ends[:-1], ends[1:]):
                n = max(1, int(on[a:b].sum())) if case["length_norm"] else 1
                d.append(((lp[a:b] - ref[a:b]) * on[a:b]).sum() / n)
            d = torch.stack(d)
            delta = d[0::2] - d[1::2]
            if case["kind"] == "sigmoid":
                log_s = torch.nn.functional.logsigmoid
                loss = -(1 - case["smoothing"]) * log_s(BETA * delta) - case["smoothing"] * log_s(-BETA * delta)
            else:
                loss = (delta - 1.0 / (2.0 * BETA)) ** 2
            loss = loss.mean()
            first = dict(loss=loss.detach().reshape(1), rewards=BETA * d.detach())
        else:
            a = s["advantages"].double()
            w = on.double() if s["weights"] is None else s["weights"].double() * on
            r = torch.exp(lp - s["old"].double())
            held = torch.clamp(r, 1 - CLIP_LOW, 1 + CLIP_HIGH)
            surrogate = -torch.minimum(r * a, held * a)
            kl = torch.zeros_like(lp)
            if s["ref"] is not None:
                q = s["ref"].double() - lp
                kl = torch.exp(q) - 1.0 - q
            mean = lambda v: torch.where(on, v * w, 0.0).sum() / s["denom"]  # noqa: E731
            loss = mean(surrogate + KL_COEF * kl)
            parts = [loss, mean(surrogate), mean(kl), mean((held * a < r * a).double())]
            first = dict(stats=torch.stack([v.detach() for v in parts]))
        coef, = torch.autograd.grad(loss * case["grad_scale"], lp)
        dz = _exact_logps(s["logits"], s["targets"], temperature, coef)[2]
        return dict(first, logps=lp.detach(), dlogits=dz)
    if op == "save":
        x = s["x"].double()
        t, m = x.shape
        pad = torch.nn.functional.pad(x, (0, -m % BLOCK)).view(t, -1, BLOCK)
        most = pad.abs().amax(2)
        e = torch.ceil(torch.log2(torch.where(most > 0, most, 1.0) / 127.5))
        e = torch.where(most / torch.exp2(e) >= 127.5, e + 1, e)
        e = torch.where(most / torch.exp2(e - 1) < 127.5, e - 1, e)
        e = e.clamp(min=-24 if case["dtype"] == "f16" else -126)
        e = torch.where(most > 0, e, 0.0)[..., None]
        v = torch.round(pad / torch.exp2(e)) * torch.exp2(e)
        if case["dtype"] == "f16":
            limit = torch.floor(65504.0 / torch.exp2(e)) * torch.exp2(e)
            v = torch.minimum(torch.maximum(v, -limit), limit)
        v = torch.where(torch.isfinite(most)[..., None], v, float("nan"))
        out = dict(values=v.reshape(t, -1)[:, :m])
        if case["act"] != "none":
            f = case["cols"]
            y = _exact_act(x[:, :f], case["act"])
            out["y"] = y * x[:, f:] if case["gated"] else y
        return out
    if op == "act_grad":
        f = case["cols"]
        x = _exact_values(s["codes"], s["scales"], f * (2 if case["gated"] else 1)).requires_grad_()
        y = _exact_act(x[:, :f], case["act"])
        if case["gated"]:
            y = y * x[:, f:]
        return torch.autograd.grad(y, x, s["dy"].double())[0]
    x = _exact_values(s["codes"], s["scales"], case["rows"])
    dw = torch.einsum("tm,tn->mn", x, s["dy"].double())
    return dw + s["dw"].double() if case["accumulate"] else dw
