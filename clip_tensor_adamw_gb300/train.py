"""Python binding of the operators of include/mica_train.h, taking torch tensors: losses over logits with the gradient
of the logits, losses from hidden states with the gradients of these and of the output embedding, and activation
checkpoints in 8 bits with the backward passes that read them.

As in mica.py, this module only marshals arguments: every element is read and written by the library's kernels, and there
is no fallback. What a call returns is allocated on the stream that it runs on (``stream``, by default the current one),
so that the caching allocator gives it out again in that stream's order.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from .mica import _check, lib

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 4}
_KINDS = {"sigmoid": 0, "hinge": 1, "ipo": 2}
_ACTS = {"none": 0, "gelu_tanh": 1, "gelu": 2, "silu": 3, "relu": 4}
_LENGTH_NORM = 1
BLOCK = 32  # columns of a checkpoint that share a step

_P, _I32, _I64, _F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


class _Logits(ctypes.Structure):
    _fields_ = [("logits", _P), ("targets", _P), ("rows", _I64), ("vocab", _I64), ("ld", _I64), ("temperature", _F64),
                ("dtype", _I32), ("target_bytes", _I32)]


class _PreferenceHP(ctypes.Structure):
    _fields_ = [("beta", _F64), ("label_smoothing", _F64), ("grad_scale", _F64), ("kind", _I32),
                ("flags", ctypes.c_uint32)]


class _PolicyHP(ctypes.Structure):
    _fields_ = [("clip_low", _F64), ("clip_high", _F64), ("kl_coef", _F64), ("denom", _F64), ("grad_scale", _F64)]


class _Packed(ctypes.Structure):
    _fields_ = [("codes", _P), ("steps", _P), ("rows", _I64), ("cols", _I64), ("ld", _I64), ("ld_s", _I64),
                ("dtype", _I32), ("reserved", _I32)]


class _Linear(ctypes.Structure):
    _fields_ = [("h", _P), ("w", _P), ("targets", _P), ("rows", _I64), ("features", _I64), ("vocab", _I64),
                ("ld_h", _I64), ("ld_w", _I64), ("temperature", _F64), ("dtype", _I32), ("target_bytes", _I32)]


class _LinearGrads(ctypes.Structure):
    _fields_ = [("dh", _P), ("dw", _P), ("add", _P), ("ld_dh", _I64), ("ld_dw", _I64), ("ld_add", _I64),
                ("dw_dtype", _I32), ("reserved", _I32)]


class _CrossEntropyHP(ctypes.Structure):
    _fields_ = [("denom", _F64), ("grad_scale", _F64)]


_LP, _QP, _OP, _KP = (ctypes.POINTER(t) for t in (_Logits, _PreferenceHP, _PolicyHP, _Packed))
_HP, _GP, _CP = (ctypes.POINTER(t) for t in (_Linear, _LinearGrads, _CrossEntropyHP))
_lib = None


def _train() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = lib()
        for name, args in {
            "mica_token_logps": [_LP, _P, _P, _P],
            "mica_token_logps_grad": [_LP, _P, _P, _I64, _P],
            "mica_preference_loss": [_LP, _P, _I32, _P, _QP, _P, _P, _P, _P, _I64, _P, _I64, _P],
            "mica_policy_loss": [_LP, _P, _P, _P, _P, _OP, _P, _P, _P, _I64, _P],
            "mica_act_pack": [_P, _I64, _KP, _I32, _I32, _P, _I64, _P],
            "mica_act_unpack": [_KP, _P, _I64, _P],
            "mica_act_grad": [_KP, _I32, _I32, _P, _I64, _I32, _P, _I64, _P],
            "mica_packed_wgrad": [_KP, _P, _I64, _I32, _I64, _P, _I64, _P, _I64, _I32, _P, _I64, _P],
            "mica_linear_logps": [_HP, _P, _P, _P, _I64, _P],
            "mica_linear_logps_grad": [_HP, _P, _P, _GP, _P, _I64, _P],
            "mica_linear_cross_entropy": [_HP, _CP, _P, _P, _GP, _P, _I64, _P],
        }.items():
            getattr(L, name).argtypes = args
            getattr(L, name).restype = ctypes.c_int
        L.mica_preference_workspace.argtypes = [_I64, _I32]
        L.mica_preference_workspace.restype = _I64
        L.mica_packed_wgrad_workspace.argtypes = [_KP, _P, _I64, _I64]
        L.mica_packed_wgrad_workspace.restype = _I64
        for name, args in {
            "mica_linear_logps_workspace": [_HP],
            "mica_linear_grad_workspace": [_HP, _GP],
            "mica_linear_cross_entropy_workspace": [_HP, _GP],
        }.items():
            getattr(L, name).argtypes = args
            getattr(L, name).restype = _I64
        _lib = L
    return _lib


class _On:
    """The stream a call runs on, current while its outputs are allocated."""

    __slots__ = ("context", "handle")

    def __init__(self, stream, device):
        if stream is None:  # (torch.cuda.current_stream builds a Stream object, 2 us of a small call's 15)
            self.context, self.handle = None, torch._C._cuda_getCurrentRawStream(device.index or 0)
            return
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        self.context, self.handle = torch.cuda.stream(stream), stream.cuda_stream

    def __enter__(self):
        if self.context is not None:
            self.context.__enter__()
        return self.handle

    def __exit__(self, *e):
        if self.context is not None:
            self.context.__exit__(*e)


def _type(t: torch.Tensor, what: str) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: unsupported dtype {t.dtype}")
    return code


def _matrix(t: torch.Tensor, what: str) -> int:
    """A matrix whose rows are contiguous; its row stride."""
    if t.ndim != 2:
        raise ValueError(f"{what} must have two dimensions, not {t.ndim}")
    rows, cols = t.shape
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{what}: the elements of a row must be contiguous")
    return ld if rows > 1 else max(ld, cols)


def _vector(t: torch.Tensor | None, n: int, what: str, dtype=torch.float32) -> int | None:
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.ndim != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n} elements, not {tuple(t.shape)}")
    return t.data_ptr()


def _output(t: torch.Tensor | None, shape: tuple, dtype, what: str, like: torch.Tensor) -> torch.Tensor:
    """`t` when given (its shape and type checked), or a new matrix."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    if tuple(t.shape) != shape or t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} of shape {shape}, not {t.dtype} of {tuple(t.shape)}")
    return t


def _logits(logits: torch.Tensor, targets: torch.Tensor, temperature: float) -> _Logits:
    code, ld = _type(logits, "logits"), _matrix(logits, "logits")
    rows, vocab = logits.shape
    if targets.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"targets must be int32 or int64, not {targets.dtype}")
    y = _vector(targets, rows, "targets", targets.dtype)
    return _Logits(logits.data_ptr(), y, rows, vocab, ld, float(temperature), code, targets.element_size())


def _dlogits(out: torch.Tensor | None, logits: torch.Tensor, ld: int) -> torch.Tensor:
    """A given buffer, or a new one whose rows lie as the logits' do within lines of 128 bytes (so that both are equally
    aligned), and no further apart than that takes: the logits may be every so many rows of a larger tensor."""
    if out is None:
        rows, vocab = logits.shape
        if ld <= vocab:
            return torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        ld = vocab + (ld - vocab) % (128 // logits.element_size())
        return torch.empty((rows, ld), dtype=logits.dtype, device=logits.device)[:, :vocab]
    if out.shape != logits.shape or out.dtype != logits.dtype:
        raise ValueError("dlogits must have the logits' shape and dtype")
    return out


def mica_token_logps(logits: torch.Tensor, targets: torch.Tensor, *, temperature: float = 1.0, entropy: bool = False,
                     stream=None):
    """Log-probabilities of ``targets`` (int32 or int64, [rows]; negative: not scored, 0) under the softmax of
    ``logits / temperature`` ([rows, vocabulary], float32, float16 or bfloat16, any row stride), float32 [rows]; with
    ``entropy``, also the rows' entropies: ``(logps, entropies)``."""
    z = _logits(logits, targets, temperature)
    with _On(stream, logits.device) as s:
        logps = torch.empty(z.rows, dtype=torch.float32, device=logits.device)
        h = torch.empty_like(logps) if entropy else None
        _check(_train().mica_token_logps(z, logps.data_ptr(), None if h is None else h.data_ptr(), s))
    return (logps, h) if entropy else logps


def mica_token_logps_grad(logits: torch.Tensor, targets: torch.Tensor, dlogps: torch.Tensor, *,
                          temperature: float = 1.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of the logits given that of mica_token_logps's result, for any loss over log-probabilities. ``out``
    may be ``logits`` itself (in place)."""
    z = _logits(logits, targets, temperature)
    g = _vector(dlogps, z.rows, "dlogps")
    with _On(stream, logits.device) as s:
        d = _dlogits(out, logits, z.ld)
        _check(_train().mica_token_logps_grad(z, g, d.data_ptr(), _matrix(d, "dlogits"), s))
    return d


class PreferenceLoss(NamedTuple):
    loss: torch.Tensor            # [1], the mean over pairs
    rewards: torch.Tensor         # [2 * pairs], beta times the sequences' log-ratios (chosen, rejected, chosen, ...)
    logps: torch.Tensor           # [rows]
    dlogits: torch.Tensor | None  # the gradient of grad_scale * loss


class PolicyLoss(NamedTuple):
    stats: torch.Tensor           # [4]: loss, surrogate, KL term, clipped share
    logps: torch.Tensor           # [rows]
    dlogits: torch.Tensor | None  # the gradient of grad_scale * loss


def mica_preference_loss(logits: torch.Tensor, targets: torch.Tensor, cu_seqlens: torch.Tensor,
                         ref_logps: torch.Tensor | None = None, *, beta: float = 0.1, kind: str = "sigmoid",
                         label_smoothing: float = 0.0, length_norm: bool = False, temperature: float = 1.0,
                         grad_scale: float = 1.0, grad: bool = True, out: torch.Tensor | None = None,
                         stream=None) -> PreferenceLoss:
    """A preference loss (``kind`` "sigmoid", "hinge" or "ipo") over pairs of sequences packed into the rows of
    ``logits``, and the gradient of the logits. ``cu_seqlens``: int32 [2 * pairs + 1], the sequences' first rows, chosen
    and rejected in turn; ``ref_logps``: the reference policy's log-probabilities, [rows], or None for zeros;
    ``length_norm`` divides a sequence's sum by its scored tokens. ``out`` takes the gradient; it may be ``logits``
    itself. ``grad=False`` leaves it out (dlogits None)."""
    z = _logits(logits, targets, temperature)
    if kind not in _KINDS:
        raise ValueError(f"kind {kind!r} is none of {sorted(_KINDS)}")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] % 2 == 0:
        raise ValueError("cu_seqlens must hold 2 * pairs + 1 entries")
    pairs = cu_seqlens.shape[0] // 2
    ends = _vector(cu_seqlens, 2 * pairs + 1, "cu_seqlens", torch.int32)
    ref = _vector(ref_logps, z.rows, "ref_logps")
    hp = _PreferenceHP(float(beta), float(label_smoothing), float(grad_scale), _KINDS[kind],
                       _LENGTH_NORM if length_norm else 0)
    L = _train()
    with _On(stream, logits.device) as s:
        dev = logits.device
        loss = torch.empty(1, dtype=torch.float32, device=dev)
        rewards = torch.empty(2 * pairs, dtype=torch.float32, device=dev)
        logps = torch.empty(z.rows, dtype=torch.float32, device=dev)
        d = _dlogits(out, logits, z.ld) if grad else None
        size = L.mica_preference_workspace(z.rows, pairs)
        work = torch.empty(size, dtype=torch.uint8, device=dev)
        _check(L.mica_preference_loss(z, ends, pairs, ref, hp, loss.data_ptr(), rewards.data_ptr(), logps.data_ptr(),
                                      None if d is None else d.data_ptr(), 0 if d is None else _matrix(d, "dlogits"),
                                      work.data_ptr(), size, s))
    return PreferenceLoss(loss, rewards, logps, d)


def mica_policy_loss(logits: torch.Tensor, targets: torch.Tensor, old_logps: torch.Tensor, advantages: torch.Tensor, *,
                     denom: float, ref_logps: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                     clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0,
                     grad_scale: float = 1.0, grad: bool = True, out: torch.Tensor | None = None,
                     stream=None) -> PolicyLoss:
    """A clipped policy loss with a KL term, token by token, and the gradient of the logits: the sum over scored rows
    of ``weights`` * (clipped surrogate + ``kl_coef`` * KL estimate) / ``denom``, all inputs float32 [rows]. ``stats`` is
    (loss, surrogate, KL, clipped share). ``out`` takes the gradient; it may be ``logits`` itself. ``grad=False``
    leaves it out (dlogits None)."""
    z = _logits(logits, targets, temperature)
    old, adv = _vector(old_logps, z.rows, "old_logps"), _vector(advantages, z.rows, "advantages")
    ref, w = _vector(ref_logps, z.rows, "ref_logps"), _vector(weights, z.rows, "weights")
    hp = _PolicyHP(float(clip_low), float(clip_high), float(kl_coef), float(denom), float(grad_scale))
    with _On(stream, logits.device) as s:
        stats = torch.empty(4, dtype=torch.float32, device=logits.device)
        logps = torch.empty(z.rows, dtype=torch.float32, device=logits.device)
        d = _dlogits(out, logits, z.ld) if grad else None
        _check(_train().mica_policy_loss(z, old, adv, ref, w, hp, stats.data_ptr(), logps.data_ptr(),
                                         None if d is None else d.data_ptr(),
                                         0 if d is None else _matrix(d, "dlogits"), s))
    return PolicyLoss(stats, logps, d)


class PackedActivation:
    """An activation's checkpoint in 8 bits: ``codes`` (int8 [rows, a multiple of 32 >= cols]) and ``steps`` (uint8
    [rows, a multiple of 4 >= blocks of 32 columns]), with the ``cols`` and ``dtype`` of its source. Rows may lie
    further apart (a stride that is a multiple of 32, and of 4)."""

    __slots__ = ("codes", "steps", "cols", "dtype", "_c")

    def __init__(self, codes: torch.Tensor, steps: torch.Tensor, cols: int, dtype: torch.dtype):
        if codes.dtype != torch.int8 or steps.dtype != torch.uint8:
            raise TypeError(f"codes must be int8 and steps uint8, not {codes.dtype} and {steps.dtype}")
        if dtype not in _TYPES:
            raise TypeError(f"unsupported dtype {dtype}")
        ld, ld_s = _matrix(codes, "codes"), _matrix(steps, "steps")
        rows, blocks = codes.shape[0], (cols + BLOCK - 1) // BLOCK
        if steps.shape[0] != rows or codes.shape[1] < blocks * BLOCK or steps.shape[1] < blocks:
            raise ValueError(f"{cols} columns need {blocks} blocks: got codes {tuple(codes.shape)} and steps "
                             f"{tuple(steps.shape)}")
        self.codes, self.steps, self.cols, self.dtype = codes, steps, int(cols), dtype
        self._c = _Packed(codes.data_ptr(), steps.data_ptr(), rows, self.cols, ld, ld_s, _TYPES[dtype], 0)

    @classmethod
    def empty(cls, rows: int, cols: int, dtype: torch.dtype, device=None) -> "PackedActivation":
        """Buffers for a rows x cols activation, for mica_act_pack to fill."""
        blocks = (cols + BLOCK - 1) // BLOCK
        return cls(torch.empty((rows, blocks * BLOCK), dtype=torch.int8, device=device),
                   torch.empty((rows, (blocks + 3) // 4 * 4), dtype=torch.uint8, device=device), cols, dtype)

    @property
    def shape(self) -> tuple:
        return (self.codes.shape[0], self.cols)


def _act(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act {act!r} is none of {sorted(_ACTS)}")
    return _ACTS[act]


def mica_act_pack(x: torch.Tensor, act: str = "none", *, gated: bool = False, packed: PackedActivation | None = None,
                  out: torch.Tensor | None = None, stream=None):
    """The 8-bit checkpoint of ``x`` ([rows, cols], any row stride). With ``act`` ("gelu_tanh", "gelu", "silu", "relu")
    also the activation function's value y at ``x``, in the same pass: ``(packed, y)``; ``gated`` takes the first half of
    the columns through the function and multiplies it by the second. ``packed`` and ``out`` are filled when given."""
    code, ld = _type(x, "x"), _matrix(x, "x")
    rows, cols = x.shape
    kind = _act(act)
    with _On(stream, x.device) as s:
        p = PackedActivation.empty(rows, cols, x.dtype, x.device) if packed is None else packed
        if p.shape != (rows, cols) or p.dtype != x.dtype:
            raise ValueError("packed must be a checkpoint of x's shape and dtype")
        y = _output(out, (rows, cols // 2 if gated else cols), x.dtype, "out", x) if kind else out
        _check(_train().mica_act_pack(x.data_ptr(), ld, p._c, kind, int(gated), None if y is None else y.data_ptr(),
                                      0 if y is None else _matrix(y, "out"), s))
    return (p, y) if kind else p


def mica_act_unpack(packed: PackedActivation, *, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values a checkpoint stands for, exactly, in its source's dtype."""
    with _On(stream, packed.codes.device) as s:
        x = _output(out, packed.shape, packed.dtype, "out", packed.codes)
        _check(_train().mica_act_unpack(packed._c, x.data_ptr(), _matrix(x, "out"), s))
    return x


def mica_act_grad(packed: PackedActivation, dy: torch.Tensor, act: str, *, gated: bool = False,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The gradient of the input of an activation function from that of its output and the input's checkpoint. ``dy``
    is [rows, cols], or [rows, cols / 2] when ``gated``; the result has ``dy``'s dtype and the checkpoint's shape. ``out``
    may be ``dy`` itself when not gated."""
    code, ld = _type(dy, "dy"), _matrix(dy, "dy")
    rows, cols = packed.shape
    kind = _act(act)
    if tuple(dy.shape) != (rows, cols // 2 if gated else cols):
        raise ValueError(f"dy must have the shape of the function's output, not {tuple(dy.shape)}")
    with _On(stream, dy.device) as s:
        dx = _output(out, (rows, cols), dy.dtype, "out", dy)
        _check(_train().mica_act_grad(packed._c, kind, int(gated), dy.data_ptr(), ld, code, dx.data_ptr(),
                                      _matrix(dx, "out"), s))
    return dx


def mica_packed_wgrad(packed: PackedActivation, dy: torch.Tensor, *, add: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                      stream=None) -> torch.Tensor:
    """The weight gradient of y = x W from x's checkpoint ([tokens, features]) and ``dy`` ([tokens, n], bfloat16, or
    float16 for the checkpoint of a float16 activation): ``add`` + x^T dy, [features, n], of ``out_dtype`` (by default
    that of ``out``, then of ``add``, then float32). ``add`` may be ``out`` itself (accumulation in place)."""
    code, ld = _type(dy, "dy"), _matrix(dy, "dy")
    tokens, features = packed.shape
    if dy.shape[0] != tokens:
        raise ValueError(f"dy has {dy.shape[0]} tokens and the checkpoint {tokens}")
    n = dy.shape[1]
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else add.dtype if add is not None else torch.float32
    if add is not None and (tuple(add.shape) != (features, n) or add.dtype != out_dtype):
        raise ValueError(f"add must be {out_dtype} of shape {(features, n)}, not {add.dtype} of {tuple(add.shape)}")
    L = _train()
    with _On(stream, dy.device) as s:
        dw = _output(out, (features, n), out_dtype, "out", dy)
        size = L.mica_packed_wgrad_workspace(packed._c, dy.data_ptr(), ld, n)
        work = torch.empty(size, dtype=torch.uint8, device=dy.device) if size else None
        _check(L.mica_packed_wgrad(packed._c, dy.data_ptr(), ld, code, n, None if add is None else add.data_ptr(),
                                   0 if add is None else _matrix(add, "add"), dw.data_ptr(), _matrix(dw, "out"),
                                   _type(dw, "out"), None if work is None else work.data_ptr(), size, s))
    return dw


class LinearCrossEntropy(NamedTuple):
    loss: torch.Tensor          # [1]
    logps: torch.Tensor         # [rows]
    dh: torch.Tensor | None     # the gradients of grad_scale * loss
    dw: torch.Tensor | None


def _linear(h: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, temperature: float) -> _Linear:
    if h.dtype not in (torch.float16, torch.bfloat16) or w.dtype != h.dtype:
        raise TypeError(f"h and w must both be float16 or bfloat16, not {h.dtype} and {w.dtype}")
    ld_h, ld_w = _matrix(h, "h"), _matrix(w, "w")
    (rows, features), (vocab, other) = h.shape, w.shape
    if other != features:
        raise ValueError(f"h has {features} features and w {other}")
    if targets.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"targets must be int32 or int64, not {targets.dtype}")
    y = _vector(targets, rows, "targets", targets.dtype)
    return _Linear(h.data_ptr(), w.data_ptr(), y, rows, features, vocab, ld_h, ld_w, float(temperature), _TYPES[h.dtype],
                   targets.element_size())


def _wanted(want_dh: bool, want_dw: bool, dh, dw, add) -> None:
    """A buffer of a gradient that is not wanted would keep what it holds, unnoticed: refused."""
    for name, given, wanted, of in (("dh", dh, want_dh, "dh"), ("dw", dw, want_dw, "dw"), ("add", add, want_dw, "dw")):
        if given is not None and not wanted:
            raise ValueError(f"{name} is given, but {of} is not wanted")


def _linear_grads(h: torch.Tensor, w: torch.Tensor, want_dh: bool, want_dw: bool, dh: torch.Tensor | None,
                  dw: torch.Tensor | None, add: torch.Tensor | None, dw_dtype: torch.dtype | None):
    """(dh, dw, the call's argument, or None where no gradient is wanted)"""
    if not (want_dh or want_dw):
        return None, None, None
    dh = _output(dh, tuple(h.shape), h.dtype, "dh", h) if want_dh else None
    if want_dw:
        if dw_dtype is None:
            dw_dtype = dw.dtype if dw is not None else add.dtype if add is not None else w.dtype
        if add is not None and (add.shape != w.shape or add.dtype != dw_dtype):
            raise ValueError(f"add must be {dw_dtype} of shape {tuple(w.shape)}, not {add.dtype} of {tuple(add.shape)}")
        dw = _output(dw, tuple(w.shape), dw_dtype, "dw", w)
    g = _LinearGrads(None if dh is None else dh.data_ptr(), None if dw is None else dw.data_ptr(),
                     None if add is None else add.data_ptr(), 0 if dh is None else _matrix(dh, "dh"),
                     0 if dw is None else _matrix(dw, "dw"), 0 if add is None else _matrix(add, "add"),
                     0 if dw is None else _type(dw, "dw"), 0)
    return dh, dw, g


def mica_linear_logps(h: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, *, temperature: float = 1.0,
                      lse: bool = False, stream=None):
    """Log-probabilities of ``targets`` (int32 or int64, [rows]; negative: not scored, 0) under the softmax of
    ``h @ w.T / temperature``, float32 [rows], without storing the logits. ``h``: hidden states [rows, features], ``w``:
    the output embedding [vocabulary, features], both float16 or bfloat16, any row stride. With ``lse`` also the
    logarithms of the sums of exp of the logits, which mica_linear_logps_grad takes: ``(logps, lse)``."""
    l = _linear(h, w, targets, temperature)
    L = _train()
    with _On(stream, h.device) as s:
        logps = torch.empty(l.rows, dtype=torch.float32, device=h.device)
        z = torch.empty_like(logps) if lse else None
        size = L.mica_linear_logps_workspace(l)
        work = torch.empty(size, dtype=torch.uint8, device=h.device)
        _check(L.mica_linear_logps(l, logps.data_ptr(), None if z is None else z.data_ptr(), work.data_ptr(), size, s))
    return (logps, z) if lse else logps


def mica_linear_logps_grad(h: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                           dlogps: torch.Tensor, *, temperature: float = 1.0, want_dh: bool = True,
                           want_dw: bool = True, dh: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                           add: torch.Tensor | None = None, dw_dtype: torch.dtype | None = None, stream=None):
    """The gradients ``(dh, dw)`` of hidden states and embedding given that of mica_linear_logps's result, for any loss
    over log-probabilities. ``dh`` has h's dtype, ``dw`` ``dw_dtype`` (by default that of ``dw``, then of ``add``, then
    of w); ``dw`` is ``add`` plus the gradient, and ``add`` may be ``dw`` itself. ``want_dh`` and ``want_dw`` leave one
    out (None), whose buffers must then not be given."""
    _wanted(want_dh, want_dw, dh, dw, add)
    l = _linear(h, w, targets, temperature)
    z, d = _vector(lse, l.rows, "lse"), _vector(dlogps, l.rows, "dlogps")
    L = _train()
    with _On(stream, h.device) as s:
        dh, dw, g = _linear_grads(h, w, want_dh, want_dw, dh, dw, add, dw_dtype)
        if g is None:
            return None, None
        size = L.mica_linear_grad_workspace(l, g)
        work = torch.empty(size, dtype=torch.uint8, device=h.device)
        _check(L.mica_linear_logps_grad(l, z, d, g, work.data_ptr(), size, s))
    return dh, dw


def mica_linear_cross_entropy(h: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, *, denom: float | None = None,
                              temperature: float = 1.0, grad_scale: float = 1.0, grad: bool = True,
                              want_dh: bool = True, want_dw: bool = True, dh: torch.Tensor | None = None,
                              dw: torch.Tensor | None = None, add: torch.Tensor | None = None,
                              dw_dtype: torch.dtype | None = None, stream=None) -> LinearCrossEntropy:
    """Softmax cross entropy of ``targets`` under ``h @ w.T / temperature``, summed over the scored rows and divided by
    ``denom`` (None: their number), and the gradients of ``grad_scale`` times it, without storing the logits. The
    workspace holds their gradient in 16 bits, for as many rows at a time as 1 GB takes (at least 256). Arguments
    as mica_linear_logps and mica_linear_logps_grad; ``grad=False`` leaves both gradients out."""
    _wanted(grad and want_dh, grad and want_dw, dh, dw, add)
    l = _linear(h, w, targets, temperature)
    if denom is not None and not denom > 0.0:
        raise ValueError(f"denom must be > 0, not {denom}")
    hp = _CrossEntropyHP(0.0 if denom is None else float(denom), float(grad_scale))
    L = _train()
    with _On(stream, h.device) as s:
        loss = torch.empty(1, dtype=torch.float32, device=h.device)
        logps = torch.empty(l.rows, dtype=torch.float32, device=h.device)
        dh, dw, g = _linear_grads(h, w, grad and want_dh, grad and want_dw, dh, dw, add, dw_dtype)
        size = L.mica_linear_cross_entropy_workspace(l, g)
        work = torch.empty(size, dtype=torch.uint8, device=h.device)
        _check(L.mica_linear_cross_entropy(l, hp, loss.data_ptr(), logps.data_ptr(), g, work.data_ptr(), size, s))
    return LinearCrossEntropy(loss, logps, dh, dw)
