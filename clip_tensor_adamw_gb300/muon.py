"""Python binding of include/mica_muon.h, taking torch tensors: lists of matrices orthogonalised by Newton-Schulz products,
and the optimizer step that takes its update from them.

As in mica.py, this module only marshals arguments; there is no fallback. The workspace of a call is allocated on the stream
that it runs on (``stream``, by default the current one).
"""
from __future__ import annotations

import ctypes

import torch

from .mica import (MICA_F16, MICA_F32, MICA_STEP_SKIP_NONFINITE, TensorList, _as_list, _check, _dtype_code, _ptr, _weights,
                   lib)
from .train import _On, _TYPES

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
_ADJUST = {"none": 0, "original": 1, "match_rms_adamw": 2}
_P, _I32, _I64, _F64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double


class _NewtonSchulz(ctypes.Structure):
    _fields_ = [("coefficients", ctypes.POINTER(_F64)), ("eps", _F64), ("steps", _I32), ("flags", ctypes.c_uint32)]


class _MuonHP(ctypes.Structure):
    _fields_ = [("lr", _F64), ("momentum", _F64), ("weight_decay", _F64), ("nesterov", _I32), ("adjust", _I32),
                ("zero_grad", _I32), ("flags", ctypes.c_uint32)]


_lib = None


def _muon() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = lib()
        array, sizes, ns = ctypes.POINTER(_P), ctypes.POINTER(_I64), ctypes.POINTER(_NewtonSchulz)
        for name, args, result in (
                ("mica_newton_schulz_workspace", [sizes, sizes, _I32, ctypes.c_uint32], _I64),
                ("mica_orthogonalize", [array, array, sizes, sizes, _I32, _I32, _I32, ns, _P, _I64, _P], ctypes.c_int),
                ("mica_muon_steps", [array, array, array, sizes, sizes, _I32, _I32, ctypes.POINTER(_MuonHP), ns, _P, _P,
                                     _I64, _P], ctypes.c_int)):
            getattr(L, name).argtypes = args
            getattr(L, name).restype = result
        _lib = L
    return _lib


def _sizes(L: TensorList, what: str, precise: bool):
    """The rows and columns of a list's matrices, and the workspace that they take (kept with the list)."""
    kept = L.__dict__.setdefault("matrices", {})
    if precise not in kept:
        for i, t in enumerate(L.tensors):
            if t.ndim != 2:
                raise ValueError(f"{what}[{i}] must have two dimensions, not {t.ndim}")
        rows, cols = ((ctypes.c_int64 * max(L.T, 1))(*(t.shape[d] for t in L.tensors)) for d in (0, 1))
        kept[precise] = rows, cols, _muon().mica_newton_schulz_workspace(rows, cols, L.T, int(precise))
    return kept[precise]


def _iteration(steps: int, coefficients, eps: float, precise: bool) -> _NewtonSchulz:
    rows = list(coefficients)
    if not rows or steps < 1:
        raise ValueError("at least one step is needed")
    if not hasattr(rows[0], "__len__"):
        rows = [rows] * steps
    if len(rows) != steps or any(len(r) != 3 for r in rows):
        raise ValueError("coefficients must be (a, b, c), or one such triple for each step")
    flat = [float(v) for r in rows for v in r]
    return _NewtonSchulz((_F64 * max(len(flat), 1))(*flat), float(eps), int(steps), int(precise))


def _same(A: TensorList, B: TensorList, names: str) -> None:
    if A.T != B.T or any(a.shape != b.shape for a, b in zip(A.tensors, B.tensors)):
        raise ValueError(f"{names} must list matrices of the same shapes")


def mica_orthogonalize(x, out=None, *, steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7,
                       precise: bool = False, out_dtype: torch.dtype | None = None, stream=None) -> TensorList:
    """Each matrix of ``x`` (float32, float16 or bfloat16, contiguous) taken by ``steps`` Newton-Schulz products towards
    the nearest one with orthogonal rows or columns, in one go for the whole list: the direction of a Muon update.
    ``coefficients``: (a, b, c) of the polynomial a t + b t^3 + c t^5 that each singular value goes through in a step, or
    one such triple for each step. ``precise`` holds what is stored between the products in pairs of float16 (three times
    the work), as matrices whose smaller side is at most 256 always are. ``out`` takes the results (float16 or bfloat16; it
    may be ``x`` itself); otherwise they are new matrices of ``out_dtype`` (by default x's, or bfloat16 for float32).
    Returns the list of results. The same list gives the same bits; beside other matrices one's may differ in the last places
    of its sums, which are split where the list is small."""
    X = _as_list(x)
    if out is not None:
        out = _as_list(out)
        if out_dtype is not None and out.T and out.dtype != out_dtype:
            raise TypeError(f"out_dtype is {out_dtype}, but out is {out.dtype}")
    rows, cols, size = _sizes(X, "x", precise)
    ns = _iteration(steps, coefficients, eps, precise)
    code = _TYPES.get(X.dtype, 0 if X.dtype is None else None)
    if code is None:
        raise TypeError(f"x: unsupported dtype {X.dtype}")
    dev = X.tensors[0].device if X.T else torch.device("cuda", torch.cuda.current_device())
    with _On(stream, dev) as s:
        if out is None:
            if out_dtype is None:
                out_dtype = X.dtype if X.dtype in (torch.float16, torch.bfloat16) else torch.bfloat16
            out = [torch.empty_like(t, dtype=out_dtype) for t in X.tensors]
        O = _as_list(out)
        _same(X, O, "x and out")
        if O.T and O.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError(f"out must be float16 or bfloat16, not {O.dtype}")
        work = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        _check(_muon().mica_orthogonalize(X.ptrs, O.ptrs, rows, cols, X.T, code, _TYPES.get(O.dtype, 1), ns, _ptr(work),
                                          size, s))
    return O


def mica_muon_steps(w, g, m, *, lr: float, momentum: float = 0.95, weight_decay: float = 0.0, nesterov: bool = True,
                    adjust: str = "original", factor: torch.Tensor | None = None, zero_grad: bool = False,
                    skip_nonfinite: bool = False, steps: int = 5, coefficients=COEFFICIENTS, eps: float = 1e-7,
                    precise: bool = False, stream=None) -> None:
    """One Muon step over a list of weight matrices, in place: m += (1 - momentum) (factor g - m), u the Nesterov blend of
    both (or m), w = w (1 - lr weight_decay) - lr adjust(w) orthogonalised(u). ``w`` and ``m``: float32, ``g``: float32 or
    float16; ``factor``: the device scalar from mica_clip_grad_norms (None: 1). ``adjust``: what a matrix's rate is
    multiplied by: "original" sqrt(max(1, rows / cols)), "match_rms_adamw" 0.2 sqrt(max(rows, cols)), or "none".
    ``skip_nonfinite`` leaves w and m as they are when the factor is not > 0. The rest as mica_orthogonalize."""
    W, G, M = _as_list(w), _as_list(g), _as_list(m)
    _weights(W)
    if M.dtype is not None and M.dtype != torch.float32:
        raise TypeError(f"m must be float32, not {M.dtype}")
    _same(W, G, "w and g")
    _same(W, M, "w and m")
    if factor is not None and (factor.dtype != torch.float32 or factor.numel() != 1):
        raise ValueError("factor must be one float32 on the device")
    if adjust not in _ADJUST:
        raise ValueError(f"adjust {adjust!r} is none of {sorted(_ADJUST)}")
    rows, cols, size = _sizes(W, "w", precise)
    gdt = _dtype_code(G, "g")
    if gdt not in (MICA_F32, MICA_F16):
        raise TypeError(f"g: unsupported dtype {G.dtype}")
    hp = _MuonHP(float(lr), float(momentum), float(weight_decay), int(bool(nesterov)), _ADJUST[adjust], int(bool(zero_grad)),
                 MICA_STEP_SKIP_NONFINITE if skip_nonfinite else 0)
    ns = _iteration(steps, coefficients, eps, precise)
    dev = W.tensors[0].device if W.T else torch.device("cuda", torch.cuda.current_device())
    with _On(stream, dev) as s:
        work = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
        _check(_muon().mica_muon_steps(W.ptrs, G.ptrs, M.ptrs, rows, cols, W.T, gdt, hp, ns, _ptr(factor), _ptr(work), size,
                                       s))
