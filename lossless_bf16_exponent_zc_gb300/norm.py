"""The norms before and after a block, with the block's gate and residual scale, in one pass each way.

    h = norm.pre_norm(x, weight)                                       # before the first block
    x, h = norm.post_norm(block(h), x, weight, gate=gate, residual_scale=a, next_weight=next_weight)

post_norm closes one block and opens the next: x_new = a x + gate * rmsnorm(y) * weight, and h = rmsnorm(x_new) *
next_weight (None: no h).  A gate has one row for all tokens, or a row for each run of tokens / rows of them (a
sequence each, say), of hidden values or of one.  Argument marshalling only: the kernels are zc_norm and
zc_norm_backward (include/zc.h, where the operators are defined), on the current torch stream.  Activations are
bfloat16, float16 or float32 matrices whose rows may be strided; weights and gate share a type, the activations' or
float32.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import zc

MAX_HIDDEN = 16384


class PostNormGrads(NamedTuple):
    dy: torch.Tensor
    dx: torch.Tensor
    dweight: torch.Tensor
    dgate: torch.Tensor | None
    dnext_weight: torch.Tensor | None


@functools.lru_cache(maxsize=4096)
def workspace_size(tokens: int, hidden: int) -> int:
    out = ctypes.c_uint64()
    zc._check(zc.load().zc_norm_workspace_size(int(tokens), int(hidden), ctypes.byref(out)), "zc_norm_workspace_size")
    return out.value


def workspace(tokens: int, hidden: int, device="cuda") -> torch.Tensor:
    """A workspace for the gradients of up to so many tokens; calls that share it must be ordered on one stream."""
    return torch.empty(workspace_size(tokens, hidden), dtype=torch.uint8, device=device)


def _param(t: torch.Tensor, hidden: int, what: str) -> int:
    if t.shape != (hidden,):
        raise ValueError(f"{what} must have the activations' width ({hidden}), not {tuple(t.shape)}")
    return zc._ptr(t)


def _params(a, x: torch.Tensor, weight, gate, next_weight) -> None:
    """Fills in the parameters of a zc_norm_args or zc_norm_backward_args."""
    tokens, hidden = x.shape
    kind = None
    for t in (weight, gate, next_weight):
        if t is None:
            continue
        if kind is None:
            kind = t.dtype
        if t.dtype != kind or (kind != x.dtype and kind != torch.float32):
            raise ValueError("weights and gate must all have the activations' type, or all be float32")
    a.tokens, a.hidden, a.dtype = tokens, hidden, zc._dtype(x)
    a.params_f32 = kind == torch.float32 and x.dtype != torch.float32
    if weight is not None:
        a.weight = _param(weight, hidden, "weight")
    if next_weight is not None:
        a.next_weight = _param(next_weight, hidden, "next_weight")
    if gate is not None:
        if gate.dim() != 2 or gate.shape[1] not in (1, hidden) or gate.shape[0] < 1 or tokens % gate.shape[0]:
            raise ValueError("gate must be [rows, hidden] or [rows, 1] with rows a divisor of the tokens")
        a.gate, a.gate_rows, a.gate_wide = zc._ptr(gate), gate.shape[0], gate.shape[1] == hidden


def _same(t: torch.Tensor, x: torch.Tensor, what: str) -> tuple[int, int]:
    if t.shape != x.shape or t.dtype != x.dtype:
        raise ValueError(f"{what} must have the shape and type of the activations")
    return zc._rows(t, what)


def pre_norm(x: torch.Tensor, weight: torch.Tensor, *, eps: float = 1e-6, out: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """h = x / sqrt(mean(x^2) + eps) * weight over the rows of x [tokens, hidden]."""
    a = zc.NormArgs()
    a.x, a.x_stride = zc._rows(x, "x")
    _params(a, x, None, None, weight)
    out = zc._output(out, x.shape, x.dtype, x.device, "out")
    a.eps, a.h = eps, out.data_ptr()
    zc._check(zc.load().zc_norm(ctypes.byref(a), zc._stream(stream, x)), "zc_norm")
    return out


def post_norm(y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *, gate: torch.Tensor | None = None,
              residual_scale: float = 1.0, next_weight: torch.Tensor | None = None, eps: float = 1e-6,
              x_new: torch.Tensor | None = None, h: torch.Tensor | None = None,
              stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(x_new, h): the block's output y normed, gated and added to the scaled residual stream x, and the next
    block's input (None without next_weight).  x_new may be x itself when x is contiguous."""
    a = zc.NormArgs()
    a.y, a.y_stride = zc._rows(y, "y")
    a.x, a.x_stride = _same(x, y, "x")
    _params(a, y, weight, gate, next_weight)
    x_new = zc._output(x_new, y.shape, y.dtype, y.device, "x_new")
    if next_weight is not None:
        h = zc._output(h, y.shape, y.dtype, y.device, "h")
        a.h = h.data_ptr()
    else:
        h = None
    a.residual_scale, a.eps, a.x_new = residual_scale, eps, x_new.data_ptr()
    zc._check(zc.load().zc_norm(ctypes.byref(a), zc._stream(stream, y)), "zc_norm")
    return x_new, h


def _backward(a, dx_new, dh, y, x_new, like, weight, gate, next_weight, ws, stream):
    """Runs zc_norm_backward; (dy, dx, dweight, dgate, dnext_weight)."""
    if dx_new is not None:
        a.dx_new, a.dx_new_stride = _same(dx_new, like, "dx_new")
    if dh is not None:
        a.dh, a.dh_stride = _same(dh, like, "dh")
    if x_new is not None:
        a.x_new, a.x_new_stride = _same(x_new, like, "x_new")
    if y is not None:
        a.y, a.y_stride = zc._rows(y, "y")
    _params(a, like, weight, gate, next_weight)
    empty = torch.empty_like if like.shape[0] else torch.zeros_like
    dx = torch.empty(like.shape, dtype=like.dtype, device=like.device)
    dy = torch.empty_like(dx) if y is not None else None
    grads = [empty(p) if p is not None else None for p in (weight, gate, next_weight)]
    if like.shape[0] == 0:  # no tokens: nothing to launch, and the sums over none are zero
        return dy, dx, *grads
    a.dx = dx.data_ptr()
    if dy is not None:
        a.dy = dy.data_ptr()
    a.dweight, a.dgate, a.dnext_weight = (g.data_ptr() if g is not None else None for g in grads)
    a.ws, a.ws_bytes = zc._ptr(ws), ws.numel() * ws.element_size()
    zc._check(zc.load().zc_norm_backward(ctypes.byref(a), zc._stream(stream, like)), "zc_norm_backward")
    return dy, dx, *grads


def pre_norm_backward(dh: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, ws: torch.Tensor, *,
                      dresidual: torch.Tensor | None = None, eps: float = 1e-6,
                      stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight); dresidual, the gradient that reaches x past the block, is added to dx in the same pass."""
    a = zc.NormBackwardArgs()
    a.residual_scale, a.eps = 1.0, eps
    _, dx, _, _, dweight = _backward(a, dresidual, dh, None, x, x, None, None, weight, ws, stream)
    return dx, dweight


def post_norm_backward(dx_new: torch.Tensor | None, dh: torch.Tensor | None, y: torch.Tensor,
                       x_new: torch.Tensor | None, weight: torch.Tensor, ws: torch.Tensor, *,
                       gate: torch.Tensor | None = None, residual_scale: float = 1.0,
                       next_weight: torch.Tensor | None = None, eps: float = 1e-6, stream=None) -> PostNormGrads:
    """Gradients of post_norm from those of its outputs.  dx_new: what reaches x_new other than through h (None:
    nothing); dh and the saved x_new are given exactly when next_weight is."""
    if (dh is None) != (next_weight is None) or (dx_new is None and dh is None):
        raise ValueError("dh goes with next_weight, and one of dx_new and dh must be given")
    if next_weight is not None and x_new is None:
        raise ValueError("the gradient through h needs the saved x_new")
    a = zc.NormBackwardArgs()
    a.residual_scale, a.eps = residual_scale, eps
    return PostNormGrads(*_backward(a, dx_new, dh, y, x_new if next_weight is not None else None, y, weight, gate,
                                    next_weight, ws, stream))
