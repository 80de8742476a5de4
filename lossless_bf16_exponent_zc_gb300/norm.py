"""The norms before and after a block, with the block's gate and residual scale, in one pass each way.

    h = norm.pre_norm(x, weight)                                       # before the first block
    x, h = norm.post_norm(block(h), x, weight, gate=gate, residual_scale=a, next_weight=next_weight)

post_norm closes one block and opens the next: x_new = a x + gate * rmsnorm(y) * weight, and h = rmsnorm(x_new) *
next_weight (None: no h).  A gate has one row for all tokens, or a row for each run of tokens / rows of them (a
sequence each, say), of hidden values or of one.  The kernels are zc_norm and zc_norm_backward (include/zc.h, where the
operators are defined); arguments are checked, and outputs that are not given allocated, in the native extension
(csrc/zc_torch.cpp).  Activations are bfloat16, float16 or float32 matrices whose rows may be strided; weights and gate
share a type, the activations' or float32.

Calls run on the current torch stream, or on the one given as ``stream``.  On a given stream, what it reads and the
outputs it is handed must be ready there (``stream.wait_stream(...)``) and stay alive until it has run; outputs it makes
are that stream's, to be used elsewhere once that place waits for it.
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


def pre_norm(x: torch.Tensor, weight: torch.Tensor, *, eps: float = 1e-6, out: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """h = x / sqrt(mean(x^2) + eps) * weight over the rows of x [tokens, hidden]."""
    return zc.native().norm_forward(None, x, None, None, 1.0, weight, eps, None, out, stream)[1]


def post_norm(y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *, gate: torch.Tensor | None = None,
              residual_scale: float = 1.0, next_weight: torch.Tensor | None = None, eps: float = 1e-6,
              x_new: torch.Tensor | None = None, h: torch.Tensor | None = None,
              stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """(x_new, h): the block's output y normed, gated and added to the scaled residual stream x, and the next
    block's input (None without next_weight).  x_new may be x itself when x is contiguous."""
    return zc.native().norm_forward(y, x, weight, gate, residual_scale, next_weight, eps, x_new, h, stream)


def pre_norm_backward(dh: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, ws: torch.Tensor, *,
                      dresidual: torch.Tensor | None = None, eps: float = 1e-6,
                      stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight); dresidual, the gradient that reaches x past the block, is added to dx in the same pass."""
    _, dx, _, _, dweight = zc.native().norm_backward(dresidual, dh, None, x, None, None, 1.0, weight, eps, ws, stream)
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
    return PostNormGrads(*zc.native().norm_backward(dx_new, dh, y, x_new, weight, gate, residual_scale, next_weight, eps,
                                                    ws, stream))
