"""Dropout from a counter-based generator, with a mask that is never stored.

    rng = dropout.new_rng(seed)                                        # int64 [2] on the device: seed, offset
    x = dropout.dropout(block(h), 0.1, rng, call, residual=x)          # the block's output dropped out, the stream added
    ...
    dy = dropout.dropout_backward(dx, 0.1, rng, call)                  # draws the same mask again
    rng[1] += 1                                                        # the next step draws others

Which values stay follows from the generator's state, the call's number and each value's row and column alone
(zc_dropout in include/zc.h has the formula), so the gradient draws the mask again and nothing is kept.  `call` tells
apart the dropouts of one step, the offset the steps; both live as long as a step: its gradients need the state
that its forward calls read.  The state is read on the device, so a captured graph draws anew when it changes.
norm.add_layer_norm does the same in one pass with the next block's norm.

The kernel is zc_dropout; arguments are checked in the native extension (csrc/zc_torch.cpp).  Activations are bfloat16,
float16 or float32 matrices whose rows may be strided.  Calls run on the current torch stream, or on the one given as
``stream``.  On a given stream, what it reads and the outputs it is handed must be ready there
(``stream.wait_stream(...)``) and stay alive until it has run; outputs it makes are that stream's, to be used elsewhere
once that place waits for it.
"""
from __future__ import annotations

import torch

from . import zc


def new_rng(seed: int, offset: int = 0, device="cuda") -> torch.Tensor:
    """A generator's state: int64 [2], a seed of up to 63 bits and an offset (of which 32 bits are used)."""
    return torch.tensor([seed, offset], dtype=torch.int64, device=device)


def dropout(x: torch.Tensor, p: float, rng: torch.Tensor, call: int = 0, *, residual: torch.Tensor | None = None,
            residual_scale: float = 1.0, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """residual_scale * residual + dropout(x): a value of x, [rows, width], is kept and multiplied by 1 / (1 - p), p
    rounded to 2^-16, or becomes zero.  out may be x or residual itself where that is contiguous."""
    return zc.native().dropout(x, p, rng, call, residual, residual_scale, out, stream)[0]


def dropout_backward(dout: torch.Tensor, p: float, rng: torch.Tensor, call: int = 0, *,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of x: dout through the same mask.  (The residual's is residual_scale * dout.)"""
    return zc.native().dropout(dout, p, rng, call, None, 1.0, out, stream)[0]
