"""Routing, dispatch and combine: what stands on both sides of an expert-parallel all-to-all.

    weights, experts = moe.route(logits, k)                      # top-k experts of every token
    rows, plan = moe.dispatch(x, experts, num_experts, ws)       # tokens sorted by expert: the pieces to exchange
    ... exchange.zipped_all_to_all, the experts, and back ...
    out = moe.combine(rows_back, weights, plan.positions, status)

    b = moe.balance_loss(logits, experts, bws)                   # a loss that keeps the experts' load even, and their counts

and the gradients of all of them (``torch.ops.zc.moe_*`` has them with autograd).  Every step runs in libzc's kernels
(zc_moe_* in include/zc.h, where the operators are defined); arguments are checked, and outputs that are not given
allocated, in the native extension (csrc/zc_torch.cpp).  Activations are bfloat16, float16 or float32 matrices whose rows
may be strided; weights are float32, expert ids int32 (or int64, in dispatch).

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

MAX_K = 32
MAX_EXPERTS = 1024


class DispatchPlan(NamedTuple):
    """Where dispatch put every slot (token * k + j) of the token-to-expert assignment."""

    positions: torch.Tensor  # int32 [tokens, k]: the slot's row, or -1 - row for a slot that is not routed
    slots: torch.Tensor      # int32 [tokens * k]: the slot of every row (the inverse)
    offsets: torch.Tensor    # int32 [experts + 1]: expert e has rows [offsets[e], offsets[e + 1])


def route(logits: torch.Tensor, k: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
          renormalize: bool = True, scale: float = 1.0, weights: torch.Tensor | None = None,
          experts: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The k best experts of every token: (weights float32 [tokens, k], experts int32 [tokens, k]).

    logits: [tokens, experts].  score "softmax" chooses by logit; "sigmoid" by sigmoid + bias (float32 [experts]),
    the bias not entering the weight.  Ties go to the lowest expert; a logit of -inf is never chosen (expert -1,
    weight 0 where too few remain)."""
    return zc.native().moe_route(logits, k, score, bias, renormalize, scale, weights, experts, stream)


def route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, *, score: str = "softmax",
                   renormalize: bool = True, scale: float = 1.0, dlogits: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Gradient of the logits, in their type, from that of the weights; experts as route returned them."""
    return zc.native().moe_route_backward(dweights, logits, experts, score, renormalize, scale, dlogits, stream)[0]


@functools.lru_cache(maxsize=4096)
def workspace_size(tokens: int, k: int, num_experts: int) -> int:
    out = ctypes.c_uint64()
    zc._check(zc.load().zc_moe_workspace_size(int(tokens), int(k), int(num_experts), ctypes.byref(out)),
              "zc_moe_workspace_size")
    return out.value


def workspace(tokens: int, k: int, num_experts: int, device="cuda") -> torch.Tensor:
    """A workspace for dispatches of up to so many tokens; calls that share it must be ordered on one stream."""
    return torch.empty(workspace_size(tokens, k, num_experts), dtype=torch.uint8, device=device)


def dispatch(x: torch.Tensor, experts: torch.Tensor, num_experts: int, ws: torch.Tensor, *,
             rows: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, DispatchPlan]:
    """Tokens sorted by expert: (rows [tokens * k, hidden], plan).  experts: int32 or int64 [tokens, k]; a value
    outside [0, num_experts) is a slot that is not routed, whose row is zero and comes after all others."""
    rows, positions, slots, offsets = zc.native().moe_dispatch(x, experts, num_experts, ws, rows, stream)
    return rows, DispatchPlan(positions, slots, offsets)


def combine(rows: torch.Tensor, weights: torch.Tensor, positions: torch.Tensor, status: torch.Tensor, *,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = sum over j of weights[t, j] * rows[positions[t, j]]: [tokens, hidden] in the rows' type.  Slots
    that are not routed add nothing; a position beyond the rows sets ERR_BAD_INDEX in status."""
    if weights is None:
        raise ValueError("combine takes weights (dispatch_backward adds without them)")
    return zc.native().moe_combine(rows, weights, positions, status, out, stream)[0]


def combine_backward(dout: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor, positions: torch.Tensor,
                     status: torch.Tensor, *, drows: torch.Tensor | None = None,
                     dweights: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(drows [rows, hidden], dweights float32 [tokens, k]).  Every row of a plan's rows is written (zero where the
    slot is not routed)."""
    return zc.native().moe_combine_backward(dout, rows, weights, positions, status, drows, dweights, stream)


def dispatch_backward(drows: torch.Tensor, positions: torch.Tensor, status: torch.Tensor, *,
                      dx: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of dispatch's x: every token gets the sum of its rows' gradients, added in the order of its slots."""
    return zc.native().moe_combine(drows, None, positions, status, dx, stream)[0]


class BalanceLoss(NamedTuple):
    """What balance_loss gives."""

    loss: torch.Tensor    # float32, one value
    counts: torch.Tensor  # int32 [sequences, experts]: slots of every expert, of the tokens that count
    slope: torch.Tensor   # float32 [sequences, experts]: the loss's derivative by the sums of p; the gradient needs it


@functools.lru_cache(maxsize=4096)
def balance_workspace_size(tokens: int, num_experts: int, sequences: int = 1) -> int:
    out = ctypes.c_uint64()
    zc._check(zc.load().zc_moe_balance_workspace_size(int(tokens), int(num_experts), int(sequences), ctypes.byref(out)),
              "zc_moe_balance_workspace_size")
    return out.value


def balance_workspace(tokens: int, num_experts: int, sequences: int = 1, device="cuda") -> torch.Tensor:
    """A workspace for the balance loss of up to so many tokens in up to so many sequences; calls that share it must be
    ordered on one stream."""
    return torch.empty(balance_workspace_size(tokens, num_experts, sequences), dtype=torch.uint8, device=device)


def balance_loss(logits: torch.Tensor, experts: torch.Tensor, ws: torch.Tensor, *, score: str = "softmax",
                 sequences: int = 1, mask: torch.Tensor | None = None, stream=None) -> BalanceLoss:
    """The loss that keeps the experts' load even: the mean over the sequences (equal runs of the tokens) of num_experts *
    sum over the experts of (fraction of the slots) * (mean probability), which is 1 for an even load.

    logits: [tokens, experts]; experts: int32 [tokens, k], as route returned them (-1: none).  p is the softmax of the
    logits, or with score "sigmoid" the sigmoids over their sum.  mask: bool or uint8 [tokens], the tokens that count
    (None: all); a token whose logits are all -inf does not.  The counts of the experts (their sums move route's bias)
    have no gradient."""
    return BalanceLoss(*zc.native().moe_balance(logits, experts, ws, score, sequences, mask, stream))


def balance_loss_backward(dloss: torch.Tensor, logits: torch.Tensor, slope: torch.Tensor, *, score: str = "softmax",
                          mask: torch.Tensor | None = None, dlogits: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """Gradient of the logits, in their type, from that of the loss (float32, one value on the device)."""
    return zc.native().moe_balance_backward(dloss, logits, slope, score, mask, dlogits, stream)[0]
