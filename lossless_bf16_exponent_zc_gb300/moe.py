"""Routing, dispatch and combine: what stands on both sides of an expert-parallel all-to-all.

    weights, experts = moe.route(logits, k)                      # top-k experts of every token
    rows, plan = moe.dispatch(x, experts, num_experts, ws)       # tokens sorted by expert: the pieces to exchange
    ... exchange.zipped_all_to_all, the experts, and back ...
    out = moe.combine(rows_back, weights, plan.positions, status)

and the gradients of all three (``torch.ops.zc.moe_*`` has them with autograd).  Argument marshalling only: every
step runs in libzc's kernels (zc_moe_* in include/zc.h, where the operators are defined) on the current torch
stream.  Activations are bfloat16, float16 or float32 matrices whose rows may be strided; weights are float32,
expert ids int32 (or int64, in dispatch).
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import zc

MAX_K = 32
MAX_EXPERTS = 1024

_SCORES = {"softmax": 0, "sigmoid": 1}


class DispatchPlan(NamedTuple):
    """Where dispatch put every slot (token * k + j) of the token-to-expert assignment."""

    positions: torch.Tensor  # int32 [tokens, k]: the slot's row, or -1 - row for a slot that is not routed
    slots: torch.Tensor      # int32 [tokens * k]: the slot of every row (the inverse)
    offsets: torch.Tensor    # int32 [experts + 1]: expert e has rows [offsets[e], offsets[e + 1])


def _score(score: str) -> int:
    code = _SCORES.get(score)
    if code is None:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    return code


def _table(t: torch.Tensor, shape: tuple, dtype: torch.dtype, what: str) -> int:
    """Device pointer of a contiguous table of the given shape and type."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} of shape {tuple(shape)}, not {t.dtype} {tuple(t.shape)}")
    return zc._ptr(t)


def route(logits: torch.Tensor, k: int, *, score: str = "softmax", bias: torch.Tensor | None = None,
          renormalize: bool = True, scale: float = 1.0, weights: torch.Tensor | None = None,
          experts: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """The k best experts of every token: (weights float32 [tokens, k], experts int32 [tokens, k]).

    logits: [tokens, experts].  score "softmax" chooses by logit; "sigmoid" by sigmoid + bias (float32 [experts]),
    the bias not entering the weight.  Ties go to the lowest expert; a logit of -inf is never chosen (expert -1,
    weight 0 where too few remain)."""
    ptr, stride = zc._rows(logits, "logits")
    tokens, n = logits.shape
    weights = zc._output(weights, (tokens, k), torch.float32, logits.device, "weights")
    experts = zc._output(experts, (tokens, k), torch.int32, logits.device, "experts")
    rc = zc.load().zc_moe_route(ptr, zc._dtype(logits), stride, tokens, n, k, _score(score),
                                _table(bias, (n,), torch.float32, "bias") if bias is not None else None,
                                renormalize, scale, weights.data_ptr(), experts.data_ptr(),
                                zc._stream(stream, logits))
    zc._check(rc, "zc_moe_route")
    return weights, experts


def route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, *, score: str = "softmax",
                   renormalize: bool = True, scale: float = 1.0, dlogits: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Gradient of the logits, in their type, from that of the weights; experts as route returned them."""
    ptr, stride = zc._rows(logits, "logits")
    tokens, n = logits.shape
    if experts.dim() != 2:
        raise ValueError("experts must be [tokens, k]")
    shape = (tokens, experts.shape[1])
    dlogits = zc._output(dlogits, (tokens, n), logits.dtype, logits.device, "dlogits")
    rc = zc.load().zc_moe_route_backward(_table(dweights, shape, torch.float32, "dweights"), ptr, zc._dtype(logits),
                                         stride, tokens, n, shape[1], _table(experts, shape, torch.int32, "experts"),
                                         _score(score), renormalize, scale, dlogits.data_ptr(),
                                         zc._stream(stream, logits))
    zc._check(rc, "zc_moe_route_backward")
    return dlogits


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
    ptr, stride = zc._rows(x, "x")
    tokens, hidden = x.shape
    if experts.dim() != 2 or experts.shape[0] != tokens or experts.dtype not in (torch.int32, torch.int64):
        raise ValueError("experts must be int32 or int64 [tokens, k]")
    k = experts.shape[1]
    dev = x.device
    rows = zc._output(rows, (tokens * k, hidden), x.dtype, dev, "rows")
    plan = DispatchPlan(torch.empty((tokens, k), dtype=torch.int32, device=dev),
                        torch.empty(tokens * k, dtype=torch.int32, device=dev),
                        torch.empty(num_experts + 1, dtype=torch.int32, device=dev))
    rc = zc.load().zc_moe_dispatch(ptr, zc._dtype(x), stride, tokens, hidden, zc._ptr(experts),
                                   experts.dtype == torch.int64, k, num_experts, rows.data_ptr(),
                                   plan.positions.data_ptr(), plan.slots.data_ptr(), plan.offsets.data_ptr(),
                                   zc._ptr(ws), ws.numel() * ws.element_size(), zc._stream(stream, x))
    zc._check(rc, "zc_moe_dispatch")
    return rows, plan


def _combine(rows, weights, positions, status, out, stream, where):
    ptr, stride = zc._rows(rows, "rows")
    if positions.dim() != 2 or positions.dtype != torch.int32:
        raise ValueError("positions must be int32 [tokens, k]")
    tokens, k = positions.shape
    hidden = rows.shape[1]
    out = zc._output(out, (tokens, hidden), rows.dtype, rows.device, "out")
    rc = zc.load().zc_moe_combine(ptr, zc._dtype(rows), stride, rows.shape[0],
                                  _table(weights, (tokens, k), torch.float32, "weights") if weights is not None
                                  else None, zc._ptr(positions), tokens, k, hidden, out.data_ptr(),
                                  _table(status, (1,), torch.int32, "status"), zc._stream(stream, rows))
    zc._check(rc, where)
    return out


def combine(rows: torch.Tensor, weights: torch.Tensor, positions: torch.Tensor, status: torch.Tensor, *,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[t] = sum over j of weights[t, j] * rows[positions[t, j]]: [tokens, hidden] in the rows' type.  Slots
    that are not routed add nothing; a position beyond the rows sets ERR_BAD_INDEX in status."""
    if weights is None:
        raise ValueError("combine takes weights (dispatch_backward adds without them)")
    return _combine(rows, weights, positions, status, out, stream, "zc_moe_combine")


def combine_backward(dout: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor, positions: torch.Tensor,
                     status: torch.Tensor, *, drows: torch.Tensor | None = None,
                     dweights: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(drows [rows, hidden], dweights float32 [tokens, k]).  Every row of a plan's rows is written (zero where the
    slot is not routed)."""
    ptr, stride = zc._rows(rows, "rows")
    dptr, dstride = zc._rows(dout, "dout")
    if positions.dim() != 2 or positions.dtype != torch.int32:
        raise ValueError("positions must be int32 [tokens, k]")
    tokens, k = positions.shape
    n_rows, hidden = rows.shape
    if dout.dtype != rows.dtype or dout.shape != (tokens, hidden):
        raise ValueError("dout must be [tokens, hidden] in the rows' type")
    drows = zc._output(drows, (n_rows, hidden), rows.dtype, rows.device, "drows")
    dweights = zc._output(dweights, (tokens, k), torch.float32, rows.device, "dweights")
    rc = zc.load().zc_moe_combine_backward(dptr, zc._dtype(rows), dstride, ptr, stride, n_rows,
                                           _table(weights, (tokens, k), torch.float32, "weights"),
                                           zc._ptr(positions), tokens, k, hidden, drows.data_ptr(),
                                           dweights.data_ptr(), _table(status, (1,), torch.int32, "status"),
                                           zc._stream(stream, rows))
    zc._check(rc, "zc_moe_combine_backward")
    return drows, dweights


def dispatch_backward(drows: torch.Tensor, positions: torch.Tensor, status: torch.Tensor, *,
                      dx: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of dispatch's x: every token gets the sum of its rows' gradients, added in the order of its slots."""
    return _combine(drows, None, positions, status, dx, stream, "zc_moe_combine")
