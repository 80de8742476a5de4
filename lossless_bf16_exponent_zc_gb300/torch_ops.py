"""PyTorch operators over libzc: ``torch.ops.zc.*``.

The codec as ordinary torch operators, so that training code and frameworks can
call it like any other op (the drop-in integration of [ZipCCL §3] and
[CCCL §4]) and graph tracers see it: each op has a fake implementation that
gives its outputs' shapes and dtypes without running it.  Every op calls the
C ABI through the binding in ``zc.py`` on the current stream; there is no CPU
path.

Ops (device tensors; bf16 data as bfloat16 / int16 / uint16):
  zc::compress(x, cb, ws, status, adaptive=False) -> (main, esc)
      main: zc_main_bytes(n) uint8; esc: the escape buffer (capacity n, or
      the RAW spill when adaptive); the escape count is in main's header.
  zc::decompress(main, esc, n, status) -> int16[n]
  zc::decompress_reduce(mains, escs, n, status) -> int16[n]
      the local stage of a zipped reduce-scatter (no re-encode).
  zc::pipelined_transfer(x, cb, chunk_elems, ws, status) -> int16[n]
      the chunked compress / link / decompress pipeline on three streams.
  zc::zq_compress(x, widths, sym, ws, status) -> uint8[zq_max_bytes(n)]
      Quad Length Codes of 1-byte symbols (uint8 / float8 e4m3), the table
      given as its 8 region widths and 256-entry rank -> symbol list.
  zc::zq_decompress(stream, n, status) -> uint8[n]
``ws`` and ``status`` are mutated (the workspace protocol and the device
status word), and declared so.

The operators around an expert-parallel exchange (moe.py, norm.py), with
autograd; they bring their own workspace, and what the device has to report is
an output (int32[1], 0 = no error), since an op with a gradient must not
mutate its inputs:
  zc::moe_route(logits, bias, k, score, renormalize, scale) -> (weights, experts)
  zc::moe_dispatch(x, experts, num_experts) -> (rows, positions, slots, offsets)
  zc::moe_combine(rows, weights, positions) -> (out, status)
  zc::pre_norm(x, weight, eps) -> h
  zc::post_norm(y, x, weight, gate, residual_scale, eps) -> x_new
  zc::post_pre_norm(y, x, weight, gate, next_weight, residual_scale, eps) -> (x_new, h)
and those of the training step around it (moe.py, norm.py, dropout.py, embedding.py), likewise; a dropout's generator
state must not change between a call and its gradient (autograd notices):
  zc::moe_balance_loss(logits, experts, mask, score, sequences) -> (loss, counts, slope)
  zc::dropout(x, rng, residual, p, call, residual_scale) -> out
  zc::layer_norm(x, weight, bias, eps) -> (h, stats)
  zc::add_layer_norm(y, x, weight, bias, rng, p, call, residual_scale, eps) -> (x_new, h, stats)
  zc::embedding(ids, table, scale, dtype) -> (rows, status)
"""
from __future__ import annotations

import ctypes

import torch

from . import dropout, embedding, moe, norm, zc


@torch.library.custom_op("zc::compress", mutates_args=("ws", "status"))
def compress(x: torch.Tensor, cb: torch.Tensor, ws: torch.Tensor, status: torch.Tensor,
             adaptive: bool = False) -> tuple[torch.Tensor, torch.Tensor]:
    fn = zc.compress_adaptive if adaptive else zc.compress
    return fn(x.contiguous(), cb, ws, status)


@compress.register_fake
def _(x, cb, ws, status, adaptive=False):
    n = x.numel()
    main_bytes, max_esc = zc.compressed_size(n)  # host-side size law of the library
    esc = max(zc.raw_spill(n) if adaptive else max_esc, 16)
    return x.new_empty(main_bytes, dtype=torch.uint8), x.new_empty(esc, dtype=torch.uint8)


@torch.library.custom_op("zc::decompress", mutates_args=("status",))
def decompress(main: torch.Tensor, esc: torch.Tensor, n: int, status: torch.Tensor) -> torch.Tensor:
    return zc.decompress(main, esc, n, status)


@decompress.register_fake
def _(main, esc, n, status):
    return main.new_empty(n, dtype=torch.int16)


@torch.library.custom_op("zc::decompress_reduce", mutates_args=("status",))
def decompress_reduce(mains: list[torch.Tensor], escs: list[torch.Tensor], n: int,
                      status: torch.Tensor) -> torch.Tensor:
    out, _, _ = zc.decompress_reduce(list(mains), list(escs), n, status)
    return out


@decompress_reduce.register_fake
def _(mains, escs, n, status):
    return mains[0].new_empty(n, dtype=torch.int16)


@torch.library.custom_op("zc::pipelined_transfer", mutates_args=("ws", "status"))
def pipelined_transfer(x: torch.Tensor, cb: torch.Tensor, chunk_elems: int, ws: torch.Tensor,
                       status: torch.Tensor) -> torch.Tensor:
    return zc.pipelined_transfer(x.contiguous(), cb, chunk_elems, ws, status)


@pipelined_transfer.register_fake
def _(x, cb, chunk_elems, ws, status):
    return x.new_empty(x.numel(), dtype=torch.int16)


@torch.library.custom_op("zc::zq_compress", mutates_args=("ws", "status"))
def zq_compress(x: torch.Tensor, widths: list[int], sym: list[int], ws: torch.Tensor,
                status: torch.Tensor) -> torch.Tensor:
    return zc.zq_compress(x.contiguous(), zc.zq_table(widths, sym), ws, status)


@zq_compress.register_fake
def _(x, widths, sym, ws, status):
    return x.new_empty(zc.zq_max_bytes(x.numel()), dtype=torch.uint8)


@torch.library.custom_op("zc::zq_decompress", mutates_args=("status",))
def zq_decompress(stream: torch.Tensor, n: int, status: torch.Tensor) -> torch.Tensor:
    return zc.zq_decompress(stream, n, status)


@zq_decompress.register_fake
def _(stream, n, status):
    return stream.new_empty(n, dtype=torch.uint8)


# ------------------------------------------------------------------ routing, dispatch, combine
def _dense(t: torch.Tensor | None) -> torch.Tensor | None:
    """A gradient as the kernels read it: rows of contiguous columns."""
    return t if t is None or (t.dim() == 2 and t.stride(1) == 1) else t.contiguous()


@torch.library.custom_op("zc::moe_route", mutates_args=())
def moe_route(logits: torch.Tensor, bias: torch.Tensor | None, k: int, score: str, renormalize: bool,
              scale: float) -> tuple[torch.Tensor, torch.Tensor]:
    return moe.route(logits, k, score=score, bias=bias, renormalize=renormalize, scale=scale)


@moe_route.register_fake
def _(logits, bias, k, score, renormalize, scale):
    shape = (logits.shape[0], k)
    return logits.new_empty(shape, dtype=torch.float32), logits.new_empty(shape, dtype=torch.int32)


@torch.library.custom_op("zc::moe_route_backward", mutates_args=())
def moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, score: str,
                       renormalize: bool, scale: float) -> torch.Tensor:
    return moe.route_backward(dweights.contiguous(), logits, experts, score=score, renormalize=renormalize,
                              scale=scale)


@moe_route_backward.register_fake
def _(dweights, logits, experts, score, renormalize, scale):
    return logits.new_empty(logits.shape)


def _route_context(ctx, inputs, output):
    logits, _, _, ctx.score, ctx.renormalize, ctx.scale = inputs
    ctx.save_for_backward(logits, output[1])
    ctx.mark_non_differentiable(output[1])


def _route_backward(ctx, dweights, _):
    logits, experts = ctx.saved_tensors
    d = moe_route_backward(dweights, logits, experts, ctx.score, ctx.renormalize, ctx.scale)
    return d, None, None, None, None, None  # the bias only chooses


moe_route.register_autograd(_route_backward, setup_context=_route_context)


@torch.library.custom_op("zc::moe_dispatch", mutates_args=())
def moe_dispatch(x: torch.Tensor, experts: torch.Tensor,
                 num_experts: int) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    ws = moe.workspace(x.shape[0], experts.shape[1], num_experts, device=x.device)
    rows, plan = moe.dispatch(x, experts, num_experts, ws)
    return rows, *plan


@moe_dispatch.register_fake
def _(x, experts, num_experts):
    tokens, k = experts.shape
    i32 = dict(dtype=torch.int32)
    return (x.new_empty((tokens * k, x.shape[1])), x.new_empty((tokens, k), **i32), x.new_empty(tokens * k, **i32),
            x.new_empty(num_experts + 1, **i32))


@torch.library.custom_op("zc::moe_dispatch_backward", mutates_args=())
def moe_dispatch_backward(drows: torch.Tensor, positions: torch.Tensor) -> torch.Tensor:
    return moe.dispatch_backward(drows, positions, zc.new_status(drows.device))


@moe_dispatch_backward.register_fake
def _(drows, positions):
    return drows.new_empty((positions.shape[0], drows.shape[1]))


def _dispatch_context(ctx, inputs, output):
    ctx.save_for_backward(output[1])
    ctx.mark_non_differentiable(*output[1:])


def _dispatch_backward(ctx, drows, *_):
    return moe_dispatch_backward(_dense(drows), *ctx.saved_tensors), None, None


moe_dispatch.register_autograd(_dispatch_backward, setup_context=_dispatch_context)


@torch.library.custom_op("zc::moe_combine", mutates_args=())
def moe_combine(rows: torch.Tensor, weights: torch.Tensor,
                positions: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    status = zc.new_status(rows.device)
    return moe.combine(rows, weights, positions, status), status


@moe_combine.register_fake
def _(rows, weights, positions):
    return rows.new_empty((positions.shape[0], rows.shape[1])), rows.new_empty(1, dtype=torch.int32)


@torch.library.custom_op("zc::moe_combine_backward", mutates_args=())
def moe_combine_backward(dout: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor,
                         positions: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    # rows that no slot names have no gradient, and the kernel does not write them
    drows = None if rows.shape[0] == positions.numel() else torch.zeros_like(rows, memory_format=torch.contiguous_format)
    return moe.combine_backward(dout, rows, weights, positions, zc.new_status(rows.device), drows=drows)


@moe_combine_backward.register_fake
def _(dout, rows, weights, positions):
    return rows.new_empty(rows.shape), weights.new_empty(weights.shape)


def _combine_context(ctx, inputs, output):
    ctx.save_for_backward(*inputs)
    ctx.mark_non_differentiable(output[1])


def _combine_backward(ctx, dout, _):
    return *moe_combine_backward(_dense(dout), *ctx.saved_tensors), None


moe_combine.register_autograd(_combine_backward, setup_context=_combine_context)


# ------------------------------------------------------------------ the norms around a block
@torch.library.custom_op("zc::pre_norm", mutates_args=())
def pre_norm(x: torch.Tensor, weight: torch.Tensor, eps: float) -> torch.Tensor:
    return norm.pre_norm(x, weight, eps=eps)


@pre_norm.register_fake
def _(x, weight, eps):
    return x.new_empty(x.shape)


@torch.library.custom_op("zc::pre_norm_backward", mutates_args=())
def pre_norm_backward(dh: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                      eps: float) -> tuple[torch.Tensor, torch.Tensor]:
    return norm.pre_norm_backward(dh, x, weight, norm.workspace(*x.shape, device=x.device), eps=eps)


@pre_norm_backward.register_fake
def _(dh, x, weight, eps):
    return x.new_empty(x.shape), weight.new_empty(weight.shape)


def _pre_context(ctx, inputs, output):
    x, weight, ctx.eps = inputs
    ctx.save_for_backward(x, weight)


def _pre_backward(ctx, dh):
    return *pre_norm_backward(_dense(dh), *ctx.saved_tensors, ctx.eps), None


pre_norm.register_autograd(_pre_backward, setup_context=_pre_context)


@torch.library.custom_op("zc::post_norm", mutates_args=())
def post_norm(y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, gate: torch.Tensor | None,
              residual_scale: float, eps: float) -> torch.Tensor:
    return norm.post_norm(y, x, weight, gate=gate, residual_scale=residual_scale, eps=eps)[0]


@post_norm.register_fake
def _(y, x, weight, gate, residual_scale, eps):
    return y.new_empty(y.shape)


@torch.library.custom_op("zc::post_pre_norm", mutates_args=())
def post_pre_norm(y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, gate: torch.Tensor | None,
                  next_weight: torch.Tensor, residual_scale: float, eps: float) -> tuple[torch.Tensor, torch.Tensor]:
    return norm.post_norm(y, x, weight, gate=gate, residual_scale=residual_scale, next_weight=next_weight, eps=eps)


@post_pre_norm.register_fake
def _(y, x, weight, gate, next_weight, residual_scale, eps):
    return y.new_empty(y.shape), y.new_empty(y.shape)


@torch.library.custom_op("zc::post_norm_backward", mutates_args=())
def post_norm_backward(dx_new: torch.Tensor | None, dh: torch.Tensor | None, y: torch.Tensor,
                       x_new: torch.Tensor | None, weight: torch.Tensor, gate: torch.Tensor | None,
                       next_weight: torch.Tensor | None, residual_scale: float, eps: float) -> list[torch.Tensor]:
    """[dy, dx, dweight], then dgate and dnext_weight where there are such inputs."""
    g = norm.post_norm_backward(dx_new, dh, y, x_new, weight, norm.workspace(*y.shape, device=y.device), gate=gate,
                                residual_scale=residual_scale, next_weight=next_weight, eps=eps)
    return [t for t in g if t is not None]


@post_norm_backward.register_fake
def _(dx_new, dh, y, x_new, weight, gate, next_weight, residual_scale, eps):
    return [t.new_empty(t.shape) for t in (y, y, weight, gate, next_weight) if t is not None]


def _post_context(ctx, inputs, output):
    y, _, weight, gate, ctx.residual_scale, ctx.eps = inputs
    ctx.save_for_backward(y, weight, gate)


def _post_backward(ctx, dx_new):
    y, weight, gate = ctx.saved_tensors
    dy, dx, dw, *dgate = post_norm_backward(_dense(dx_new), None, y, None, weight, gate, None, ctx.residual_scale,
                                            ctx.eps)
    return dy, dx, dw, dgate[0] if dgate else None, None, None


post_norm.register_autograd(_post_backward, setup_context=_post_context)


def _post_pre_context(ctx, inputs, output):
    y, _, weight, gate, next_weight, ctx.residual_scale, ctx.eps = inputs
    ctx.save_for_backward(y, output[0], weight, gate, next_weight)
    ctx.set_materialize_grads(False)


def _post_pre_backward(ctx, dx_new, dh):
    y, x_new, weight, gate, next_weight = ctx.saved_tensors
    if dx_new is None and dh is None:
        return (None,) * 7
    if dh is None:  # nothing came through the next block
        dy, dx, dw, *dgate = post_norm_backward(_dense(dx_new), None, y, None, weight, gate, None, ctx.residual_scale,
                                                ctx.eps)
        return dy, dx, dw, dgate[0] if dgate else None, None, None, None
    dy, dx, dw, *rest = post_norm_backward(_dense(dx_new), _dense(dh), y, x_new, weight, gate, next_weight,
                                           ctx.residual_scale, ctx.eps)
    return dy, dx, dw, rest[0] if gate is not None else None, rest[-1], None, None


post_pre_norm.register_autograd(_post_pre_backward, setup_context=_post_pre_context)


# ------------------------------------------------------------------ balance loss
@torch.library.custom_op("zc::moe_balance_loss", mutates_args=())
def moe_balance_loss(logits: torch.Tensor, experts: torch.Tensor, mask: torch.Tensor | None, score: str,
                     sequences: int) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    ws = moe.balance_workspace(*logits.shape, sequences, device=logits.device)
    return tuple(moe.balance_loss(logits, experts, ws, score=score, sequences=sequences, mask=mask))


@moe_balance_loss.register_fake
def _(logits, experts, mask, score, sequences):
    shape = (sequences, logits.shape[1])
    f32 = dict(dtype=torch.float32)
    return logits.new_empty((), **f32), logits.new_empty(shape, dtype=torch.int32), logits.new_empty(shape, **f32)


@torch.library.custom_op("zc::moe_balance_loss_backward", mutates_args=())
def moe_balance_loss_backward(dloss: torch.Tensor, logits: torch.Tensor, slope: torch.Tensor,
                              mask: torch.Tensor | None, score: str) -> torch.Tensor:
    return moe.balance_loss_backward(dloss, logits, slope, score=score, mask=mask)


@moe_balance_loss_backward.register_fake
def _(dloss, logits, slope, mask, score):
    return logits.new_empty(logits.shape)


def _balance_context(ctx, inputs, output):
    logits, _, mask, ctx.score, _ = inputs
    ctx.save_for_backward(logits, output[2], mask)
    ctx.mark_non_differentiable(*output[1:])


def _balance_backward(ctx, dloss, *_):
    return moe_balance_loss_backward(dloss, *ctx.saved_tensors, ctx.score), None, None, None, None


moe_balance_loss.register_autograd(_balance_backward, setup_context=_balance_context)


# ------------------------------------------------------------------ dropout
@torch.library.custom_op("zc::dropout", mutates_args=())
def dropout_op(x: torch.Tensor, rng: torch.Tensor, residual: torch.Tensor | None, p: float, call: int,
               residual_scale: float) -> torch.Tensor:
    return dropout.dropout(x, p, rng, call, residual=residual, residual_scale=residual_scale)


@dropout_op.register_fake
def _(x, rng, residual, p, call, residual_scale):
    return x.new_empty(x.shape)


def _dropout_context(ctx, inputs, output):
    _, rng, residual, ctx.p, ctx.call, ctx.residual_scale = inputs
    ctx.residual = residual is not None
    ctx.save_for_backward(rng)  # a state that moved on before the gradient is an error


def _dropout_backward(ctx, dout):
    rng, = ctx.saved_tensors
    dresidual = None
    if ctx.residual:
        dresidual = dout if ctx.residual_scale == 1.0 else dout * ctx.residual_scale
    return dropout_op(_dense(dout), rng, None, ctx.p, ctx.call, 1.0), None, dresidual, None, None, None


dropout_op.register_autograd(_dropout_backward, setup_context=_dropout_context)


# ------------------------------------------------------------------ layer norms
@torch.library.custom_op("zc::layer_norm", mutates_args=())
def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None,
               eps: float) -> tuple[torch.Tensor, torch.Tensor]:
    return norm.layer_norm(x, weight, bias, eps=eps, save=True)


@layer_norm.register_fake
def _(x, weight, bias, eps):
    return x.new_empty(x.shape), x.new_empty((x.shape[0], 2), dtype=torch.float32)


@torch.library.custom_op("zc::add_layer_norm", mutates_args=())
def add_layer_norm(y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None,
                   rng: torch.Tensor | None, p: float, call: int, residual_scale: float,
                   eps: float) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    return norm.add_layer_norm(y, x, weight, bias, p=p, rng=rng, call=call, residual_scale=residual_scale, eps=eps,
                               save=True)


@add_layer_norm.register_fake
def _(y, x, weight, bias, rng, p, call, residual_scale, eps):
    return x.new_empty(x.shape), x.new_empty(x.shape), x.new_empty((x.shape[0], 2), dtype=torch.float32)


@torch.library.custom_op("zc::layer_norm_backward", mutates_args=())
def layer_norm_backward(dx_new: torch.Tensor | None, dh: torch.Tensor, x_new: torch.Tensor, stats: torch.Tensor,
                        weight: torch.Tensor, bias: bool, rng: torch.Tensor | None, p: float, call: int,
                        residual_scale: float) -> list[torch.Tensor]:
    """[dx, dweight], then dy where it is not dx, and dbias where there is one."""
    ws = norm.workspace(*x_new.shape, device=x_new.device)
    g = norm.add_layer_norm_backward(dx_new, dh, x_new, stats, weight, ws, bias=bias, p=p, rng=rng, call=call,
                                     residual_scale=residual_scale)
    return [t for t in (g.dx, g.dweight, g.dy if g.dy is not g.dx else None, g.dbias) if t is not None]


def _own_dy(p, residual_scale):
    return p > 0 or ctypes.c_float(residual_scale).value != 1.0  # the extension's rule: of the scale that the kernel gets


@layer_norm_backward.register_fake
def _(dx_new, dh, x_new, stats, weight, bias, rng, p, call, residual_scale):
    like = [x_new, weight] + [x_new] * _own_dy(p, residual_scale) + [weight] * bias
    return [t.new_empty(t.shape) for t in like]


def _layer_context(ctx, inputs, output):
    x, weight, bias, _ = inputs
    ctx.bias = bias is not None
    ctx.save_for_backward(x, output[1], weight)
    ctx.mark_non_differentiable(output[1])


def _layer_backward(ctx, dh, _):
    x, stats, weight = ctx.saved_tensors
    dx, dw, *db = layer_norm_backward(None, _dense(dh), x, stats, weight, ctx.bias, None, 0.0, 0, 1.0)
    return dx, dw, db[0] if db else None, None


layer_norm.register_autograd(_layer_backward, setup_context=_layer_context)


def _add_layer_context(ctx, inputs, output):
    _, _, weight, bias, rng, ctx.p, ctx.call, ctx.residual_scale, _ = inputs
    ctx.bias = bias is not None
    ctx.save_for_backward(output[0], output[2], weight, rng)
    ctx.mark_non_differentiable(output[2])
    ctx.set_materialize_grads(False)


def _add_layer_backward(ctx, dx_new, dh, _):
    x_new, stats, weight, rng = ctx.saved_tensors
    if dx_new is None and dh is None:
        return (None,) * 9
    if dh is None:  # nothing came through the norm
        g = _dense(dx_new)
        dy = dropout_op(g, rng, None, ctx.p, ctx.call, 1.0) if ctx.p > 0 else g
        return dy, g if ctx.residual_scale == 1.0 else g * ctx.residual_scale, *(None,) * 7
    dx, dw, *rest = layer_norm_backward(_dense(dx_new), _dense(dh), x_new, stats, weight, ctx.bias, rng, ctx.p, ctx.call,
                                        ctx.residual_scale)
    dy = rest[0] if _own_dy(ctx.p, ctx.residual_scale) else dx
    return dy, dx, dw, rest[-1] if ctx.bias else None, *(None,) * 5


add_layer_norm.register_autograd(_add_layer_backward, setup_context=_add_layer_context)


# ------------------------------------------------------------------ embedding
@torch.library.custom_op("zc::embedding", mutates_args=())
def embedding_op(ids: torch.Tensor, table: torch.Tensor, scale: float,
                 dtype: torch.dtype | None) -> tuple[torch.Tensor, torch.Tensor]:
    status = zc.new_status(table.device)
    return embedding.lookup(ids, table, status, scale=scale, dtype=dtype), status


@embedding_op.register_fake
def _(ids, table, scale, dtype):
    return (table.new_empty((ids.shape[0], table.shape[1]), dtype=dtype or table.dtype),
            table.new_empty(1, dtype=torch.int32))


@torch.library.custom_op("zc::embedding_backward", mutates_args=())
def embedding_backward(dout: torch.Tensor, ids: torch.Tensor, vocab: int, scale: float,
                       dtype: torch.dtype) -> torch.Tensor:
    ws = embedding.workspace(ids.shape[0], vocab, dout.shape[1], device=dout.device)
    return embedding.lookup_backward(dout, ids, vocab, ws, zc.new_status(dout.device), scale=scale, dtype=dtype)


@embedding_backward.register_fake
def _(dout, ids, vocab, scale, dtype):
    return dout.new_empty((vocab, dout.shape[1]), dtype=dtype)


def _embedding_context(ctx, inputs, output):
    ids, table, ctx.scale, _ = inputs
    ctx.vocab, ctx.dtype = table.shape[0], table.dtype
    ctx.save_for_backward(ids)
    ctx.mark_non_differentiable(output[1])


def _embedding_backward(ctx, dout, _):
    return None, embedding_backward(_dense(dout), *ctx.saved_tensors, ctx.vocab, ctx.scale, ctx.dtype), None, None


embedding_op.register_autograd(_embedding_backward, setup_context=_embedding_context)
