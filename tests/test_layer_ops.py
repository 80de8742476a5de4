"""torch.ops.zc.moe_* and the norms: registered, traceable, and differentiable together as a block uses them.

CPU part: the operators register and give their outputs' shapes and types under fake tensors, their backward operators
too.  GPU part: the gradients of a whole block (norm, router, dispatch, a product per expert, combine, norm) against
automatic differentiation of the plain formulas in 64 bits, and the example block trained for a few steps.
"""
import math
import os
import sys

import pytest
import torch

from lossless_bf16_exponent_zc_gb300 import torch_ops  # noqa: F401  (registers torch.ops.zc)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ops = torch.ops.zc


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_fake_shapes(dtype):
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        x = torch.empty((12, 40), dtype=dtype, device="cuda")
        w = torch.empty(40, dtype=dtype, device="cuda")
        gate = torch.empty((3, 40), dtype=dtype, device="cuda")
        logits = torch.empty((12, 9), dtype=dtype, device="cuda")
        weights, experts = ops.moe_route(logits, None, 4, "softmax", True, 1.0)
        assert weights.shape == experts.shape == (12, 4) and (weights.dtype, experts.dtype) == (torch.float32, torch.int32)
        assert ops.moe_route_backward(weights, logits, experts, "softmax", True, 1.0).shape == logits.shape
        rows, positions, slots, offsets = ops.moe_dispatch(x, experts, 9)
        assert rows.shape == (48, 40) and rows.dtype == dtype and rows.device.type == "cuda"
        assert positions.shape == (12, 4) and slots.shape == (48,) and offsets.shape == (10,)
        assert ops.moe_dispatch_backward(rows, positions).shape == x.shape
        out, status = ops.moe_combine(rows, weights, positions)
        assert out.shape == x.shape and out.dtype == dtype and status.dtype == torch.int32
        drows, dweights = ops.moe_combine_backward(out, rows, weights, positions)
        assert drows.shape == rows.shape and dweights.shape == weights.shape
        assert ops.pre_norm(x, w, 1e-6).shape == x.shape and ops.post_norm(x, x, w, gate, 1.0, 1e-6).shape == x.shape
        a, b = ops.post_pre_norm(x, x, w, gate, w, 1.0, 1e-6)
        assert a.shape == b.shape == x.shape
        shapes = [tuple(t.shape) for t in ops.post_norm_backward(a, b, x, a, w, gate, w, 1.0, 1e-6)]
        assert shapes == [(12, 40), (12, 40), (40,), (3, 40), (40,)]
    for name in ("moe_route", "moe_dispatch", "moe_combine", "pre_norm", "post_norm", "post_pre_norm"):
        schema = getattr(ops, name).default._schema
        assert not any(a.alias_info is not None and a.alias_info.is_write for a in schema.arguments)


def plain_block(v, experts, k, score, mask):
    """The block of test_gradients_of_a_block in elementary operations, the chosen experts given: closed experts have
    no probability, and a token with none chosen gets nothing."""
    def rms(z):
        return z * torch.rsqrt(z.square().mean(1, keepdim=True) + 1e-6)

    h = rms(v["x"]) * v["w0"]
    logits = h @ v["router"]
    open_ = mask == 0
    p = torch.where(open_, torch.exp(logits - logits.detach().amax(1, keepdim=True)), 0) if score == "softmax" \
        else torch.where(open_, torch.sigmoid(logits), 0)
    chosen = torch.gather(p, 1, experts.clamp(min=0).long()) * (experts >= 0)
    weights = chosen / (chosen.sum(1, keepdim=True) + 1e-20)
    y = sum(weights[:, j:j + 1] * torch.einsum("td,tde->te", h, v["up"][experts[:, j].clamp(min=0).long()])
            for j in range(k))
    x_new = 0.8 * v["x"] + v["gate"].repeat_interleave(h.shape[0] // v["gate"].shape[0], 0) * rms(y) * v["w1"]
    return x_new, rms(x_new) * v["w2"]


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("masked", [False, True])
def test_gradients_of_a_block(zc, score, masked):
    """fp32 sums of up to 48 terms through eight operators: each is good to about 2^-20 of its terms, and the norms pass on
    the relative error of their input's, so 2^-14 of the largest gradient of a tensor leaves a wide margin."""
    torch.manual_seed(1)
    tokens, hidden, n, k = 60, 48, 6, 2
    shapes = {"x": (tokens, hidden), "w0": (hidden,), "router": (hidden, n), "up": (n, hidden, hidden),
              "gate": (4, hidden), "w1": (hidden,), "w2": (hidden,)}
    v = {name: torch.randn(s, device="cuda") * (hidden ** -0.5 if len(s) == 3 else 1) for name, s in shapes.items()}
    leaf = {name: t.clone().requires_grad_(True) for name, t in v.items()}
    mask = torch.zeros((tokens, n), device="cuda")
    if masked:
        mask[torch.rand((tokens, n), device="cuda") < 0.5] = -math.inf
        mask[3] = -math.inf
        mask[5] = -math.inf
        mask[5, 2] = 0

    h = ops.pre_norm(leaf["x"], leaf["w0"], 1e-6)
    logits = h @ leaf["router"] + mask
    weights, experts = ops.moe_route(logits, None, k, score, True, 1.0)
    rows, positions, _, offsets = ops.moe_dispatch(h, experts, n)
    at = offsets.tolist()
    out = torch.cat([rows[at[e]:at[e + 1]] @ leaf["up"][e] for e in range(n)])  # the unrouted tail is not sent
    y, status = ops.moe_combine(out, weights, positions)
    got = ops.post_pre_norm(y, leaf["x"], leaf["w1"], leaf["gate"], leaf["w2"], 0.8, 1e-6)
    assert zc.status_value(status) == 0
    exact = {name: t.double().requires_grad_(True) for name, t in v.items()}
    want = plain_block(exact, experts, k, score, mask.double())
    c = [torch.randn_like(g) for g in got]
    sum((g * w).sum() for g, w in zip(got, c)).backward()
    sum((g * w.double()).sum() for g, w in zip(want, c)).backward()
    for g, w in zip(got, want):
        g, w = g.detach(), w.detach()
        assert float((g.double() - w).abs().max()) < 2 ** -14 * float(w.abs().max())
    for name in v:
        d, e = leaf[name].grad.double(), exact[name].grad
        assert float((d - e).abs().max()) < 2 ** -14 * float(e.abs().max()), name


@pytest.mark.gpu
def test_partly_used_outputs(zc):
    """Gradients that reach only one of two outputs, or come as views with other strides."""
    torch.manual_seed(2)
    y, x = (torch.randn((10, 24), device="cuda", requires_grad=True) for _ in range(2))
    w, w2 = (torch.ones(24, device="cuda", requires_grad=True) for _ in range(2))
    a, _ = ops.post_pre_norm(y, x, w, None, w2, 0.5, 1e-6)
    a.t().contiguous().sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 0.5)) and w2.grad is None and y.grad is not None
    x.grad = y.grad = w.grad = None
    _, b = ops.post_pre_norm(y, x, w, None, w2, 0.5, 1e-6)
    b.sum().backward()                                   # an expanded gradient
    assert w2.grad is not None and x.grad is not None
    one = ops.post_norm(y, x, w, None, 1.0, 1e-6)
    one.sum().backward()
    weights, experts = ops.moe_route(torch.randn((10, 4), device="cuda", requires_grad=True), None, 2, "softmax", False,
                                     1.0)
    weights.sum().backward()
    rows, positions, _, _ = ops.moe_dispatch(x, experts, 4)
    x.grad = None
    rows.sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0))


@pytest.mark.gpu
def test_example_block_trains(zc):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import moe_block
        import torch.distributed as dist
        losses = moe_block.main()
        dist.destroy_process_group()
    finally:
        sys.path.pop(0)
    assert all(math.isfinite(v) for v in losses) and losses[-1] < losses[0]
