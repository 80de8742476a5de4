"""Shapes at which the layer operators take ways of their own: more than eight slots a token with weights, many tokens off
16 bytes, sorts in chunks of rows off 16 bytes; the router's weights and gradients of every row; a norm's gradient
against differences output by output.

Bounds as in test_gpu_moe.py and test_gpu_norm.py: the result's own rounding plus its fp32 roundings.  The products of
dout and a row are added by a thread over its pieces in turn, at most hidden / 32 + 16 of them, then by a tree of up to
10 levels: hidden / 32 + 40 roundings cover both.
"""
import math

import numpy as np
import pytest
import torch

from test_gpu_moe import TYPES, moe, route_reference, within  # noqa: F401  (moe is a fixture)

pytestmark = pytest.mark.gpu


def inside(t, before, after):
    """The same matrix as columns of a wider one that holds NaN elsewhere."""
    wide = torch.full((t.shape[0], before + t.shape[1] + after), math.nan, dtype=t.dtype, device=t.device)
    wide[:, before:before + t.shape[1]] = t
    return wide[:, before:before + t.shape[1]]


def assignment(seed, tokens, k, experts, dropped):
    """Ids on the GPU, distinct within a token, and the positions, slots and offsets of their stable sort."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.argsort(torch.rand((tokens, experts), device="cuda", generator=g), dim=1)[:, :k].int()
    ids = torch.where(torch.rand((tokens, k), device="cuda", generator=g) < dropped, -1, ids).contiguous()
    key = torch.where(ids < 0, experts, ids).reshape(-1)
    ordered, slots = torch.sort(key, stable=True)
    row = torch.empty_like(slots)
    row[slots] = torch.arange(slots.numel(), device="cuda")
    positions = torch.where(key < experts, row, -1 - row).reshape(tokens, k).int()
    offsets = torch.searchsorted(ordered, torch.arange(experts + 1, device="cuda", dtype=ordered.dtype))
    return ids, positions, slots.int(), offsets.int()


def check_combine(moe, zc, rows, w, positions, dout):
    """combine, its gradient and dispatch's gradient against 64 bits."""
    tokens, k = positions.shape
    hidden, st = rows.shape[1], zc.new_status()
    there = positions >= 0
    at = positions.clamp(min=0).long()
    place = torch.where(there, positions, -1 - positions).long()
    out = moe.combine(rows, w, positions, st)
    drows, dw = moe.combine_backward(dout, rows, w, positions, st)
    dx = moe.dispatch_backward(rows, positions, st)
    sums = torch.zeros((6, tokens, hidden), dtype=torch.float64, device="cuda")
    for j in range(k):
        one = there[:, j, None]
        y = torch.where(one, rows[at[:, j]].double(), 0)
        wj = torch.where(one, w[:, j, None].double(), 0)
        sums[0] += wj * y
        sums[1] += (wj * y).abs()
        sums[2] += y
        sums[3] += y.abs()
        prod = y * dout.double()
        within(dw[:, j], prod.sum(1), prod.abs().sum(1), hidden // 32 + 40)
        grad = wj * dout.double()
        within(drows[place[:, j]], grad, grad.abs(), 1)
    within(out, sums[0], sums[1], k + 1)
    within(dx, sums[2], sums[3], k)
    assert zc.status_value(st) == 0


@pytest.mark.parametrize("k", [9, 16, 32])
@pytest.mark.parametrize("tokens", [20, 310])
@pytest.mark.parametrize("hidden,before", [(264, 0), (2048, 0), (4608, 0), (263, 0), (2049, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_than_eight_slots(moe, zc, k, tokens, hidden, before, dtype):  # noqa: F811
    """combine adds eight slots at a time, its gradient takes four (two off 16 bytes) and, of 304 tokens on, all of a
    token's in one CTA, or a warp."""
    g = torch.Generator(device="cuda").manual_seed(k * tokens + hidden)
    _, positions, _, _ = assignment(k, tokens, k, 40, 0.2)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    rows, dout = (inside(randn(n, hidden).to(TYPES[dtype]), before, 0) for n in (tokens * k, tokens))
    check_combine(moe, zc, rows, randn(tokens, k), positions, dout)


@pytest.mark.parametrize("tokens,hidden,k", [(3000, 4095, 2), (1500, 1021, 5), (700, 2047, 3), (20000, 35, 4)])
@pytest.mark.parametrize("dtype,before,after", [("bf16", 0, 0), ("bf16", 5, 8), ("f16", 1, 2), ("f32", 3, 0)])
def test_many_tokens_off_sixteen_bytes(moe, zc, tokens, hidden, k, dtype, before, after):  # noqa: F811
    """Several units of an output a lane, and all slots of a token in one CTA of the gradient."""
    g = torch.Generator(device="cuda").manual_seed(tokens + hidden)
    _, positions, _, _ = assignment(hidden, tokens, k, 16, 0.1)

    def matrix(n):
        return inside(torch.randn((n, hidden), device="cuda", generator=g).to(TYPES[dtype]), before, after)

    w = torch.rand((tokens, k), device="cuda", generator=g)
    check_combine(moe, zc, matrix(tokens * k), w, positions, matrix(tokens))


@pytest.mark.parametrize("tokens,experts,k", [(900, 7, 3), (1300, 40, 2), (5000, 7, 3), (5000, 200, 3), (9000, 500, 1),
                                              (2500, 1024, 32)])
@pytest.mark.parametrize("hidden,before,after", [(37, 0, 0), (1, 0, 0), (70, 3, 0), (261, 1, 7), (64, 1, 7)])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_dispatch_in_chunks_off_sixteen_bytes(moe, zc, tokens, experts, k, hidden, before, after, dtype):  # noqa: F811
    """Sorts of two and of three launches, one to eight tokens a CTA, rows that start anywhere."""
    g = torch.Generator(device="cuda").manual_seed(tokens + hidden)
    ids, positions, slots, offsets = assignment(tokens, tokens, k, experts, 0.15)
    x = inside(torch.randn((tokens, hidden), device="cuda", generator=g).to(TYPES[dtype]), before, after)
    rows, plan = moe.dispatch(x, ids, experts, moe.workspace(tokens, k, experts))
    assert torch.equal(plan.positions, positions) and torch.equal(plan.slots, slots)
    assert torch.equal(plan.offsets, offsets)
    want = torch.zeros_like(rows)
    routed = int(offsets[-1])
    want[:routed] = x[slots[:routed].long() // k]
    assert torch.equal(rows, want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,experts,k", [(5, 33, 4), (130, 256, 8), (6, 511, 32), (3, 1024, 32)])
def test_router_values_of_every_row(moe, tokens, experts, k, dtype, renormalize, score):  # noqa: F811
    """The weights and gradients are those of the experts chosen; which of two choices that fp32 cannot tell apart was
    taken (the only way the ids may differ) is left to the kernel."""
    rng = np.random.default_rng(tokens + experts)
    logits = torch.from_numpy(rng.standard_normal((tokens, experts)) * 2).to(TYPES[dtype])
    logits[torch.from_numpy(rng.random((tokens, experts)) < 0.2)] = -math.inf
    bias = torch.from_numpy(rng.integers(-2, 3, experts) / 4.0).float() if score == "sigmoid" else None
    dw = torch.from_numpy(rng.standard_normal((tokens, k))).float()
    l64 = logits.double().numpy()
    got_w, got_e = moe.route(logits.cuda(), k, score=score, bias=bias.cuda() if bias is not None else None,
                             renormalize=renormalize, scale=2.5)
    got_d = moe.route_backward(dw.cuda(), logits.cuda(), got_e, score=score, renormalize=renormalize, scale=2.5)
    ids = got_e.cpu().numpy()
    choice = l64 if bias is None else 1 / (1 + np.exp(-l64)) + bias.double().numpy()
    choice = np.where(l64 == -np.inf, -np.inf, choice)
    best = -np.sort(-choice, axis=1)[:, :k]
    assert (np.sort(ids, axis=1)[:, 1:] != np.sort(ids, axis=1)[:, :-1]).all()
    for t in range(tokens):
        assert (np.abs(choice[t, ids[t]] - best[t]) <= 4 * 2.0 ** -23).all()
        order = None
        if bias is not None:  # for the reference, a bias that makes the choice take these ids in this order
            order = np.zeros(experts)
            order[ids[t]] = 1e6 - np.arange(k)
        w, e, dl = route_reference(l64[t:t + 1], k, score, order, renormalize, 2.5, dw[t:t + 1].double().numpy())
        assert np.array_equal(e[0], ids[t])
        within(got_w[t], torch.from_numpy(w[0]), torch.from_numpy(np.abs(w[0])), 32 + experts)
        size = np.abs(dl[0]).max() + 2.5 * float(dw[t].abs().max())
        within(got_d[t], torch.from_numpy(dl[0]), torch.full((experts,), size, dtype=torch.float64), 32 + experts)


@pytest.mark.parametrize("gate", [None, (1, 12), (3, 1), (3, 12)])
def test_norm_gradient_against_differences_of_each_output(zc, gate):
    """Differences of the fp32 forward along a random way, by five points (f(-2h) - 8 f(-h) + 8 f(h) - f(2h)) / 12 h with
    h = 1/8 of a way of a quarter of the inputs' size: its own error h^4 / 30 times a fifth derivative below 10 is below
    1e-4.  An output is up to 20 in size and good to 64 x 2^-24 of that, 8e-5, which the differences make 18 / 12 h = 12
    times as much: 1e-3.  2e-3 covers both and the gradient's own error."""
    from lossless_bf16_exponent_zc_gb300 import norm
    g = torch.Generator(device="cuda").manual_seed(11)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    rows, hidden, a, eps = 3, 12, 0.75, 1e-6
    args = {"y": randn(rows, hidden), "x": randn(rows, hidden), "w": 1 + 0.2 * randn(hidden),
            "w2": 1 + 0.2 * randn(hidden)}
    if gate:
        args["k"] = randn(*gate)
    way = {n: randn(*v.shape) / 4 for n, v in args.items()}

    def forward(v):
        out = norm.post_norm(v["y"], v["x"], v["w"], gate=v.get("k"), residual_scale=a, next_weight=v["w2"], eps=eps)
        return torch.stack(out).double()

    ws, x_new = norm.workspace(rows, hidden), forward(args)[0].float()
    assert float(forward(args).abs().max()) < 20
    h = 1 / 8
    for name in args:
        f = [forward({**args, name: args[name] + s * h * way[name]}) for s in (-2, -1, 1, 2)]
        diff = (f[0] - 8 * f[1] + 8 * f[2] - f[3]) / (12 * h)
        for i in range(2):
            for t in range(rows):
                for c in range(hidden):
                    one = torch.zeros((2, rows, hidden), device="cuda")
                    one[i, t, c] = 1
                    d = norm.post_norm_backward(one[0], one[1], args["y"], x_new, args["w"], ws, gate=args.get("k"),
                                                residual_scale=a, next_weight=args["w2"], eps=eps)
                    grad = {"y": d.dy, "x": d.dx, "w": d.dweight, "w2": d.dnext_weight, "k": d.dgate}[name]
                    assert abs(float((grad.double() * way[name]).sum()) - float(diff[i, t, c])) < 2e-3, (name, i, t, c)
