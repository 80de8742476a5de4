"""Routing, dispatch and combine against plain implementations in 64 bits, at the sizes and masks where they can go wrong.

Bounds: a result of type T may be off by its own rounding, u |exact| (u = 2^-8 bf16, 2^-11 f16, 2^-24 fp32, and half
the smallest subnormal below the normal range), plus the error of its fp32 sums, at most (terms + a few roundings) x 2^-24
times the sum of the terms' magnitudes.  Integers and moved values are exact.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
E32 = 2.0 ** -24


@pytest.fixture(scope="module")
def moe(zc):
    from lossless_bf16_exponent_zc_gb300 import moe as m
    return m


def within(got, want, terms, ops, dtype=None):
    """got (any type) against want (64 bits); terms: the sum of the magnitudes behind each value, ops: its roundings."""
    dt = dtype or got.dtype
    got, want = got.double().cpu(), want.cpu()
    bound = UNIT[dt] * want.abs() + ops * E32 * terms.cpu() + TINY[dt]
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= bound))
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4], bound[bad][:4])


def ids_of(g, tokens, k, experts, dropped=0.0, dtype=torch.int32):
    ids = torch.argsort(torch.rand((tokens, experts), generator=g), dim=1)[:, :k]
    ids = torch.where(torch.rand((tokens, k), generator=g) < dropped, -1, ids)
    return ids.to(dtype).contiguous()


def place(ids, experts):
    """Positions, slots and offsets of the stable sort, one slot at a time."""
    flat = [int(v) if 0 <= int(v) < experts else experts for v in ids.reshape(-1)]
    slots = sorted(range(len(flat)), key=lambda s: (flat[s], s))
    positions = [0] * len(flat)
    for r, s in enumerate(slots):
        positions[s] = r if flat[s] < experts else -1 - r
    offsets = [sum(f < e for f in flat) for e in range(experts + 1)]
    return positions, slots, offsets


# ------------------------------------------------------------------ routing
def route_reference(logits, k, score, bias, renormalize, scale, dweights):
    """Weights, experts and the logits' gradient of one row at a time, in 64 bits (numpy)."""
    tokens, n = logits.shape
    weights, experts = np.zeros((tokens, k)), np.full((tokens, k), -1)
    dlogits = np.zeros((tokens, n))
    for t in range(tokens):
        l = logits[t].astype(np.float64)
        open_ = l != -np.inf
        with np.errstate(over="ignore"):
            p = 1 / (1 + np.exp(-l))
        choice = l if score == "softmax" else p + bias
        if score == "softmax":
            p = np.exp(l - l.max()) if open_.any() else np.zeros(n)
            p = p / p.sum() if open_.any() else p
        order = [e for e in sorted(range(n), key=lambda e: (-choice[e], e)) if open_[e]][:k]
        experts[t, :len(order)] = order
        total = p[order].sum() + 1e-20
        f = p / total if renormalize else p
        weights[t, :len(order)] = scale * f[order]
        g = np.zeros(n)
        g[order] = scale * dweights[t, :len(order)]
        if renormalize:
            chosen = np.zeros(n)
            chosen[order] = 1
            g = chosen * (g - (g * f * chosen).sum()) / total
        dlogits[t] = p * (1 - p) * g if score == "sigmoid" else p * (g - (p * g).sum())
    return weights, experts, dlogits


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (3, 2, 2), (5, 33, 4), (9, 64, 8), (7, 100, 6), (130, 256, 8),
                                              (6, 511, 32), (2, 1024, 32)])
def test_route(moe, tokens, experts, k, dtype, renormalize, score):
    rng = np.random.default_rng(tokens * experts + k)
    # a permutation of a grid: scores are distinct after rounding to any type up to 64 experts, ties beyond (by design)
    grid = np.linspace(-4, 4, experts)
    logits = torch.from_numpy(np.stack([rng.permutation(grid) for _ in range(tokens)])).to(TYPES[dtype])
    logits[torch.from_numpy(rng.random((tokens, experts)) < 0.2)] = -math.inf
    if tokens > 2:
        logits[1] = -math.inf                      # nothing to choose
        logits[2] = -math.inf
        logits[2, experts // 2] = 0.5              # a single expert left
    bias = None
    if score == "sigmoid":
        bias = torch.from_numpy(rng.integers(-2, 3, experts) / 4.0).float()
    dw = torch.from_numpy(rng.standard_normal((tokens, k))).float()
    lf = logits.float().numpy()
    w, e, dl = route_reference(lf, k, score, bias.numpy() if bias is not None else None, renormalize, 2.5,
                               dw.numpy().astype(np.float64))
    gl = logits.cuda()
    got_w, got_e = moe.route(gl, k, score=score, bias=bias.cuda() if bias is not None else None,
                             renormalize=renormalize, scale=2.5)
    got_d = moe.route_backward(dw.cuda(), gl, got_e, score=score, renormalize=renormalize, scale=2.5)
    assert got_d.dtype == logits.dtype
    ge = got_e.cpu().numpy()
    if score == "softmax":
        assert np.array_equal(ge, e)
    else:  # equal up to choices that fp32 cannot tell apart
        s = 1 / (1 + np.exp(-lf.astype(np.float64))) + bias.numpy()
        diff = np.argwhere(ge != e)
        for t, j in diff:
            assert abs(s[t, ge[t, j]] - s[t, e[t, j]]) < 4 * 2.0 ** -23
    # exp is good to 2 ulp, arguments up to 8 in size add their own rounding: 8 + 2 + sums of k (or experts) terms
    ops = 32 + experts
    if np.array_equal(ge, e):
        within(got_w, torch.from_numpy(w), torch.from_numpy(np.abs(w)), ops)
        terms = np.abs(dl).max(1, keepdims=True) + 2.5 * np.abs(dw.numpy()).max(1, keepdims=True)
        within(got_d, torch.from_numpy(dl), torch.from_numpy(np.broadcast_to(terms, dl.shape).copy()), ops)


def test_route_ties_and_special_values(moe):
    inf, nan = math.inf, math.nan
    logits = torch.tensor([[1.0, 2.0, 2.0, 2.0, -0.0, 0.0],
                           [0.0, -0.0, 0.0, -inf, -inf, -inf],
                           [-inf] * 6,
                           [1.0, nan, 3.0, 2.0, -inf, 0.0],
                           [1.0, inf, 3.0, 2.0, -inf, 0.0],
                           [-3e38, 3e38, 0.0, -3e38, -inf, -inf]], device="cuda")
    w, e = moe.route(logits, 4)
    assert e.tolist() == [[1, 2, 3, 0], [0, 1, 2, -1], [-1] * 4, [1, 2, 3, 0], [1, 2, 3, 0], [1, 2, 0, 3]]
    assert w[2].tolist() == [0.0] * 4 and w[1, 3] == 0.0
    assert torch.isnan(w[3]).all()                 # a NaN logit shows in the weights
    assert torch.isnan(w[4, 0])                    # inf - inf
    assert w[5].tolist() == [1.0, 0.0, 0.0, 0.0]
    d = moe.route_backward(torch.ones_like(w), logits, e)
    assert torch.equal(d[2], torch.zeros(6, device="cuda"))


@pytest.mark.parametrize("experts", [8, 61, 256, 1000])
@pytest.mark.parametrize("width", [0.001, 1.0, 30.0])
@pytest.mark.parametrize("bias_scale", [None, 0.0, 0.05, 100.0])
def test_route_chooses_as_a_stable_sort_of_the_fp32_scores(moe, experts, width, bias_scale):
    """The choice is by sigmoid + bias rounded to fp32, however near the scores are."""
    g = torch.Generator(device="cuda").manual_seed(experts)
    logits = torch.randn((3000, experts), device="cuda", generator=g) * width
    k = min(8, experts)
    if bias_scale is None:
        bias, scores = None, 1 / (1 + torch.exp(-logits))
    else:
        bias = torch.randn(experts, device="cuda", generator=g) * bias_scale
        scores = 1 / (1 + torch.exp(-logits)) + bias
    order = torch.sort(scores, dim=1, descending=True, stable=True).indices[:, :k]
    w, e = moe.route(logits, k, score="sigmoid", bias=bias, renormalize=False)
    assert torch.equal(e.long(), order)
    assert torch.equal(w, (1 / (1 + torch.exp(-logits))).gather(1, order))


@pytest.mark.parametrize("experts", [40, 64, 300, 1024])
@pytest.mark.parametrize("k", [1, 8, 32])
def test_route_many_equal_or_few_open(moe, experts, k):
    """More experts tie for the last place than a warp has lanes; all that are open stand next to one another."""
    logits = torch.zeros((4, experts), device="cuda")
    logits[1, experts // 2:] = 1.0                 # ties above ties
    logits[2, experts // 4:] = -math.inf           # few open, all equal
    logits[3] = -math.inf
    logits[3, -39:] = torch.arange(39.0)           # few open, in the last lanes alone
    w, e = moe.route(logits, k)
    half, quarter = experts // 2, experts // 4

    def padded(ids):
        return (ids + [-1] * k)[:k]

    assert e[0].tolist() == list(range(k))
    upper = list(range(half, experts))
    assert e[1].tolist() == (upper + list(range(half)))[:k]
    assert e[2].tolist() == padded(list(range(quarter)))
    assert e[3].tolist() == padded(list(range(experts - 1, experts - 40, -1)))
    assert torch.allclose(w.sum(1), torch.ones(4, device="cuda"), rtol=0, atol=2.0 ** -20)


def test_route_strides_bias_and_empty(moe):
    g = torch.Generator().manual_seed(3)
    base = torch.randn((40, 100), generator=g).cuda()
    view = base[::2, 3:90]                         # row stride 200, not 16-byte aligned
    w, e = moe.route(view, 5)
    w2, e2 = moe.route(view.contiguous(), 5)
    assert torch.equal(w, w2) and torch.equal(e, e2)
    assert torch.equal(moe.route_backward(w, view, e), moe.route_backward(w, view.contiguous(), e))
    w, e = moe.route(base[:0], 5)
    assert w.shape == (0, 5) and moe.route_backward(w, base[:0], e).shape == (0, 100)
    # experts that a caller dropped, or that lie outside, pass no gradient on
    w, e = moe.route(base, 3)
    e2 = e.clone()
    e2[:, 1] = -1
    e2[:, 2] = 100
    d = moe.route_backward(torch.ones_like(w), base, e2, score="sigmoid", renormalize=False)
    p = torch.sigmoid(base.double())
    want = torch.zeros_like(p).scatter(1, e[:, :1].long(), (p * (1 - p)).gather(1, e[:, :1].long()))
    within(d, want, torch.ones_like(want) * want.abs().max(), 16)


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                               ("sigmoid", False)])
def test_route_gradient_against_differences(moe, score, renormalize):
    """Central differences of the weights (experts fixed by a wide margin), step 2^-6: the third derivative is below
    a few units, so the error is below 2^-12 + 2^-24 / 2^-6 = 3e-4 a term."""
    g = torch.Generator().manual_seed(5)
    logits = torch.randn((16, 24), generator=g)
    logits[:, :4] += 6
    logits = logits.cuda()
    dw = torch.randn((16, 4), generator=g).cuda()
    w, e = moe.route(logits, 4, score=score, renormalize=renormalize)
    d = moe.route_backward(dw, logits, e, score=score, renormalize=renormalize)
    h = 2.0 ** -6
    for c in (0, 1, 3, 9):
        step = torch.zeros_like(logits)
        step[:, c] = h
        up, eu = moe.route(logits + step, 4, score=score, renormalize=renormalize)
        dn, ed = moe.route(logits - step, 4, score=score, renormalize=renormalize)
        # the same experts in some order: compare by expert
        full = torch.zeros((2, 16, 24), dtype=torch.float64, device="cuda")
        full[0].scatter_(1, eu.long(), up.double())
        full[1].scatter_(1, ed.long(), dn.double())
        diff = ((full[0] - full[1]) / (2 * h)).gather(1, e.long())
        want = (diff * dw.double()).sum(1)
        assert torch.allclose(d[:, c].double(), want, rtol=0, atol=4 * 3e-4 * float(dw.abs().max()))


# ------------------------------------------------------------------ dispatch
SHAPES = [(1, 1, 1, 8), (1, 8, 8, 64), (2, 3, 2, 1), (5, 4, 3, 7), (33, 16, 4, 100), (64, 7, 2, 513), (257, 61, 8, 72),
          (700, 5, 3, 24), (1500, 300, 8, 16), (4096, 2, 1, 8), (2100, 1024, 32, 8)]


@pytest.mark.parametrize("tokens,experts,k,hidden", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
def test_dispatch(moe, zc, tokens, experts, k, hidden, dtype, dropped):
    g = torch.Generator().manual_seed(tokens + experts)
    ids = ids_of(g, tokens, k, experts, dropped)
    x = torch.randn((tokens, hidden), generator=g).to(TYPES[dtype])
    positions, slots, offsets = place(ids, experts)
    ws, st = moe.workspace(tokens, k, experts), zc.new_status()
    rows, plan = moe.dispatch(x.cuda(), ids.cuda(), experts, ws)
    assert plan.positions.reshape(-1).tolist() == positions
    assert plan.slots.tolist() == slots
    assert plan.offsets.tolist() == offsets
    want = torch.zeros((tokens * k, hidden), dtype=x.dtype)
    want[:offsets[-1]] = x[torch.tensor(slots, dtype=torch.long)[:offsets[-1]] // k]
    assert torch.equal(rows.cpu(), want)
    # and its gradient
    drows = torch.randn((tokens * k, hidden), generator=g).to(x.dtype)
    dx = moe.dispatch_backward(drows.cuda(), plan.positions, st)
    at = torch.tensor(positions).reshape(tokens, k)
    picked = torch.where((at >= 0)[..., None], drows[at.clamp(min=0)].double(), 0)
    within(dx, picked.sum(1), picked.abs().sum(1), k)
    assert zc.status_value(st) == 0


@pytest.mark.parametrize("tokens,experts,k", [(1024, 8, 1), (1025, 8, 1), (512, 64, 4), (513, 64, 4), (341, 40, 3),
                                              (342, 40, 3), (16384, 8, 1), (16385, 8, 1), (1900, 100, 8),
                                              (2000, 100, 8)])
def test_dispatch_around_its_choices(moe, tokens, experts, k):
    """Numbers of slots and of counts on both sides of where the sort takes another way, skewed experts."""
    g = torch.Generator().manual_seed(tokens)
    scores = torch.randn((tokens, experts), generator=g) - torch.arange(experts).add(1).log()
    ids = torch.topk(scores, k, dim=1).indices.int()
    x = torch.randn((tokens, 8), generator=g).to(torch.bfloat16)
    rows, plan = moe.dispatch(x.cuda(), ids.cuda(), experts, moe.workspace(tokens, k, experts))
    positions, slots, offsets = place(ids, experts)
    assert plan.positions.reshape(-1).tolist() == positions and plan.slots.tolist() == slots
    assert plan.offsets.tolist() == offsets
    assert torch.equal(rows.cpu(), x[torch.tensor(slots) // k])


def test_dispatch_equal_ids_and_one_expert(moe):
    """Everything to one expert, and the same expert several times in a token: the order is the slots' own."""
    x = torch.arange(3000, device="cuda", dtype=torch.float32)[:, None].repeat(1, 4)
    ids = torch.zeros((3000, 4), dtype=torch.int32, device="cuda")
    rows, plan = moe.dispatch(x, ids, 3, moe.workspace(3000, 4, 3))
    assert torch.equal(plan.slots, torch.arange(12000, device="cuda", dtype=torch.int32))
    assert plan.offsets.tolist() == [0, 12000, 12000, 12000]
    assert torch.equal(rows, x.repeat_interleave(4, 0))


@pytest.mark.parametrize("tokens", [0, 7, 900])
def test_dispatch_int64_ids_and_out_of_range(moe, tokens):
    g = torch.Generator().manual_seed(9)
    ids = ids_of(g, tokens, 4, 12, 0.0, torch.int64)
    if tokens:
        ids[0] = torch.tensor([2 ** 32, -2 ** 40, 12, 2 ** 31 + 3])
        ids[3, 1] = 2 ** 63 - 1
    x = torch.randn((tokens, 16), generator=g).cuda()
    rows, plan = moe.dispatch(x, ids.cuda(), 12, moe.workspace(tokens, 4, 12))
    positions, slots, offsets = place(ids, 12)
    assert plan.positions.reshape(-1).tolist() == positions and plan.slots.tolist() == slots
    assert plan.offsets.tolist() == offsets
    assert rows.shape == (tokens * 4, 16) and (tokens == 0 or not rows[offsets[-1]:].any())


@pytest.mark.parametrize("k", [1, 5])
@pytest.mark.parametrize("cut", [(0, 1), (1, 1), (0, 2), (8, 1)])
def test_strided_and_misaligned_inputs(moe, zc, cut, k):
    """Views whose rows are strided or start off a 16-byte boundary give what their copies give."""
    start, step = cut
    g = torch.Generator().manual_seed(11)
    base = torch.randn((400, 300), generator=g).to(torch.bfloat16).cuda()
    x = base[start:start + 96 * step:step, start:start + 264]
    ids = ids_of(g, 96, k, 10, 0.2).cuda()
    ws, st = moe.workspace(96, k, 10), zc.new_status()
    rows, plan = moe.dispatch(x, ids, 10, ws)
    rows2, plan2 = moe.dispatch(x.contiguous(), ids, 10, ws)
    assert torch.equal(rows, rows2) and torch.equal(plan.slots, plan2.slots)
    w = torch.rand((96, k), generator=g).cuda()
    wide = torch.randn((96 * k, 300), generator=g).to(torch.bfloat16).cuda()[:, start:start + 264]
    assert torch.equal(moe.combine(wide, w, plan.positions, st), moe.combine(wide.contiguous(), w, plan.positions, st))
    a = moe.combine_backward(x, wide, w, plan.positions, st)
    b = moe.combine_backward(x.contiguous(), wide.contiguous(), w, plan.positions, st)
    assert torch.equal(a[0], b[0])
    within(a[1], b[1].double(), (x.float().abs().max() * wide.float().abs().max() * 264).expand(96, k).double(), 64)
    # every row the same one (an expanded gradient)
    one = x[:1].expand(96, 264)
    assert torch.equal(moe.combine_backward(one, wide, w, plan.positions, st)[0],
                       moe.combine_backward(one.contiguous(), wide, w, plan.positions, st)[0])
    assert zc.status_value(st) == 0


# ------------------------------------------------------------------ combine
@pytest.mark.parametrize("hidden", [1, 2, 3, 6, 9, 15, 17, 23, 33, 255, 1021, 4095])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("before,after", [(0, 0), (1, 2), (3, 8)])
def test_rows_off_sixteen_bytes(moe, zc, hidden, dtype, before, after):
    """All four moves of rows that start anywhere, NaN beside them."""
    g = torch.Generator().manual_seed(hidden)

    def matrix(n):
        wide = torch.full((n, before + hidden + after), math.nan, dtype=TYPES[dtype])
        wide[:, before:before + hidden] = torch.randn((n, hidden), generator=g).to(TYPES[dtype])
        return wide.cuda()[:, before:before + hidden]

    tokens, k, experts = 37, 5, 9
    ids = ids_of(g, tokens, k, experts, 0.2).cuda()
    x, rows, dout = matrix(tokens), matrix(tokens * k), matrix(tokens)
    w = torch.rand((tokens, k), generator=g).cuda()
    st = zc.new_status()
    sent, plan = moe.dispatch(x, ids, experts, moe.workspace(tokens, k, experts))
    at = plan.positions.long()
    routed = at >= 0
    want = torch.zeros_like(sent)
    want[at[routed]] = x[:, None].expand(tokens, k, hidden)[routed]
    assert torch.equal(sent, want)
    picked = torch.where(routed[..., None], rows[at.clamp(min=0)].double(), 0)
    within(moe.dispatch_backward(rows, plan.positions, st), picked.sum(1), picked.abs().sum(1), k)
    terms = picked * w.double()[..., None]
    within(moe.combine(rows, w, plan.positions, st), terms.sum(1), terms.abs().sum(1), k + 1)
    drows, dw = moe.combine_backward(dout, rows, w, plan.positions, st)
    grad = torch.zeros_like(drows, dtype=torch.float64)
    grad[at[routed]] = (w.double()[..., None] * dout.double()[:, None])[routed]
    within(drows, grad, grad.abs(), 1)
    prod = picked * dout.double()[:, None]
    within(dw, prod.sum(2), prod.abs().sum(2), hidden // 8 + 32)
    assert zc.status_value(st) == 0


def test_a_row_of_more_than_two_to_the_31_bytes(moe, zc):
    hidden = 2 ** 30 + 5
    x = torch.randint(0, 2 ** 20, (1, hidden), device="cuda", dtype=torch.int32).float()
    ids = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    rows, plan = moe.dispatch(x, ids, 1, moe.workspace(1, 1, 1))
    assert torch.equal(rows, x)
    st, w = zc.new_status(), torch.full((1, 1), 0.5, device="cuda")
    out = moe.combine(rows, w, plan.positions, st)
    assert torch.equal(out, x / 2)
    drows, _ = moe.combine_backward(out, rows, w, plan.positions, st)
    assert torch.equal(drows, x / 4)
    assert zc.status_value(st) == 0


@pytest.mark.parametrize("tokens,experts,k,hidden", [s for s in SHAPES if s[0] < 2000])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dropped", [0.0, 0.3, 1.0])
def test_combine(moe, zc, tokens, experts, k, hidden, dtype, dropped):
    g = torch.Generator().manual_seed(tokens * 3 + k)
    positions = torch.tensor(place(ids_of(g, tokens, k, experts, dropped), experts)[0], dtype=torch.int32)
    positions = positions.reshape(tokens, k)
    rows = torch.randn((tokens * k, hidden), generator=g).to(TYPES[dtype])
    w = torch.rand((tokens, k), generator=g)
    dout = torch.randn((tokens, hidden), generator=g).to(TYPES[dtype])
    off = positions < 0
    w[off] = math.nan                              # what stands in unrouted slots is not looked at
    rows[(-1 - positions[off]).long()] = math.inf
    st = zc.new_status()
    out = moe.combine(rows.cuda(), w.cuda(), positions.cuda(), st)
    drows, dw = moe.combine_backward(dout.cuda(), rows.cuda(), w.cuda(), positions.cuda(), st)
    wd = torch.where(off, 0, w).double()
    picked = torch.where(off[..., None], 0, rows[positions.clamp(min=0).long()].double())
    terms = picked * wd[..., None]
    within(out, terms.sum(1), terms.abs().sum(1), k + 1)
    want = torch.zeros((tokens * k, hidden), dtype=torch.float64)
    want[torch.where(off, -1 - positions, positions).reshape(-1).long()] = \
        (wd[..., None] * dout.double()[:, None]).reshape(tokens * k, hidden)
    within(drows, want, want.abs(), 1)
    prod = picked * dout.double()[:, None]
    # a thread adds its pieces' products in turn, then a tree over at most 256 threads
    within(dw, prod.sum(2), prod.abs().sum(2), hidden // 32 + 24)
    assert zc.status_value(st) == 0


def test_combine_of_fewer_rows_and_bad_positions(moe, zc):
    """The unrouted tail need not be there; a routed position beyond the rows is reported and adds nothing."""
    g = torch.Generator().manual_seed(2)
    rows = torch.randn((6, 40), generator=g).cuda()
    positions = torch.tensor([[0, 5], [3, -8], [-7, 2]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]], device="cuda")
    st = zc.new_status()
    want = torch.stack([rows[0] + 2 * rows[5], 3 * rows[3], 6 * rows[2]])
    assert torch.allclose(moe.combine(rows, w, positions, st), want, rtol=1e-6, atol=1e-6)
    assert zc.status_value(st) == 0
    bad = positions.clone()
    bad[1, 0] = 6
    got = moe.combine(rows, w, bad, st)
    torch.cuda.synchronize()
    assert zc.status_value(st) == zc.ERR_BAD_INDEX and not got[1].any()
    st = zc.new_status()
    dout = torch.ones((3, 40), device="cuda")
    drows, dw = moe.combine_backward(dout, rows, w, bad, st, drows=torch.zeros_like(rows))
    torch.cuda.synchronize()
    assert zc.status_value(st) == zc.ERR_BAD_INDEX and dw[1].tolist() == [0.0, 0.0]
    assert not drows[3].any() and torch.equal(drows[2], torch.full((40,), 6.0, device="cuda"))


def test_offsets_past_32_bits(moe, zc):
    """More than 2^32 bytes and 2^31 values of rows: the last rows are right, both ways."""
    tokens, k, hidden, experts = 66000, 8, 4352, 8
    x = torch.empty((tokens, hidden), dtype=torch.bfloat16, device="cuda")
    x.copy_((torch.arange(tokens, device="cuda") % 251)[:, None])
    ids = torch.arange(8, dtype=torch.int32, device="cuda").repeat(tokens, 1)
    rows, plan = moe.dispatch(x, ids, experts, moe.workspace(tokens, k, experts))
    assert rows.numel() > 2 ** 31
    for e in (0, 7):
        assert torch.equal(rows[e * tokens:(e + 1) * tokens], x)
    w = torch.full((tokens, k), 0.125, device="cuda")
    st = zc.new_status()
    assert torch.equal(moe.combine(rows, w, plan.positions, st), x)
    drows, dw = moe.combine_backward(x, rows, w, plan.positions, st)
    assert torch.equal(drows[7 * tokens:], x / 8) and torch.equal(drows[:tokens], x / 8)
    assert zc.status_value(st) == 0


def test_same_bits_every_time_on_any_stream(moe, zc):
    g = torch.Generator().manual_seed(21)
    x = torch.randn((3001, 520), generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn((3001, 48), generator=g).cuda()

    def step(ws, st):
        w, e = moe.route(logits, 6, score="sigmoid")
        rows, plan = moe.dispatch(x, e, 48, ws)
        out = moe.combine(rows, w, plan.positions, st)
        drows, dw = moe.combine_backward(x, rows, w, plan.positions, st)
        return [w, e, rows, *plan, out, drows, dw, moe.dispatch_backward(drows, plan.positions, st)]

    st = zc.new_status()
    first = step(moe.workspace(3001, 6, 48), st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = moe.workspace(3001, 6, 48)
        again = [step(ws, st) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    for other in again:
        for a, b in zip(first, other):
            assert torch.equal(a, b)
    # a decode step as a CUDA graph
    lg, xs = logits[:4].contiguous(), x[:4].contiguous()
    ws = moe.workspace(4, 6, 48)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w, e = moe.route(lg, 6, score="sigmoid")
        rows, plan = moe.dispatch(xs, e, 48, ws)
        out = moe.combine(rows, w, plan.positions, st)
    lg.copy_(logits[100:104])
    xs.copy_(x[100:104])
    graph.replay()
    w2, e2 = moe.route(logits[100:104], 6, score="sigmoid")
    rows2, plan2 = moe.dispatch(x[100:104], e2, 48, moe.workspace(4, 6, 48))
    assert torch.equal(rows, rows2) and torch.equal(out, moe.combine(rows2, w2, plan2.positions, st))
    assert zc.status_value(st) == 0


def test_refusals(moe, zc):
    x = torch.zeros((6, 32), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((6, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((6, 2), device="cuda")
    rows = torch.zeros((12, 32), dtype=torch.bfloat16, device="cuda")
    ws, st = moe.workspace(6, 2, 4), zc.new_status()
    for bad in (lambda: moe.route(x.cpu(), 2), lambda: moe.route(x[0], 2), lambda: moe.route(x.double(), 2),
                lambda: moe.route(x.t(), 2), lambda: moe.route(x, 2, score="tanh"),
                lambda: moe.route(x, 2, score="sigmoid", bias=w[0]),
                lambda: moe.route(x, 2, score="sigmoid", bias=torch.zeros(32, dtype=torch.float64, device="cuda")),
                lambda: moe.route(x, 2, weights=w[:, :1]),
                lambda: moe.route_backward(w, x, ids.long()), lambda: moe.route_backward(w[:5], x, ids),
                lambda: moe.dispatch(x, ids[:5], 4, ws), lambda: moe.dispatch(x, ids.float(), 4, ws),
                lambda: moe.dispatch(x, ids.cpu(), 4, ws), lambda: moe.dispatch(x, ids.t(), 4, ws),
                lambda: moe.dispatch(x, ids, 4, ws, rows=rows[:3]),
                lambda: moe.combine(rows, None, ids, st), lambda: moe.combine(rows, w[:3], ids, st),
                lambda: moe.combine(rows, w.double(), ids, st), lambda: moe.combine(rows, w, ids.long(), st),
                lambda: moe.combine(rows, w, ids, st.cpu()), lambda: moe.combine(rows.long(), w, ids, st),
                lambda: moe.combine_backward(x.float(), rows, w, ids, st),
                lambda: moe.combine_backward(x[:5], rows, w, ids, st),
                lambda: moe.combine_backward(x, rows, w, ids, st, drows=rows[:5])):
        with pytest.raises(ValueError):
            bad()

    def code(call):
        with pytest.raises(zc.ZcError) as e:
            call()
        return e.value.code

    assert code(lambda: moe.route(x, 33)) == zc.ERR_TOO_LARGE
    assert code(lambda: moe.route(x[:, :3], 4)) == zc.ERR_INVALID_ARG
    assert code(lambda: moe.route(x, 2, bias=torch.zeros(32, device="cuda"))) == zc.ERR_INVALID_ARG
    assert code(lambda: moe.route(torch.zeros((1, 1025), device="cuda"), 2)) == zc.ERR_TOO_LARGE
    assert code(lambda: moe.dispatch(x, ids, 4, ws[:-1])) == zc.ERR_WORKSPACE
    assert code(lambda: moe.dispatch(x, ids, 4, ws[1:])) == zc.ERR_ALIGNMENT
    assert code(lambda: moe.dispatch(x, ids, 1025, ws)) == zc.ERR_TOO_LARGE
