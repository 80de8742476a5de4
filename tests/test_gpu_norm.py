"""The norms around a block, forward and backward, against their definitions in 64 bits.

Bounds: a result of type T may be off by its own rounding, u |exact|, plus its fp32 roundings: with S the sum of
the magnitudes that make up a value, ops x 2^-24 x S.  A row's sums run over at most 16 values a thread and a tree of
10 levels (27 roundings, halved by the square root), which with the products around them gives the ops below; sums
over tokens add one rounding for each token.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
E32 = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def norm(zc):
    from lossless_bf16_exponent_zc_gb300 import norm as m
    return m


def within(got, want, terms, ops):
    bound = UNIT[got.dtype] * want.abs() + ops * E32 * terms + TINY[got.dtype]
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4], bound[bad][:4])


def near(got, want):
    """Two roundings of nearly the same value: sums taken in two orders, each result rounded."""
    size = want.double().abs().max().clamp(min=1)
    bound = 2 * UNIT[got.dtype] * want.double().abs() + 4096 * E32 * size
    assert ((got.double() - want.double()).abs() <= bound).all()


def gate_rows(gate, tokens):
    return torch.ones((tokens, 1), dtype=torch.float64, device="cuda") if gate is None else \
        gate.double().repeat_interleave(tokens // gate.shape[0], 0)


def rinv(z):
    return 1 / torch.sqrt((z * z).mean(1, keepdim=True) + EPS)


def forward_reference(y, x, w, gate, a, w2):
    y, x, w = y.double(), x.double(), w.double()
    branch = gate_rows(gate, y.shape[0]) * (y * rinv(y) * w)
    x_new = a * x + branch
    size = (a * x).abs() + branch.abs()
    if w2 is None:
        return x_new, size, None, None
    r2 = rinv(x_new)
    return x_new, size, x_new * r2 * w2.double(), size * r2 * w2.double().abs()


def backward_reference(gx, gh, y, x, w, gate, a, w2):
    """name -> (exact, sum of magnitudes)."""
    t = y.shape[0]
    y, w, k = y.double(), w.double(), gate_rows(gate, t)
    g = gx.double() if gx is not None else torch.zeros_like(y)
    s = g.abs()
    out = {}
    if w2 is not None:
        x, h = x.double(), gh.double()
        r2 = rinv(x)
        n2, u = x * r2, h * w2.double()
        g = g + r2 * (u - n2 * (u * n2).mean(1, keepdim=True))
        s = s + r2 * (u.abs() + n2.abs() * (u * n2).abs().mean(1, keepdim=True))
        out["dnext_weight"] = ((h * n2).sum(0), (h * n2).abs().sum(0))
    r = rinv(y)
    n = y * r
    out["dx"] = (a * g, abs(a) * s)
    out["dweight"] = ((g * k * n).sum(0), (s * (k * n).abs()).sum(0))
    if gate is not None:
        e, es = g * n * w, s * (n * w).abs()
        if gate.shape[1] == 1:
            e, es = e.sum(1, keepdim=True), es.sum(1, keepdim=True)
        rows = gate.shape[0]
        out["dgate"] = tuple(m.reshape(rows, t // rows, -1).sum(1) for m in (e, es))
    v, vs = g * k * w, s * (k * w).abs()
    out["dy"] = (r * (v - n * (v * n).mean(1, keepdim=True)), r * (vs + n.abs() * (vs * n.abs()).mean(1, keepdim=True)))
    return out


def make(seed, tokens, hidden, dtype, params, gate, with_next):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    dt, pt = TYPES[dtype], TYPES[params]
    shape = {"none": None, "channel": (1, hidden), "token": (tokens, 1), "scalar": (1, 1), "full": (tokens, hidden),
             "sequence": (tokens // 3, hidden), "narrow": (tokens // 3, 1)}[gate]
    return dict(y=(randn(tokens, hidden) * 3).to(dt), x=randn(tokens, hidden).to(dt),
                gx=randn(tokens, hidden).to(dt), gh=randn(tokens, hidden).to(dt),
                w=(1 + 0.2 * randn(hidden)).to(pt), w2=(1 + 0.2 * randn(hidden)).to(pt) if with_next else None,
                gate=randn(*shape).to(pt) if shape else None, a=0.75)


def check(norm, d, ws=None):
    tokens, hidden = d["y"].shape
    x_new, h = norm.post_norm(d["y"], d["x"], d["w"], gate=d["gate"], residual_scale=d["a"], next_weight=d["w2"],
                              eps=EPS)
    ex, sx, eh, sh = forward_reference(d["y"], d["x"], d["w"], d["gate"], d["a"], d["w2"])
    within(x_new, ex, sx, 32)
    if d["w2"] is not None:
        within(h, eh, sh, 64)
    else:
        assert h is None
    ws = norm.workspace(tokens, hidden) if ws is None else ws
    gh = d["gh"] if d["w2"] is not None else None
    got = norm.post_norm_backward(d["gx"], gh, d["y"], d["x"], d["w"], ws, gate=d["gate"], residual_scale=d["a"],
                                  next_weight=d["w2"], eps=EPS)
    want = backward_reference(d["gx"], gh, d["y"], d["x"], d["w"], d["gate"], d["a"], d["w2"])
    for name in got._fields:
        v = getattr(got, name)
        if name not in want:
            assert v is None
            continue
        assert v.dtype == (d["w"].dtype if name in ("dweight", "dgate", "dnext_weight") else d["y"].dtype)
        e, s = want[name]
        within(v, e.reshape(v.shape), s.reshape(v.shape), 128 + (0 if name in ("dx", "dy") else tokens + hidden // 16))
    return x_new, h, got


WIDTHS = [1, 7, 64, 100, 256, 264, 512, 513, 520, 1531, 4096, 4100, 5120, 8192, 16383, 16384]


@pytest.mark.parametrize("hidden", WIDTHS)
@pytest.mark.parametrize("dtype,params", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("with_next", [True, False])
def test_widths(norm, hidden, dtype, params, with_next):
    check(norm, make(hidden, 21, hidden, dtype, params, "channel", with_next))


@pytest.mark.parametrize("gate", ["none", "channel", "token", "scalar", "full", "sequence", "narrow"])
@pytest.mark.parametrize("tokens", [3, 18, 999, 3000])
@pytest.mark.parametrize("hidden", [72, 130, 1024])
def test_gates(norm, gate, tokens, hidden):
    check(norm, make(tokens, tokens, hidden, "bf16", "f32", gate, True))
    check(norm, make(tokens, tokens, hidden, "f32", "f32", gate, False))


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full", "sequence", "narrow"])
@pytest.mark.parametrize("hidden", [4099, 8200, 12288])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_of_wide_rows(norm, gate, hidden, dtype):
    check(norm, make(hidden, 402, hidden, dtype, "f32", gate, True))


@pytest.mark.parametrize("tokens", [1, 2, 151, 305, 2049])
def test_token_counts_and_a_reused_workspace(norm, tokens):
    """The workspace holds whatever an earlier call left there."""
    ws = norm.workspace(2049, 768)
    ws.fill_(0xFF)
    check(norm, make(tokens, tokens, 768, "bf16", "bf16", "channel", True), ws)
    check(norm, make(tokens + 1, tokens, 96, "bf16", "bf16", "channel", True), ws)


@pytest.mark.parametrize("hidden", [64, 1030, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pre_norm(norm, hidden, dtype):
    d = make(7, 45, hidden, dtype, dtype, "none", True)
    x, w, gh = d["x"], d["w2"], d["gh"]
    h = norm.pre_norm(x, w, eps=EPS)
    xd, wd = x.double(), w.double()
    r = rinv(xd)
    within(h, xd * r * wd, (xd * r * wd).abs(), 32)
    ws = norm.workspace(45, hidden)
    n, u = xd * r, gh.double() * wd
    core = r * (u - n * (u * n).mean(1, keepdim=True))
    size = r * (u.abs() + n.abs() * (u * n).abs().mean(1, keepdim=True))
    for res in (None, d["gx"]):
        dx, dw = norm.pre_norm_backward(gh, x, w, ws, dresidual=res, eps=EPS)
        extra = res.double() if res is not None else torch.zeros_like(core)
        within(dx, core + extra, size + extra.abs(), 128)
        within(dw, (gh.double() * n).sum(0), (gh.double() * n).abs().sum(0), 128 + 45)


def test_only_through_h(norm):
    """No gradient reaches x_new past the next block."""
    d = make(3, 30, 264, "f32", "f32", "channel", True)
    ws = norm.workspace(30, 264)
    got = norm.post_norm_backward(None, d["gh"], d["y"], d["x"], d["w"], ws, gate=d["gate"], residual_scale=d["a"],
                                  next_weight=d["w2"], eps=EPS)
    want = backward_reference(None, d["gh"], d["y"], d["x"], d["w"], d["gate"], d["a"], d["w2"])
    for name in got._fields:
        within(getattr(got, name), want[name][0].reshape(getattr(got, name).shape),
               want[name][1].reshape(getattr(got, name).shape), 256)


def test_views_expanded_gradients_and_in_place(norm):
    """Strided, misaligned and expanded inputs give what their copies give; x_new may replace x."""
    d = make(5, 40, 96, "bf16", "bf16", "channel", True)
    base = torch.randn((80, 113), device="cuda").to(torch.bfloat16)
    for view in (base[::2, :96], base[:40, 1:97], base[:1, 8:104].expand(40, 96)):
        a = norm.post_norm(view, d["x"], d["w"], gate=d["gate"], next_weight=d["w2"])
        b = norm.post_norm(view.contiguous(), d["x"], d["w"], gate=d["gate"], next_weight=d["w2"])
        near(a[0], b[0])
        near(a[1], b[1])
        ws = norm.workspace(40, 96)
        ga = norm.post_norm_backward(view, view, view, view, d["w"], ws, gate=d["gate"], next_weight=d["w2"])
        gb = norm.post_norm_backward(*[view.contiguous()] * 4, d["w"], ws, gate=d["gate"], next_weight=d["w2"])
        for u, v in zip(ga, gb):
            near(u, v)
    x = d["x"].clone()
    want = norm.post_norm(d["y"], d["x"], d["w"], gate=d["gate"], next_weight=d["w2"])
    got = norm.post_norm(d["y"], x, d["w"], gate=d["gate"], next_weight=d["w2"], x_new=x)
    assert got[0] is x and torch.equal(x, want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("hidden", [1, 3, 65, 129, 255])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "narrow"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_narrow_odd_rows(norm, hidden, gate, dtype):
    check(norm, make(hidden, 6000, hidden, dtype, "f32", gate, True))


def inside(t, before, after):
    """The same matrix as columns of a wider one that holds NaN elsewhere."""
    wide = torch.full((t.shape[0], before + t.shape[1] + after), math.nan, dtype=t.dtype, device=t.device)
    wide[:, before:before + t.shape[1]] = t
    return wide[:, before:before + t.shape[1]]


@pytest.mark.parametrize("before,after", [(0, 0), (0, 16), (8, 24), (0, 3), (1, 0), (5, 8)])
@pytest.mark.parametrize("hidden", [259, 515, 1018, 1531, 4085, 4095])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_off_sixteen_bytes(norm, hidden, dtype, before, after):
    """Rows that start in the same place as the outputs' and others; what lies beside them is not looked at."""
    d = make(hidden + before, 700, hidden, dtype, "f32", "channel", True)
    d["gate"] = 1 + 0.3 * torch.randn(7, hidden, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    for name in ("y", "x", "gx", "gh"):
        d[name] = inside(d[name], before, after)
    check(norm, d)


@pytest.mark.parametrize("hidden", [515, 1531, 4081, 4095])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_off_sixteen_bytes(norm, hidden, dtype):
    """x_new over x where neighbouring rows share 16 bytes."""
    d = make(hidden, 2000, hidden, dtype, "f32", "token", True)
    want = norm.post_norm(d["y"], d["x"], d["w"], gate=d["gate"], next_weight=d["w2"])
    got = norm.post_norm(d["y"], d["x"], d["w"], gate=d["gate"], next_weight=d["w2"], x_new=d["x"])
    assert got[0] is d["x"] and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("hidden", [515, 1531, 4085])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_a_row_of_nan_stays_alone(norm, hidden, dtype):
    d = make(hidden, 610, hidden, dtype, "f32", "none", True)

    def rows(d):
        x_new, h = norm.post_norm(d["y"], d["x"], d["w"], residual_scale=0.5, next_weight=d["w2"])
        dy, dx = norm.post_norm_backward(d["gx"], d["gh"], d["y"], d["x"], d["w"], norm.workspace(610, hidden),
                                         residual_scale=0.5, next_weight=d["w2"])[:2]
        return [m[::2] for m in (x_new, h, dy, dx)]

    want = rows(d)
    for name in ("y", "x", "gx", "gh"):
        d[name][1::2] = math.nan
    for g, w in zip(rows(d), want):
        assert torch.equal(g, w)


def test_offsets_past_32_bits(norm):
    """More than 2^32 bytes and 2^31 values: the last rows are those of a call with them alone."""
    tokens, hidden = 140000, 16384
    g = torch.Generator(device="cuda").manual_seed(13)
    one = torch.randn((7, hidden), device="cuda", generator=g).to(torch.bfloat16)
    x = torch.empty((tokens, hidden), dtype=torch.bfloat16, device="cuda")
    x.zero_()
    x[-7:] = one
    w = torch.rand(hidden, device="cuda", generator=g) + 0.5
    assert x.numel() > 2 ** 31
    got, want = norm.post_norm(x, x, w, next_weight=w), norm.post_norm(one, one, w, next_weight=w)
    for a, b in zip(got, want):
        assert torch.equal(a[-7:], b) and not a[:-7].any()
    del got
    ws = norm.workspace(tokens, hidden)
    a = norm.post_norm_backward(x, x, x, x, w, ws, next_weight=w)
    b = norm.post_norm_backward(one, one, one, one, w, ws, next_weight=w)
    assert torch.equal(a.dy[-7:], b.dy) and torch.equal(a.dx[-7:], b.dx)
    # the rows of zeros add nothing; the seven are shared out among other CTAs, so their sums have another order
    for u, v in ((a.dweight, b.dweight), (a.dnext_weight, b.dnext_weight)):
        assert float((u - v).abs().max()) <= 32 * E32 * float(v.abs().max())


def test_zeros_infinities_and_nan(norm):
    """A row of zeros norms to zero; a row with an infinity or NaN spoils itself alone."""
    d = make(6, 12, 128, "f32", "f32", "token", True)
    d["y"][2] = 0
    check(norm, d)
    clean = norm.post_norm(d["y"], d["x"], d["w"], gate=d["gate"], next_weight=d["w2"])
    d["y"][4, 9] = float("nan")
    d["x"][7, 0] = float("inf")
    x_new, h = norm.post_norm(d["y"], d["x"], d["w"], gate=d["gate"], next_weight=d["w2"])
    keep = torch.tensor([t not in (4, 7) for t in range(12)], device="cuda")
    assert torch.equal(x_new[keep], clean[0][keep]) and torch.equal(h[keep], clean[1][keep])
    assert torch.isnan(x_new[4]).all() and torch.isnan(h[4]).all() and torch.isinf(x_new[7, 0])


def test_no_tokens(norm):
    d = make(1, 3, 64, "bf16", "f32", "channel", True)
    none = d["x"][:0]
    x_new, h = norm.post_norm(none, none, d["w"], gate=d["gate"], next_weight=d["w2"])
    assert x_new.shape == h.shape == (0, 64) and norm.pre_norm(none, d["w2"]).shape == (0, 64)
    got = norm.post_norm_backward(none, none, none, none, d["w"], norm.workspace(0, 64), gate=d["gate"],
                                  next_weight=d["w2"])
    assert got.dx.shape == (0, 64) and not got.dweight.any() and not got.dgate.any() and not got.dnext_weight.any()


@pytest.mark.parametrize("gate", ["channel", "token", "sequence"])
def test_gradient_against_differences(norm, gate):
    """Directional central differences of the kernels' own fp32 forward, step 2^-7.  The loss is a sum of 2 x 9 x 40 outputs
    of unit size, each off by under 2^-20 in fp32 and, for its curvature, 2^-14 x a few: 1e-3 of the
    sum of magnitudes (about 700) covers both."""
    d = make(8, 9, 40, "f32", "f32", gate, True)
    c1, c2 = torch.randn((9, 40), device="cuda"), torch.randn((9, 40), device="cuda")

    def loss(y, x, w, k, w2):
        x_new, h = norm.post_norm(y, x, w, gate=k, residual_scale=d["a"], next_weight=w2, eps=EPS)
        return float((x_new.double() * c1).sum() + (h.double() * c2).sum())

    args = [d["y"], d["x"], d["w"], d["gate"], d["w2"]]
    x_new, _ = norm.post_norm(*args[:3], gate=d["gate"], residual_scale=d["a"], next_weight=d["w2"], eps=EPS)
    g = norm.post_norm_backward(c1, c2, d["y"], x_new, d["w"], norm.workspace(9, 40), gate=d["gate"],
                                residual_scale=d["a"], next_weight=d["w2"], eps=EPS)
    step = 2.0 ** -7
    for i, grad in enumerate([g.dy, g.dx, g.dweight, g.dgate, g.dnext_weight]):
        way = torch.randn_like(args[i])
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + step * way, args[i] - step * way
        diff = (loss(*up) - loss(*dn)) / (2 * step)
        assert abs(diff - float((grad.double() * way).sum())) < 0.7


def test_same_bits_every_time_on_any_stream(norm):
    d = make(12, 1998, 640, "bf16", "f32", "sequence", True)
    ws = norm.workspace(1998, 640)

    def step():
        x_new, h = norm.post_norm(d["y"], d["x"], d["w"], gate=d["gate"], next_weight=d["w2"])
        return [x_new, h, *norm.post_norm_backward(d["gx"], d["gh"], d["y"], x_new, d["w"], ws, gate=d["gate"],
                                                   next_weight=d["w2"])]

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_refusals(norm, zc):
    d = make(4, 6, 32, "bf16", "bf16", "channel", True)
    y, x, w, k = d["y"], d["x"], d["w"], d["gate"]
    ws = norm.workspace(6, 32)
    for bad in (lambda: norm.post_norm(y.cpu(), x, w), lambda: norm.post_norm(y, x.cpu(), w),
                lambda: norm.post_norm(y, x, w.cpu()), lambda: norm.post_norm(y, x[:5], w),
                lambda: norm.post_norm(y, x.float(), w), lambda: norm.post_norm(y, x, w[:31]),
                lambda: norm.post_norm(y, x, w.half()), lambda: norm.post_norm(y, x, w, gate=k.float()),
                lambda: norm.post_norm(y, x, w, gate=k[0]), lambda: norm.post_norm(y, x, w, gate=k[:, :5]),
                lambda: norm.post_norm(y, x, w, gate=k.expand(4, 32).contiguous()),
                lambda: norm.post_norm(y.t(), x.t(), w[:6]), lambda: norm.post_norm(y.double(), x.double(), w.double()),
                lambda: norm.post_norm(y, x, w, x_new=y[:3]), lambda: norm.pre_norm(y[0], w),
                lambda: norm.post_norm_backward(x, None, y, x, w, ws, next_weight=w),
                lambda: norm.post_norm_backward(x, x, y, x, w, ws),
                lambda: norm.post_norm_backward(x, x, y, None, w, ws, next_weight=w),
                lambda: norm.post_norm_backward(None, None, y, x, w, ws)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(zc.ZcError) as e:
        norm.post_norm_backward(x, x, y, x, w, ws[:-1], next_weight=w)
    assert e.value.code == zc.ERR_WORKSPACE
    wide = torch.zeros((2, norm.MAX_HIDDEN + 8), device="cuda")
    with pytest.raises(zc.ZcError) as e:
        norm.pre_norm(wide, wide[0])
    assert e.value.code == zc.ERR_TOO_LARGE
    with pytest.raises(zc.ZcError) as e:
        norm.pre_norm(x, w, eps=-1.0)
    assert e.value.code == zc.ERR_INVALID_ARG
