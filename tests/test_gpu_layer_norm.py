"""Layer norm, alone and behind dropout and the residual addition, against the formulas in 64 bits, both directions.

Tolerances, with u = 2^-24: a sum of a row takes at most 16 additions in a thread and 10 steps of a tree, so it is off by
at most 27 u of the sum of its magnitudes; sums over the rows by (rows + 40) u. The terms below follow the operators'
steps with those; the last rounding is half a step of the output's type.
"""
import pytest
import torch

from test_gpu_dropout import kept

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
U, EPS = 2.0**-24, 1e-5


@pytest.fixture(scope="module")
def norm(zc):
    from lossless_bf16_exponent_zc_gb300 import norm
    return norm


def within(got, want, room, dtype=None):
    f = torch.finfo(dtype or got.dtype)
    room = room + (f.eps / 2 * want.abs() + f.smallest_normal * f.eps)
    bad = (got.double() - want).abs() > room
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()}, by {float(((got.double() - want).abs() / room).max())}"


def check_forward(h, stats, x, dx, w, b):
    """x in 64 bits, what the kernel has of it off by up to dx."""
    w, b = w.double(), b.double() if b is not None else torch.zeros_like(w, dtype=torch.float64)
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    root = 1 / torch.sqrt(var + EPS)
    n = (x - mean) * root
    dmean = 27 * U * x.abs().mean(1, keepdim=True) + U * mean.abs() + dx.mean(1, keepdim=True)
    dc = dmean + dx + 2 * U * (x.abs() + mean.abs())                     # of x - mean
    # of the root: half the relative error of the variance, and the reciprocal square root's own
    droot = root * (0.5 * root**2 * (2 * ((x - mean).abs() * dc).mean(1, keepdim=True) + dc.square().mean(1, keepdim=True)
                                     + 30 * U * var) + 8 * U)
    if h is not None:
        within(h, n * w + b, w.abs() * (root * dc + (x - mean).abs() * droot) + 4 * U * ((n * w).abs() + b.abs()))
    if stats is not None:
        within(stats, torch.cat([mean, root], 1), torch.cat([dmean, droot], 1) + 2 * U)


def check_backward(got, dpast, dh, x, stats, w, scale, keep, factor):
    """got: (dy or None, dx, dweight, dbias or None)"""
    dy, dx, dweight, dbias = got
    dh, x, w = dh.double(), x.double(), w.double()
    mean, root = stats[:, :1].double(), stats[:, 1:].double()
    n, u = (x - mean) * root, dh * w
    dn = 3 * U * ((x.abs() + mean.abs()) * root)
    a, b = u.mean(1, keepdim=True), (u * n).mean(1, keepdim=True)
    da = 29 * U * u.abs().mean(1, keepdim=True)
    db = 29 * U * (u * n).abs().mean(1, keepdim=True) + (u.abs() * dn).mean(1, keepdim=True)
    g = root * (u - a - n * b) + (dpast.double() if dpast is not None else 0)
    dg = root * (da + n.abs() * db + dn * b.abs() + 6 * U * (u.abs() + a.abs() + (n * b).abs())) + 4 * U * g.abs()
    if dpast is not None:
        dg = dg + 2 * U * dpast.double().abs()
    within(dx, scale * g, abs(scale) * dg + 2 * U * (scale * g).abs())
    if dy is not None:
        f = keep * factor if keep is not None else 1.0
        within(dy, g * f, dg * f + 2 * U * (g * f).abs())
    sums = (x.shape[0] + 40) * U
    within(dweight, (dh * n).sum(0), sums * (dh * n).abs().sum(0) + (dh.abs() * dn).sum(0))
    if dbias is not None:
        within(dbias, dh.sum(0), sums * dh.abs().sum(0))


WIDTHS = [1, 2, 7, 8, 33, 64, 129, 256, 264, 511, 512, 520, 1000, 1021, 1024, 1531, 2048, 4088, 4095, 4096, 4104, 5003, 8192,
          12001, 16384]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_layer_norm(norm, dtype, width):
    g = torch.Generator(device="cuda").manual_seed(width)
    for rows, ptype, biased in [(1, dtype, True), (23, torch.float32, False), (700, dtype, True)]:
        x, dh, past = (torch.randn((rows, width), device="cuda", generator=g).to(dtype) for _ in range(3))
        x = (x.float() * 2 + torch.randn((rows, 1), device="cuda", generator=g) * 3).to(dtype)
        w = (1 + 0.2 * torch.randn(width, device="cuda", generator=g)).to(ptype)
        b = torch.randn(width, device="cuda", generator=g).to(ptype) if biased else None
        h, stats = norm.layer_norm(x, w, b, eps=EPS, save=True)
        check_forward(h, stats, x.double(), torch.zeros_like(x, dtype=torch.float64), w, b)
        assert torch.equal(norm.layer_norm(x, w, b, eps=EPS)[0], h) and norm.layer_norm(x, w, b)[1] is None
        ws = norm.workspace(rows, width)
        for dpast in (None, past):
            got = norm.layer_norm_backward(dh, x, stats, w, ws, bias=biased, dresidual=dpast)
            assert (got[2] is not None) == biased and got[1].dtype == ptype
            check_backward((None, *got), dpast, dh, x, stats, w, 1.0, None, None)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("p", [0.0, 0.35])
def test_add_layer_norm(norm, dtype, width, p):
    from lossless_bf16_exponent_zc_gb300 import dropout
    g = torch.Generator(device="cuda").manual_seed(width)
    for rows, scale in [(1, 1.0), (19, -0.5), (330, 1.0)]:
        y, x, dh, past = (torch.randn((rows, width), device="cuda", generator=g).to(dtype) for _ in range(4))
        w, b = (torch.randn(width, device="cuda", generator=g) for _ in range(2))
        rng, call = dropout.new_rng(width, rows), 9
        keep, factor = kept(rows, width, p, width, rows, call) if p else (None, 1.0)
        kw = dict(p=p, rng=rng if p else None, call=call, residual_scale=scale)
        x_new, h, stats = norm.add_layer_norm(y, x, w, b, eps=EPS, save=True, **kw)
        branch = y.double() * (keep * factor if p else 1.0)
        want = scale * x.double() + branch
        off = 3 * U * ((scale * x.double()).abs() + branch.abs())
        within(x_new, want, off)
        check_forward(h, stats, want, off, w, b)
        ws = norm.workspace(rows, width)
        for dpast in (None, past):
            got = norm.add_layer_norm_backward(dpast, dh, x_new, stats, w, ws, **kw)
            assert (got.dy is got.dx) == (p == 0 and scale == 1.0)
            check_backward(got, dpast, dh, x_new, stats, w, scale, keep, factor)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [24, 250, 1024, 1531, 4096, 6001])
@pytest.mark.parametrize("lead,other", [(1, 1), (1, 0), (0, 3), (5, 2)])
def test_strides_and_alignment(norm, dtype, width, lead, other):
    """Rows of wider matrices that start alike or not, one row for all of them, outputs off 16 bytes."""
    from lossless_bf16_exponent_zc_gb300 import dropout
    rows, p = 61, 0.2
    g = torch.Generator(device="cuda").manual_seed(width + lead)

    def strided(first, extra):
        return torch.randn((rows, width + extra), device="cuda", generator=g).to(dtype)[:, first:first + width]

    y, x, dh, past = strided(lead, 8), strided(other, 8), strided(lead, 9), strided(other, 8)
    one = torch.randn((1, width), device="cuda", generator=g).to(dtype).expand(rows, width)
    w, b = (torch.randn(width + 3, device="cuda", generator=g)[lead % 4:][:width] for _ in range(2))
    rng = dropout.new_rng(8)
    keep, factor = kept(rows, width, p, 8, 0, 0)
    room = torch.full((2, rows * width + 8), 7.0, device="cuda").to(dtype)
    a, h = (t[lead:lead + rows * width].view(rows, width) for t in room)
    for res in (x, one):
        got = norm.add_layer_norm(y, res, w, b, p=p, rng=rng, eps=EPS, save=True, x_new=a, h=h)
        assert got[0] is a and got[1] is h
        branch = y.double() * keep * factor
        off = 3 * U * (res.double().abs() + branch.abs())
        within(a, res.double() + branch, off)
        check_forward(h, got[2], res.double() + branch, off, w, b)
        assert bool((room[:, :lead] == 7).all()) and bool((room[:, lead + rows * width:] == 7).all())
        back = norm.add_layer_norm_backward(past, dh, res, got[2], w, norm.workspace(rows, width), p=p, rng=rng)
        check_backward(back, past, dh, res, got[2], w, 1.0, keep, factor)
    check_forward(norm.layer_norm(x, w, b, eps=EPS)[0], None, x.double(), torch.zeros_like(x, dtype=torch.float64), w, b)


@pytest.mark.parametrize("width", [64, 1000, 4096, 16384])
def test_a_large_mean_and_no_variance(norm, width):
    """Means of 1000 times the deviation lose no more than the inputs' own bits; equal values give the bias."""
    x = torch.randn((40, width), device="cuda") + 1000
    w, b = torch.ones(width, device="cuda"), torch.full((width,), 0.25, device="cuda")
    h, stats = norm.layer_norm(x, w, b, eps=EPS, save=True)
    check_forward(h, stats, x.double(), torch.zeros_like(x, dtype=torch.float64), w, b)
    same = torch.full((40, width), 2.0, device="cuda")
    assert torch.equal(norm.layer_norm(same, w, b)[0], b.expand(40, width))
    x[3, 7 % width] = float("nan")
    x[5, 0] = float("inf")
    bad = torch.isnan(norm.layer_norm(x, w, b)[0]).all(1)
    assert bad[3] and bad[5] and int(bad.sum()) == 2


@pytest.mark.parametrize("width", [96, 1024, 4096, 1021])
def test_in_place_and_again(norm, width):
    from lossless_bf16_exponent_zc_gb300 import dropout
    y, x = (torch.randn((500, width), device="cuda").bfloat16() for _ in range(2))
    w, rng = torch.rand(width, device="cuda"), dropout.new_rng(2)
    want = norm.add_layer_norm(y, x, w, p=0.1, rng=rng)
    for target in ("x", "y"):
        t = {"x": x.clone(), "y": y.clone()}
        got = norm.add_layer_norm(t["y"], t["x"], w, p=0.1, rng=rng, x_new=t[target])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    alone, again = norm.layer_norm(x, w)[0], x.clone()
    assert torch.equal(norm.layer_norm(again, w, out=again)[0], alone)
    _, stats = norm.layer_norm(x, w, save=True)
    ws = norm.workspace(500, width)
    first = norm.layer_norm_backward(y, x, stats, w, ws)
    for _ in range(50):
        for a, c in zip(first, norm.layer_norm_backward(y, x, stats, w, ws)):
            assert torch.equal(a, c)


@pytest.mark.parametrize("width", [64, 129, 1000, 1021, 4096])
def test_a_row_for_all_tokens(norm, width):
    """Rows without a stride between them give what a copy gives, whatever kernel either takes, to the tolerances."""
    from lossless_bf16_exponent_zc_gb300 import dropout
    one = torch.randn((1, width), device="cuda").bfloat16().expand(300, width)
    x = torch.randn((300, width), device="cuda").bfloat16()
    w, rng, ws = torch.rand(width, device="cuda"), dropout.new_rng(4), norm.workspace(300, width)
    h, stats = norm.layer_norm(one, w, save=True)
    check_forward(h, stats, one.double(), torch.zeros_like(one, dtype=torch.float64), w, None)
    keep, factor = kept(300, width, 0.2, 4, 0, 0)
    z = torch.where(keep, one.double() * factor, 0.0) + x.double()
    x_new, h, stats = norm.add_layer_norm(one, x, w, p=0.2, rng=rng, save=True)
    off = 3 * U * (one.double().abs() * factor + x.double().abs())
    within(x_new, z, off)
    check_forward(h, stats, z, off, w, None)
    got = norm.add_layer_norm_backward(one, one, x_new, stats, w, ws, p=0.2, rng=rng)
    check_backward(got, one, one, x_new, stats, w, 1.0, keep, factor)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [40, 129, 1000, 1021, 4096, 9001])
def test_all_and_none_dropped(norm, dtype, width):
    """p = 1 leaves the residual, infinities and NaN in what is dropped too; a p that rounds to no step keeps all."""
    from lossless_bf16_exponent_zc_gb300 import dropout
    x, dh = (torch.randn((9, width), device="cuda").to(dtype) for _ in range(2))
    y = torch.full_like(x, float("nan"))
    y[::2] = float("inf")
    w, rng, ws = torch.rand(width, device="cuda"), dropout.new_rng(5), norm.workspace(9, width)
    x_new, h, stats = norm.add_layer_norm(y, x, w, p=1.0, rng=rng, save=True)
    assert torch.equal(x_new, x) and torch.equal(h, norm.layer_norm(x, w)[0])
    g = norm.add_layer_norm_backward(None, dh, x_new, stats, w, ws, p=1.0, rng=rng)
    assert not g.dy.any() and torch.equal(g.dx, norm.layer_norm_backward(dh, x, stats, w, ws)[0])
    for a, b in zip(norm.add_layer_norm(dh, x, w, p=1e-7, rng=rng), norm.add_layer_norm(dh, x, w)):
        assert a is b or torch.equal(a, b)
    g = norm.add_layer_norm_backward(None, dh, x_new, stats, w, ws, p=1e-7, rng=rng)
    assert torch.equal(g.dy, g.dx)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [65, 520, 1021, 1531, 4081])
def test_many_rows_a_walker(norm, dtype, width):
    """Odd widths over more rows than a walker draws ahead for (32), every row against dropout.dropout's mask."""
    from lossless_bf16_exponent_zc_gb300 import dropout
    rows = 40 * 1300 if width < 1000 else 40 * 650
    y = torch.ones((1, width), device="cuda").to(dtype).expand(rows, width).contiguous()
    x, w, rng = torch.zeros_like(y), torch.ones(width, device="cuda"), dropout.new_rng(77, 5)
    mask = dropout.dropout(y, 0.5, rng, 4)
    x_new, _, stats = norm.add_layer_norm(y, x, w, p=0.5, rng=rng, call=4, save=True)
    assert torch.equal(x_new, mask)
    g = norm.add_layer_norm_backward(y, x, x_new, stats, w, norm.workspace(rows, width), p=0.5, rng=rng, call=4)
    assert torch.equal(g.dy, mask) and torch.equal(g.dx, y)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(40, 2049), (2500, 2049), (40, 3001), (2500, 3001), (1000, 3066), (2431, 1536),
                                        (2600, 1536), (2600, 2560), (2433, 4096), (6000, 520), (5000, 385), (1000, 3200)])
@pytest.mark.parametrize("p", [0.0, 0.35])
def test_shapes_for_few_and_many_rows(norm, dtype, rows, width, p):
    """A walker has one row, several or many of them, in CTAs of all sizes."""
    from lossless_bf16_exponent_zc_gb300 import dropout
    g = torch.Generator(device="cuda").manual_seed(rows)
    y, x, dh, past = (torch.randn((rows, width), device="cuda", generator=g).to(dtype) for _ in range(4))
    w, b = (torch.randn(width, device="cuda", generator=g) for _ in range(2))
    keep, factor = kept(rows, width, p, width, rows, 3) if p else (None, 1.0)
    kw = dict(p=p, rng=dropout.new_rng(width, rows) if p else None, call=3)
    x_new, h, stats = norm.add_layer_norm(y, x, w, b, save=True, **kw)
    branch = y.double() * (keep * factor if p else 1.0)
    want = x.double() + branch
    off = 3 * U * (x.double().abs() + branch.abs())
    within(x_new, want, off)
    check_forward(h, stats, want, off, w, b)
    got = norm.add_layer_norm_backward(past, dh, x_new, stats, w, norm.workspace(rows, width), **kw)
    check_backward(got, past, dh, x_new, stats, w, 1.0, keep, factor)
    alone, stats = norm.layer_norm(x, w, b, save=True)
    check_forward(alone, stats, x.double(), torch.zeros_like(x, dtype=torch.float64), w, b)


def test_no_tokens(norm):
    x, w = torch.zeros((0, 40), device="cuda"), torch.ones(40, device="cuda")
    h, stats = norm.layer_norm(x, w, save=True)
    assert h.shape == (0, 40) and stats.shape == (0, 2)
    dx, dw, db = norm.layer_norm_backward(x, x, stats, w, norm.workspace(0, 40))
    assert dx.shape == (0, 40) and not dw.any() and not db.any()


def test_more_than_2_31_values(norm):
    rows, width = 530000, 4100
    x = torch.randn((1, width), device="cuda").bfloat16().expand(rows, width)
    w = torch.ones(width, device="cuda")
    h, stats = norm.layer_norm(x, w, eps=EPS, save=True)
    check_forward(h[-2:], stats[-2:], x[-2:].double(), torch.zeros((2, width), dtype=torch.float64, device="cuda"), w, None)
    assert torch.equal(h[0], h[-1])
