"""The router's balance loss against its definition in 64 bits, both directions; the counts exactly.

Tolerances, with u = 2^-24: a probability takes an exponential of at most 32 in magnitude (its argument's rounding 32 u),
a sum of up to 32 + 5 terms and a few operations, 100 u in all; the loss adds at most `tokens` of them.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0**-24
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def moe(zc):
    from lossless_bf16_exponent_zc_gb300 import moe
    return moe


def reference(logits, experts, dloss, score, sequences, mask):
    l = logits.double()
    valid = ~(l == -math.inf).all(1)
    if mask is not None:
        valid &= mask.bool()
    tokens, n = l.shape
    k = experts.shape[1]
    l = torch.where(valid[:, None], l, 0.0).requires_grad_(True)
    p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l) / (torch.sigmoid(l).sum(1, keepdim=True) + 1e-20)
    counts = torch.zeros((sequences, n), dtype=torch.int32, device="cuda")
    slope = torch.zeros((sequences, n), dtype=torch.float64, device="cuda")
    loss = 0.0
    for s in range(sequences):
        at = slice(s * tokens // sequences, (s + 1) * tokens // sequences)
        v, ids = valid[at], experts[at][valid[at]]
        ids = ids[(ids >= 0) & (ids < n)].long()
        counts[s] = torch.bincount(ids, minlength=n)
        t = int(v.sum())
        if t:
            slope[s] = n * counts[s].double() / (sequences * k * t * t)
        loss = loss + (slope[s].clone() * (p[at] * v[:, None]).sum(0)).sum()
    g, = torch.autograd.grad(loss, l, dloss.double()) if tokens else (l.detach(),)
    return loss.detach(), counts, slope, g, p.detach() * valid[:, None]


def check(moe, logits, experts, score="softmax", sequences=1, mask=None, dloss=1.0):
    dloss = torch.tensor(dloss, device="cuda")
    tokens, n = logits.shape
    ws = moe.balance_workspace(tokens, n, sequences)
    ws.fill_(0xA5)                                                      # needs no initialisation
    got = moe.balance_loss(logits, experts, ws, score=score, sequences=sequences, mask=mask)
    d = moe.balance_loss_backward(dloss, logits, got.slope, score=score, mask=mask)
    loss, counts, slope, g, p = reference(logits, experts, dloss, score, sequences, mask)
    assert torch.equal(got.counts, counts)
    assert bool(((got.slope.double() - slope).abs() <= 8 * U * slope).all())
    assert abs(float(got.loss.double() - loss)) <= (tokens + 140) * U * float(loss)
    c = slope.repeat_interleave(max(tokens // sequences, 1), 0)[:tokens]
    mean = (c * p).sum(1, keepdim=True)
    f = torch.finfo(logits.dtype)
    room = abs(float(dloss)) * p * (c + mean) * 250 * U + f.eps / 2 * g.abs() + f.smallest_normal * f.eps
    assert bool(((d.double() - g).abs() <= room).all())
    again = moe.balance_loss(logits, experts, ws, score=score, sequences=sequences, mask=mask)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    return got


def make(tokens, n, k, dtype, masked=0.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn((tokens, n), device="cuda", generator=g) * 2
    shut = torch.rand((tokens, n), device="cuda", generator=g) < masked
    logits = torch.where(shut, -math.inf, logits).to(dtype)
    ids = torch.randint(-1, n + 1, (tokens, k), device="cuda", generator=g, dtype=torch.int32)  # n: beyond the experts
    return logits, ids


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,n,k", [(1, 1, 1), (3, 2, 2), (40, 31, 3), (7, 32, 1), (64, 33, 4), (129, 64, 2), (200, 100, 6),
                                        (333, 128, 8), (50, 255, 5), (300, 256, 8), (97, 300, 4), (65, 512, 32), (33, 1000, 7),
                                        (40, 1024, 3)])
def test_values(moe, score, dtype, tokens, n, k):
    check(moe, *make(tokens, n, k, dtype, seed=n), score=score, dloss=float(tokens))
    check(moe, *make(tokens, n, k, dtype, 0.6, seed=n), score=score, dloss=-0.5 * tokens)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,sequences", [(12, 12), (60, 5), (4000, 40), (5000, 2), (3000, 3000), (40000, 1)])
def test_sequences_and_masks(moe, score, tokens, sequences):
    logits, ids = make(tokens, 20, 3, torch.float32, 0.3, tokens)
    logits[tokens // 2] = -math.inf
    mask = torch.rand(tokens, device="cuda") < 0.7
    mask[:tokens // sequences] = False                                  # a sequence of padding alone
    check(moe, logits, ids, score, sequences, mask, 10.0)
    check(moe, logits, ids, score, sequences, mask.to(torch.uint8) * 255, 10.0)
    check(moe, logits, ids, score, sequences, None, 10.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_even_load_costs_one(moe, score):
    tokens, n = 96, 16
    ids = torch.arange(tokens * 2, device="cuda", dtype=torch.int32).view(tokens, 2) % n
    assert abs(float(check(moe, torch.zeros((tokens, n), device="cuda"), ids, score).loss) - 1) < 1e-5


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_padding_may_hold_anything(moe, score):
    logits, ids = make(100, 24, 4, torch.bfloat16)
    mask = torch.arange(100, device="cuda") % 3 != 0
    clean = check(moe, logits, ids, score, 4, mask)
    for rubbish in (math.nan, math.inf, -math.inf, 1e30):
        dirty = torch.where(mask[:, None], logits, rubbish)
        got = moe.balance_loss(dirty, ids, moe.balance_workspace(100, 24, 4), score=score, sequences=4, mask=mask)
        assert all(torch.equal(a, b) for a, b in zip(got, clean))
        d = moe.balance_loss_backward(torch.ones((), device="cuda"), dirty, got.slope, score=score, mask=mask)
        assert not d[~mask].any() and bool(torch.isfinite(d).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_logits_of_the_lowest_value_are_open(moe, dtype):
    """Masks of the type's lowest value are logits like others: a row of them alone is uniform, one beside others nothing."""
    logits, ids = make(40, 24, 3, dtype)
    logits[::3] = torch.finfo(dtype).min
    logits[1::3, 5:] = torch.finfo(dtype).min
    got = check(moe, logits, ids)
    assert int(got.counts.sum()) == int(((ids >= 0) & (ids < 24)).sum())


def test_a_nan_that_counts_shows(moe):
    logits, ids = make(50, 24, 4, torch.float32)
    logits[7, 3] = math.nan
    got = moe.balance_loss(logits, ids, moe.balance_workspace(50, 24))
    d = moe.balance_loss_backward(torch.ones((), device="cuda"), logits, got.slope)
    assert bool(torch.isnan(got.loss)) and bool(torch.isnan(d[7]).all()) and int(torch.isnan(d).any(1).sum()) == 1
    assert int(got.counts.sum()) == int(((ids >= 0) & (ids < 24)).sum())


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("n", [61, 64])
def test_strides_and_alignment(moe, shift, n):
    wide, ids = make(70, n + 7, 3, torch.bfloat16)
    ids = ids.clamp(max=n)
    check(moe, wide[:, shift:shift + n], ids)
    check(moe, wide[:1, shift:shift + n].expand(70, n), ids, "sigmoid")


def test_nothing_counts(moe):
    ids = torch.zeros((0, 2), device="cuda", dtype=torch.int32)
    got = moe.balance_loss(torch.zeros((0, 5), device="cuda"), ids, moe.balance_workspace(0, 5, 3), sequences=3)
    assert float(got.loss) == 0 and not got.counts.any() and not got.slope.any() and got.counts.shape == (3, 5)
    assert moe.balance_loss_backward(got.loss, torch.zeros((0, 5), device="cuda"), got.slope).shape == (0, 5)
    check(moe, torch.full((9, 5), -math.inf, device="cuda"), torch.zeros((9, 2), device="cuda", dtype=torch.int32))
    check(moe, torch.randn((9, 5), device="cuda"), torch.zeros((9, 2), device="cuda", dtype=torch.int32),
          mask=torch.zeros(9, dtype=torch.bool, device="cuda"))


def test_gradient_against_differences(moe):
    """The loss of logits moved by 2^-6 either way along the gradient, in fp32, its counts fixed: differences are good to
    the third derivative's 2^-12 and the loss's own rounding over the step."""
    logits, ids = make(60, 12, 2, torch.float32, seed=3)
    ws = moe.balance_workspace(60, 12)
    for score in ("softmax", "sigmoid"):
        got = moe.balance_loss(logits, ids, ws, score=score)
        d = moe.balance_loss_backward(torch.ones((), device="cuda"), logits, got.slope, score=score)
        along = d / d.norm()
        up, down = (float(moe.balance_loss(logits + s * along, ids, ws, score=score).loss) for s in (2**-6, -2**-6))
        assert abs((up - down) / 2**-5 - float((d * along).sum())) < 2**-12 * float(d.norm()) + 200 * U * 2**5


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [8, 61, 300, 1024])
def test_the_gradient_of_saturated_sigmoids(moe, dtype, n):
    """Logits up to 60 either way, where s is 1 to fp32 from 17 on: s (1 - s) keeps its relative error.  With u = 2^-24: of
    s (1 - s) 12 u (an exponential, a reciprocal and four operations), of the sigmoids' sum 45 u (32 + 5 terms of 4 u), of
    the mean slope 90 u more; below 250 u of s (1 - s) / Z (c + mean) in all, and half a step of the output.  So a value
    larger than its room cannot be zero; one in whose row c and the mean agree to 250 u may be."""
    g = torch.Generator(device="cuda").manual_seed(n)
    logits = (torch.rand((120, n), device="cuda", generator=g) * 50 + 10).to(dtype)
    logits = torch.where(torch.rand((120, n), device="cuda", generator=g) < 0.3, -logits, logits)
    logits[0] = torch.linspace(10, 30, n, device="cuda").to(dtype)
    ids = torch.randint(0, n, (120, 3), device="cuda", generator=g, dtype=torch.int32)
    ws, dloss = moe.balance_workspace(120, n), torch.tensor(2.0**40, device="cuda")  # normal numbers up to logits of 60
    slope = moe.balance_loss(logits, ids, ws, score="sigmoid").slope
    d = moe.balance_loss_backward(dloss, logits, slope, score="sigmoid").double()
    l, c = logits.double(), slope.double()
    s, rest = torch.sigmoid(l), torch.sigmoid(-l)
    z = s.sum(1, keepdim=True) + 1e-20
    mean = (s / z * c).sum(1, keepdim=True)
    want, f = 2.0**40 * s * rest / z * (c - mean), torch.finfo(dtype)
    room = 2.0**40 * s * rest / z * (c + mean) * 250 * U + f.eps / 2 * want.abs() + f.smallest_normal * f.eps
    past = want.abs() > f.max                                          # fp16: infinite
    assert bool((((d - want).abs() <= room) | past).all())
    assert bool(((logits > 17) & (want.abs() > room)).any())           # what a difference from 1 makes zero
    logits[1::2] = math.inf
    ends = moe.balance_loss_backward(dloss, logits, slope, score="sigmoid")
    assert not ends[1::2].any() and torch.equal(ends[::2].double(), d[::2])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,n,k,sequences,dtype", [(81920, 20, 2, 1, torch.bfloat16), (77825, 130, 3, 1, torch.float16),
                                                        (84000, 33, 2, 7, torch.float32), (40001, 1024, 2, 1, torch.bfloat16),
                                                        (39000, 600, 4, 2, torch.float32), (250000, 8, 1, 1250, torch.float32)])
def test_many_tokens(moe, score, tokens, n, k, sequences, dtype):
    """Chunks of more tokens than the shortest, in one sequence and in several, and more sequences than chunks."""
    check(moe, *make(tokens, n, k, dtype, 0.2, seed=n), score=score, sequences=sequences, dloss=float(tokens))


def test_a_workspace_for_the_largest_batch_serves_smaller_ones(moe):
    """Fewer tokens may have more chunks: 77824 have the most."""
    logits, ids = make(90112, 40, 2, torch.float32)
    ws = moe.balance_workspace(90112, 40, 8)
    for tokens, sequences in ((90112, 1), (77824, 1), (81920, 8), (77824, 4), (1024, 8), (512, 1), (90112, 8)):
        want = check(moe, logits[:tokens], ids[:tokens], sequences=sequences)
        got = moe.balance_loss(logits[:tokens], ids[:tokens], ws, sequences=sequences)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 31, 32, 61, 64, 100, 128, 250, 256, 400, 512])
@pytest.mark.parametrize("tokens,sequences", [(1025, 1), (1400, 7), (600, 3)])
def test_widths_of_the_two_launches(moe, score, dtype, n, tokens, sequences):
    """Every number of experts a lane, in pieces and one at a time, past what one cluster takes."""
    check(moe, *make(tokens, n, min(n, 5), dtype, 0.3, seed=n), score=score, sequences=sequences, dloss=float(tokens))
