"""The router's gradient for experts that the router cannot have chosen, and its values row by row."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

FORMS = [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)]


@pytest.mark.parametrize("score,renormalize", FORMS)
@pytest.mark.parametrize("experts", [5, 40, 300])
def test_closed_experts_pass_nothing_on(zc, score, renormalize, experts):
    """Ids from before a mask was laid over the logits: an expert whose logit is -inf is one that the router does not
    choose, so its weight's gradient goes nowhere, also where no expert is left open, and whatever it is."""
    from lossless_bf16_exponent_zc_gb300 import moe
    g = torch.Generator(device="cuda").manual_seed(experts)
    logits = torch.randn((4, experts), device="cuda", generator=g)
    _, ids = moe.route(logits, 3, score=score, renormalize=renormalize)
    dw = torch.randn((4, 3), device="cuda", generator=g)
    masked = logits.clone()
    masked[0] = -math.inf                              # nothing open
    masked[1, ids[1, 1].long()] = -math.inf            # one of the three closed
    masked[2, ids[2].long()] = -math.inf               # all three closed, others open
    dw[1, 1] = math.inf
    got = moe.route_backward(dw, masked, ids, score=score, renormalize=renormalize)
    open_ids = torch.where(masked.gather(1, ids.long()) == -math.inf, -1, ids)
    want = moe.route_backward(torch.where(open_ids < 0, 0.0, dw), masked, open_ids, score=score, renormalize=renormalize)
    assert torch.equal(got, want) and torch.isfinite(got).all()
    assert not got[0].any() and not got[2].any()
    assert torch.equal(got[3], moe.route_backward(dw, logits, ids, score=score, renormalize=renormalize)[3])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("renormalize", [False, True])
def test_the_gradient_of_saturated_sigmoids(zc, dtype, renormalize):
    """Chosen logits up to 60 either way, where a sigmoid s is 1 to fp32 from 17 on: s (1 - s) keeps its relative error.  With
    u = 2^-24 it is off by 12 u (an exponential, a reciprocal and four operations), the sums over k = 4 slots by 20 u more
    of their magnitudes: below 60 u of s (1 - s) times those in all, and half a step of the output."""
    from lossless_bf16_exponent_zc_gb300 import moe
    g = torch.Generator(device="cuda").manual_seed(5)
    tokens, n, k = 200, 24, 4
    logits = (torch.rand((tokens, n), device="cuda", generator=g) * 50 + 10).to(dtype)
    logits = torch.where(torch.rand((tokens, n), device="cuda", generator=g) < 0.3, -logits, logits)
    logits[0] = torch.linspace(10, 30, n, device="cuda").to(dtype)
    ids = torch.rand((tokens, n), device="cuda", generator=g).argsort(1)[:, :k].int()
    dw = torch.randn((tokens, k), device="cuda", generator=g) * 2.0**20
    got = moe.route_backward(dw, logits, ids, score="sigmoid", renormalize=renormalize).double()
    at, f = ids.long(), torch.finfo(dtype)
    l, d = logits.double().gather(1, at), dw.double()
    s, rest, size = torch.sigmoid(l), torch.sigmoid(-l), d.abs()
    if renormalize:
        z = s.sum(1, keepdim=True) + 1e-20
        d, size = (d - (d * s).sum(1, keepdim=True) / z) / z, (size + (size * s).sum(1, keepdim=True) / z) / z
    want, room = (torch.zeros_like(got).scatter_(1, at, s * rest * v) for v in (d, size))
    room = 60 * 2.0**-24 * room + f.eps / 2 * want.abs() + f.smallest_normal * f.eps
    past = want.abs() > f.max                                          # fp16: infinite
    assert bool((((got - want).abs() <= room) | past).all())
    assert bool(((logits > 17) & (want.abs() > room)).any())
