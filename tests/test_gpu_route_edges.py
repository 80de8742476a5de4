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
