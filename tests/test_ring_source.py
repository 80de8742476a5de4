"""Source check of the ring kernels' sums over a CTA (no GPU), and many launches that do little but their first sum.

block_sum_shared() adds every slot of its buffer, those of absent warps too, so the buffer is cleared by all threads
before the first sum; a warp's slots are cleared by other warps.  Without a barrier of the whole CTA in between, a late
warp can clear a partial sum that another one has already left there.  A barrier that only some instances of the kernel
reach does not count.
"""
import os
import re

import pytest
import torch

from test_launch_contract import _kernels, _sources

RINGS = {name: body for _, text in _sources() for name, body in _kernels(text) if "block_sum_shared" in body}


def top_level(body):
    """The kernel's statements that every thread of every instance runs, as one text: nothing inside braces, and no
    statement that an if or a loop guards."""
    code = re.sub(r"//.*", "", body)
    flat, depth = [], 0
    for c in code:
        depth += c == "{"
        if depth == 0:
            flat.append(c)
        depth -= c == "}"
    statements = [s.strip() for s in "".join(flat).split(";")]
    return [s for s in statements if s and not re.match(r"(if|else|for|while)\b", s)]


@pytest.mark.parametrize("kernel", ["norm_ring_kernel", "norm_bwd_ring_kernel"])
def test_a_barrier_between_clearing_and_the_first_sum(kernel):
    body = RINGS[kernel]
    clear = body.index("red[0][i] = 0.f;")
    # the first sum is the first one behind the clearing, wherever its braces
    between = body[clear + len("red[0][i] = 0.f;"):]
    between = between[:between.index("block_sum_shared<")]
    assert "__syncthreads()" in top_level(between), "a late warp may clear a sum that is already there"


def test_the_kernels_are_found():
    assert set(RINGS) == {"norm_ring_kernel", "norm_bwd_ring_kernel"}


def test_the_check_itself():
    assert "__syncthreads()" in top_level("a(); __syncthreads(); b();")
    for guarded in ("if (kWords) __syncthreads();", "if (k) { __syncthreads(); }", "auto f = [&] { __syncthreads(); };"):
        assert "__syncthreads()" not in top_level("a(); " + guarded + " b();")


@pytest.mark.gpu
@pytest.mark.parametrize("hidden,dtype", [(4096, torch.bfloat16), (1531, torch.bfloat16), (4095, torch.float32)])
def test_first_sums_of_many_launches(zc, hidden, dtype):
    """A row or two a CTA, so that the first sum is most of the work, 300 times: the same bits."""
    from lossless_bf16_exponent_zc_gb300 import norm
    g = torch.Generator(device="cuda").manual_seed(hidden)
    y, x, gx, gh = (torch.randn((305, hidden), device="cuda", generator=g).to(dtype) for _ in range(4))
    w = torch.rand(hidden, device="cuda", generator=g) + 0.5
    ws = norm.workspace(305, hidden)
    first = norm.post_norm_backward(gx, gh, y, x, w, ws, next_weight=w)
    for _ in range(300):
        again = norm.post_norm_backward(gx, gh, y, x, w, ws, next_weight=w)
        for a, b in zip(first, again):
            assert a is b or torch.equal(a, b)
