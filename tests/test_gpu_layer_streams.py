"""The operators around an expert-parallel exchange on a stream that is given (``stream=``), and from several threads.

A block of the caching allocator may be written only on the stream it was allocated for: its last reader there may still
be queued.  So a call's outputs have to come from the pool of the stream it launches on, and a caller who uses and drops
them on the stream that was current has to find them whole.
"""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

TOKENS, K, EXPERTS, HIDDEN = 700, 3, 12, 264
CYCLES = 30_000_000  # about 15 ms of a sleeping kernel in front of a queued reader


@pytest.fixture(scope="module")
def calls(zc):
    """name -> call(stream=...) of every entry point, its tensor outputs in a list."""
    from lossless_bf16_exponent_zc_gb300 import moe, norm
    g = torch.Generator(device="cuda").manual_seed(5)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    logits, x, y, gx = randn(TOKENS, EXPERTS), *(randn(TOKENS, HIDDEN).bfloat16() for _ in range(3))
    w, gate = randn(HIDDEN), randn(7, HIDDEN)
    st = zc.new_status()
    weights, experts = moe.route(logits, K)
    ws, nws = moe.workspace(TOKENS, K, EXPERTS), norm.workspace(TOKENS, HIDDEN)
    rows, plan = moe.dispatch(x, experts, EXPERTS, ws)

    def backward(stream=None):
        return norm.post_norm_backward(gx, gx, y, x, w, nws, gate=gate, next_weight=w, stream=stream)

    def none(stream=None):  # no tokens: the gradients are zeros that no kernel of ours writes
        return norm.post_norm_backward(gx[:0], gx[:0], y[:0], x[:0], w, nws, gate=gate, next_weight=w, stream=stream)

    def flat(r):
        if torch.is_tensor(r):
            return [r]
        return [t for part in r if part is not None for t in flat(part)]

    table = {
        "route": lambda **kw: moe.route(logits, K, **kw),
        "route_backward": lambda **kw: moe.route_backward(weights, logits, experts, **kw),
        "dispatch": lambda **kw: moe.dispatch(x, experts, EXPERTS, ws, **kw),
        "dispatch_backward": lambda **kw: moe.dispatch_backward(rows, plan.positions, st, **kw),
        "combine": lambda **kw: moe.combine(rows, weights, plan.positions, st, **kw),
        "combine_backward": lambda **kw: moe.combine_backward(gx, rows, weights, plan.positions, st, **kw),
        "pre_norm": lambda **kw: norm.pre_norm(x, w, **kw),
        "pre_norm_backward": lambda **kw: norm.pre_norm_backward(gx, x, w, nws, **kw),
        "post_norm": lambda **kw: norm.post_norm(y, x, w, gate=gate, next_weight=w, **kw),
        "post_norm_backward": backward, "no_tokens": none,
    }
    torch.cuda.synchronize()
    return {name: (lambda stream=None, f=f: flat(f(stream=stream))) for name, f in table.items()}


NAMES = ["route", "route_backward", "dispatch", "dispatch_backward", "combine", "combine_backward", "pre_norm",
         "pre_norm_backward", "post_norm", "post_norm_backward", "no_tokens"]


def pool_of(t):
    """The stream that the allocator keeps a tensor's block for."""
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= t.data_ptr() < segment["address"] + segment["total_size"]:
            return segment["stream"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_belong_to_the_given_stream(calls, name):
    want = calls[name]()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = calls[name](stream=side)
    assert torch.cuda.current_stream() != side         # the caller's stream is current again
    for t in got:
        assert t.numel() == 0 or pool_of(t) == side.cuda_stream
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for t in calls[name](stream=torch.cuda.current_stream()):
        assert t.numel() == 0 or pool_of(t) == torch.cuda.current_stream().cuda_stream


def test_a_block_with_a_queued_reader_is_left_alone(calls):
    """On the current stream a reader of a dropped tensor is still queued when the given stream writes its output."""
    want = calls["combine"]()[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = torch.full_like(want, 7.0)
    torch.cuda._sleep(CYCLES)
    seen = old.clone()
    del old                                            # the next block of this size on the current stream
    out = calls["combine"](stream=side)[0]
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert torch.equal(seen, torch.full_like(want, 7.0))


def test_a_dropped_output_is_not_written_again_too_early(calls):
    """The caller's stream still has to read an output when it is dropped and the given stream makes another."""
    want = calls["combine"]()[0]
    side, cur = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    out = calls["combine"](stream=side)[0]
    cur.wait_stream(side)
    torch.cuda._sleep(CYCLES)
    seen = out.clone()
    del out
    others = [calls["dispatch_backward"](stream=side)[0] for _ in range(3)]  # of the same size
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(seen, want) and not torch.equal(others[0], want)


def test_given_outputs_stay_the_callers(zc):
    from lossless_bf16_exponent_zc_gb300 import norm
    x, w = torch.randn((40, 96), device="cuda"), torch.rand(96, device="cuda")
    out, side = torch.empty_like(x), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert norm.pre_norm(x, w, out=out, stream=side) is out
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, norm.pre_norm(x, w))


def test_from_several_threads(zc):
    """Two threads, each on its own stream with its own workspaces, get what one gets."""
    from lossless_bf16_exponent_zc_gb300 import moe, norm

    def step(seed, rounds, out):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn((TOKENS, HIDDEN), device="cuda", generator=g).bfloat16()
        logits, w = torch.randn((TOKENS, EXPERTS), device="cuda", generator=g), torch.ones(HIDDEN, device="cuda")
        ws, nws, st = moe.workspace(TOKENS, K, EXPERTS), norm.workspace(TOKENS, HIDDEN), zc.new_status()
        for _ in range(rounds):
            weights, experts = moe.route(logits, K, score="sigmoid")
            rows, plan = moe.dispatch(x, experts, EXPERTS, ws)
            y = moe.combine(rows, weights, plan.positions, st)
            x_new, h = norm.post_norm(y, x, w, next_weight=w)
            out.append([rows, y, x_new, h, *norm.post_norm_backward(x, x, y, x_new, w, nws, next_weight=w)[:3]])
        torch.cuda.current_stream().synchronize()

    want = [[], []]
    for seed in (0, 1):
        step(seed, 1, want[seed])
    got, errors = [[], []], []

    def work(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                step(seed, 30, got[seed])
        except Exception as e:  # raised again by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(seed,)) for seed in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    torch.cuda.synchronize()
    for seed in (0, 1):
        assert len(got[seed]) == 30
        for run in got[seed]:
            for a, b in zip(run, want[seed][0]):
                assert torch.equal(a, b)
