"""Sizes beyond 32 bits are refused, not cut to their low 32 (no GPU: fake tensors, refused before anything is made)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from lossless_bf16_exponent_zc_gb300 import moe, norm, zc

WIDE = 2 ** 32 + 8  # its low 32 bits are 8


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda")


def ids(*shape):
    return empty(*shape, dtype=torch.int32)


def f32(*shape):
    return empty(*shape, dtype=torch.float32)


CALLS = {
    "route": lambda: moe.route(empty(1, WIDE), 2),
    "route_backward": lambda: moe.route_backward(f32(1, 2), empty(1, WIDE), ids(1, 2)),
    "route_backward-k": lambda: moe.route_backward(f32(1, WIDE), empty(1, 64), ids(1, WIDE)),
    "dispatch": lambda: moe.dispatch(empty(1, WIDE), ids(1, 2), 4, empty(64, dtype=torch.uint8)),
    "dispatch-k": lambda: moe.dispatch(empty(1, 16), ids(1, WIDE), 64, empty(64, dtype=torch.uint8)),
    "dispatch_backward": lambda: moe.dispatch_backward(empty(2, WIDE), ids(1, 2), ids(1)),
    "combine": lambda: moe.combine(empty(2, WIDE), f32(1, 2), ids(1, 2), ids(1)),
    "combine-k": lambda: moe.combine(empty(2, 16), f32(1, WIDE), ids(1, WIDE), ids(1)),
    "combine_backward": lambda: moe.combine_backward(empty(1, WIDE), empty(2, WIDE), f32(1, 2), ids(1, 2), ids(1)),
    "combine_backward-k": lambda: moe.combine_backward(empty(1, 16), empty(2, 16), f32(1, WIDE), ids(1, WIDE), ids(1)),
}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS.keys())
def test_too_wide(call):
    with FakeTensorMode(), pytest.raises(zc.ZcError) as e:
        call()
    assert e.value.code == zc.ERR_TOO_LARGE


@pytest.mark.gpu
def test_too_wide_without_rows(zc):
    """The same widths of matrices without rows, which take no memory."""
    st = zc.new_status()
    none, no_ids = empty(0, WIDE), ids(0, 2)
    for call in (lambda: moe.route(none, 2), lambda: moe.route_backward(f32(0, 2), none, no_ids),
                 lambda: moe.dispatch(none, no_ids, 4, moe.workspace(0, 2, 4)),
                 lambda: moe.combine(none, f32(0, 2), no_ids, st), lambda: moe.dispatch_backward(none, no_ids, st),
                 lambda: moe.combine_backward(none, none, f32(0, 2), no_ids, st)):
        with pytest.raises(zc.ZcError) as e:
            call()
        assert e.value.code == zc.ERR_TOO_LARGE
    with pytest.raises((zc.ZcError, ValueError)):
        norm.pre_norm(none, f32(8))
