"""All tensors of a call lie on one device (no GPU: fake tensors stand in for those of two, and are refused before
anything looks at their memory)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from lossless_bf16_exponent_zc_gb300 import moe, norm

TOKENS, K, EXPERTS, HIDDEN = 6, 2, 4, 32


def tensors(device):
    """Every argument of the calls below, by name, on one device."""
    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=device)

    i32 = dict(dtype=torch.int32)
    return {"logits": empty(TOKENS, EXPERTS), "bias": empty(EXPERTS), "weights": empty(TOKENS, K),
            "experts": empty(TOKENS, K, **i32), "dlogits": empty(TOKENS, EXPERTS), "dweights": empty(TOKENS, K),
            "x": empty(TOKENS, HIDDEN), "y": empty(TOKENS, HIDDEN), "dout": empty(TOKENS, HIDDEN),
            "dh": empty(TOKENS, HIDDEN), "out": empty(TOKENS, HIDDEN), "h": empty(TOKENS, HIDDEN),
            "rows": empty(TOKENS * K, HIDDEN), "drows": empty(TOKENS * K, HIDDEN),
            "positions": empty(TOKENS, K, **i32), "status": empty(1, **i32), "w": empty(HIDDEN), "w2": empty(HIDDEN),
            "gate": empty(3, HIDDEN), "ws": empty(1 << 16, dtype=torch.uint8)}


CALLS = {
    "route": (lambda t: moe.route(t["logits"], K, score="sigmoid", bias=t["bias"], weights=t["weights"],
                                  experts=t["experts"]), ("logits", "bias", "weights", "experts")),
    "route_backward": (lambda t: moe.route_backward(t["dweights"], t["logits"], t["experts"], dlogits=t["dlogits"]),
                       ("dweights", "logits", "experts", "dlogits")),
    "dispatch": (lambda t: moe.dispatch(t["x"], t["experts"], EXPERTS, t["ws"], rows=t["rows"]),
                 ("x", "experts", "ws", "rows")),
    "dispatch_backward": (lambda t: moe.dispatch_backward(t["drows"], t["positions"], t["status"], dx=t["out"]),
                          ("drows", "positions", "status", "out")),
    "combine": (lambda t: moe.combine(t["rows"], t["weights"], t["positions"], t["status"], out=t["out"]),
                ("rows", "weights", "positions", "status", "out")),
    "combine_backward": (lambda t: moe.combine_backward(t["dout"], t["rows"], t["weights"], t["positions"], t["status"],
                                                        drows=t["drows"], dweights=t["dweights"]),
                         ("dout", "rows", "weights", "positions", "status", "drows", "dweights")),
    "pre_norm": (lambda t: norm.pre_norm(t["x"], t["w"], out=t["out"]), ("x", "w", "out")),
    "pre_norm_backward": (lambda t: norm.pre_norm_backward(t["dh"], t["x"], t["w"], t["ws"], dresidual=t["dout"]),
                          ("dh", "x", "w", "ws", "dout")),
    "post_norm": (lambda t: norm.post_norm(t["y"], t["x"], t["w"], gate=t["gate"], next_weight=t["w2"], x_new=t["out"],
                                           h=t["h"]), ("y", "x", "w", "gate", "w2", "out", "h")),
    "post_norm_backward": (lambda t: norm.post_norm_backward(t["dout"], t["dh"], t["y"], t["x"], t["w"], t["ws"],
                                                             gate=t["gate"], next_weight=t["w2"]),
                           ("dout", "dh", "y", "x", "w", "ws", "gate", "w2")),
}


@pytest.mark.parametrize("call,names,other", [(c, n, o) for c, n in CALLS.values() for o in n],
                         ids=[f"{c}-{o}" for c, (_, n) in CALLS.items() for o in n])
def test_a_tensor_on_another_device(monkeypatch, call, names, other):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)  # or fake tensors first try the device they name
    with FakeTensorMode():
        here, there = tensors("cuda:0"), tensors("cuda:1")
        with pytest.raises(ValueError, match="device"):
            call({**here, other: there[other]})


@pytest.mark.gpu
def test_a_stream_of_another_device(zc):
    class Elsewhere:
        cuda_stream, device_index = 0, 1

    with pytest.raises(ValueError, match="device"):
        norm.pre_norm(torch.zeros((2, 8), device="cuda:0"), torch.ones(8, device="cuda:0"), stream=Elsewhere())

    class Plain:  # a handle alone is taken to be of the tensors' device
        cuda_stream = torch.cuda.current_stream().cuda_stream

    x = torch.randn((2, 8), device="cuda:0")
    assert torch.equal(norm.pre_norm(x, torch.ones(8, device="cuda:0"), stream=Plain()),
                       norm.pre_norm(x, torch.ones(8, device="cuda:0")))
    assert torch.cuda.current_device() == 0
