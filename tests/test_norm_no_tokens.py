"""zc_norm and zc_norm_backward without tokens, at the C ABI: tensors without rows may be NULL, and the sums over no
tokens are zero."""
import ctypes

import pytest

from lossless_bf16_exponent_zc_gb300 import zc
from test_layer_args import NormBackwardArgs, prototypes  # noqa: F401  (the fixture sets the prototypes)


def args(**kw):
    a = NormBackwardArgs()
    a.hidden, a.eps, a.dtype = 16, 1e-6, 0
    for n, v in kw.items():
        setattr(a, n, v)
    return ctypes.byref(a)


def test_nothing_to_do():
    lib = zc.load()
    some = 0x10000  # never looked at: no such output was asked for
    assert lib.zc_norm_backward(args(), None) == zc.OK
    assert lib.zc_norm_backward(args(weight=some, next_weight=some, gate=some, gate_rows=5), None) == zc.OK
    assert lib.zc_norm_backward(args(hidden=0), None) == zc.ERR_INVALID_ARG
    assert lib.zc_norm_backward(args(dtype=9), None) == zc.ERR_INVALID_ARG
    assert lib.zc_norm_backward(args(hidden=1 << 20), None) == zc.ERR_TOO_LARGE
    assert lib.zc_norm_backward(args(dweight=some + 1, weight=some), None) == zc.ERR_ALIGNMENT


@pytest.mark.gpu
@pytest.mark.parametrize("params_f32", [0, 1])
@pytest.mark.parametrize("gate_wide,gate_rows", [(1, 1), (1, 7), (1, 70000), (0, 70000)])
def test_sums_over_no_tokens(zc, gate_wide, gate_rows, params_f32):
    import torch
    hidden, dt = 16, torch.float32 if params_f32 else torch.bfloat16
    width = hidden if gate_wide else 1
    grads = {"dweight": hidden, "dnext_weight": hidden, "dgate": gate_rows * width}
    # a value behind each that has to stay
    out = {n: torch.full((size + 1,), 3.0, dtype=dt, device="cuda") for n, size in grads.items()}
    ins = {n: torch.ones(grads["d" + n], dtype=dt, device="cuda") for n in ("weight", "next_weight", "gate")}
    a = args(gate_rows=gate_rows, gate_wide=gate_wide, params_f32=params_f32,
             **{n: t.data_ptr() for n, t in [*out.items(), *ins.items()]})
    assert zc.load().zc_norm_backward(a, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == zc.OK
    for n, size in grads.items():
        assert not out[n][:size].any() and float(out[n][size]) == 3.0
