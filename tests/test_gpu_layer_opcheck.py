"""torch.ops.zc's layer operators under torch's own checks (schema, fake outputs, autograd, traced with fixed and with
symbolic sizes), and the gradients of an empty batch: a rank that gets no tokens still takes its step."""
import pytest
import torch

from lossless_bf16_exponent_zc_gb300 import torch_ops  # noqa: F401  (registers torch.ops.zc)

pytestmark = pytest.mark.gpu
ops = torch.ops.zc


def leaf(*shape, dtype=torch.float32, grad=True):
    return torch.randn(shape, device="cuda").to(dtype).requires_grad_(grad)


def calls(tokens, dtype):
    """name -> (op, arguments)"""
    ids = torch.randint(-1, 4, (tokens, 2), device="cuda", dtype=torch.int32)
    positions = ops.moe_dispatch(leaf(tokens, 24, dtype=dtype, grad=False), ids, 4)[1]

    def act():
        return leaf(tokens, 24, dtype=dtype)

    return {"route": (ops.moe_route, (leaf(tokens, 9, dtype=dtype), None, 3, "softmax", True, 1.0)),
            "route_sigmoid": (ops.moe_route, (leaf(tokens, 9, dtype=dtype), leaf(9, grad=False), 3, "sigmoid", False, 2.0)),
            "dispatch": (ops.moe_dispatch, (act(), ids, 4)),
            "combine": (ops.moe_combine, (leaf(tokens * 2, 24, dtype=dtype), leaf(tokens, 2), positions)),
            "combine_more_rows": (ops.moe_combine, (leaf(tokens * 2 + 3, 24, dtype=dtype), leaf(tokens, 2), positions)),
            "pre_norm": (ops.pre_norm, (act(), leaf(24), 1e-6)),
            "post_norm": (ops.post_norm, (act(), act(), leaf(24), leaf(3, 24), 0.5, 1e-6)),
            "post_pre_norm": (ops.post_pre_norm, (act(), act(), leaf(24), None, leaf(24), 0.5, 1e-6)),
            "post_pre_norm_gate": (ops.post_pre_norm, (act(), act(), leaf(24), leaf(1, 1), leaf(24), 0.5, 1e-6))}


NAMES = ["route", "route_sigmoid", "dispatch", "combine", "combine_more_rows", "pre_norm", "post_norm", "post_pre_norm",
         "post_pre_norm_gate"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("tokens,dtype", [(6, torch.bfloat16), (0, torch.float32)])
def test_opcheck(zc, name, tokens, dtype):
    op, args = calls(tokens, dtype)[name]
    torch.library.opcheck(op, args)


@pytest.mark.parametrize("name", NAMES)
def test_gradients_of_an_empty_batch(zc, name):
    """Through a sum, whose gradient comes expanded, with strides of its own."""
    op, args = calls(0, torch.bfloat16)[name]
    out = op(*args)
    out = out if isinstance(out, tuple) else (out,)
    sum(o.float().sum() for o in out if o.requires_grad).backward()
    for a in args:
        if isinstance(a, torch.Tensor) and a.requires_grad:
            assert a.grad.shape == a.shape and not a.grad.any()


def test_empty_matrices_of_any_strides(zc):
    from lossless_bf16_exponent_zc_gb300 import moe, norm
    none = torch.zeros((24, 0), device="cuda").t()         # no rows, columns not next to one another
    far = torch.empty_strided((0, 24), (2 ** 41, 3), device="cuda")
    w = torch.ones(24, device="cuda")
    for x in (none, far):
        assert norm.pre_norm(x, w).shape == (0, 24) and moe.route(x, 2)[0].shape == (0, 2)
        assert norm.post_norm(x, x, w, next_weight=w)[1].shape == (0, 24)
        rows, plan = moe.dispatch(x, torch.zeros((0, 2), dtype=torch.int32, device="cuda"), 4, moe.workspace(0, 2, 4))
        assert rows.shape == (0, 24) and not plan.offsets.any()
        assert moe.combine(x, torch.zeros((0, 2), device="cuda"), plan.positions, zc.new_status()).shape == (0, 24)
