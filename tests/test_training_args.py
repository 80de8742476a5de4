"""Argument checks of the balance loss, dropout, layer norms and embedding: the C ABI's codes (nothing is launched, no
GPU) and the Python entry points' refusals (fake tensors)."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from lossless_bf16_exponent_zc_gb300 import dropout, embedding, moe, norm, zc

VP, U64, U32, I32, F32, F64 = (ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int32, ctypes.c_float,
                               ctypes.c_double)


class LayerNormArgs(ctypes.Structure):
    _fields_ = [("y", VP), ("x", VP), ("y_stride", U64), ("x_stride", U64), ("tokens", U64), ("weight", VP), ("bias", VP),
                ("rng", VP), ("p", F64), ("call", U32), ("hidden", U32), ("dtype", I32), ("params_f32", I32),
                ("residual_scale", F32), ("eps", F32), ("x_new", VP), ("h", VP), ("stats", VP)]


class LayerNormBackwardArgs(ctypes.Structure):
    _fields_ = [("dx_new", VP), ("dh", VP), ("x_new", VP), ("dx_new_stride", U64), ("dh_stride", U64),
                ("x_new_stride", U64), ("tokens", U64), ("stats", VP), ("weight", VP), ("rng", VP), ("p", F64),
                ("call", U32), ("hidden", U32), ("dtype", I32), ("params_f32", I32), ("residual_scale", F32), ("dy", VP),
                ("dx", VP), ("dweight", VP), ("dbias", VP), ("ws", VP), ("ws_bytes", U64)]


F = 0x10000  # an aligned address that is never dereferenced: every call below is refused first


@pytest.fixture(scope="module", autouse=True)
def prototypes():
    lib = zc.load()
    lib.zc_moe_balance.argtypes = [VP, I32, U64, U64, U32, U32, VP, I32, U64, VP, VP, VP, VP, VP, U64, VP]
    lib.zc_moe_balance_backward.argtypes = [VP, VP, I32, U64, U64, U32, I32, U64, VP, VP, VP, VP]
    lib.zc_dropout.argtypes = [VP, I32, U64, VP, U64, F32, U64, U32, F64, VP, U32, VP, VP]
    lib.zc_layer_norm.argtypes = [ctypes.POINTER(LayerNormArgs), VP]
    lib.zc_layer_norm_backward.argtypes = [ctypes.POINTER(LayerNormBackwardArgs), VP]
    lib.zc_embedding.argtypes = [VP, I32, U64, VP, I32, I32, U64, U64, U32, F32, VP, VP, VP]
    lib.zc_embedding_backward.argtypes = [VP, I32, U64, VP, I32, U64, U64, U32, F32, I32, I32, VP, VP, U64, VP, VP]


def expect(call, code, cases):
    for kw in cases:
        assert call(**kw) == code, kw


def test_balance():
    need = moe.balance_workspace_size(12, 8, 3)

    def call(logits=F, dtype=2, stride=8, tokens=12, experts=8, k=2, ids=F, score=0, sequences=3, mask=F, loss=F, counts=F,
             slope=F, ws=F, ws_bytes=need):
        return zc.load().zc_moe_balance(logits, dtype, stride, tokens, experts, k, ids, score, sequences, mask, loss, counts,
                                        slope, ws, ws_bytes, None)

    expect(call, zc.ERR_INVALID_ARG, [{"logits": None}, {"dtype": 3}, {"experts": 0}, {"k": 0}, {"k": 9}, {"ids": None},
                                      {"score": 2}, {"sequences": 0}, {"sequences": 5}, {"loss": None}, {"counts": None},
                                      {"slope": None}, {"ws": None}])
    expect(call, zc.ERR_TOO_LARGE, [{"experts": 1025}, {"k": 33, "experts": 64}, {"tokens": 3 << 30}, {"stride": 1 << 41},
                                    {"tokens": 0, "sequences": 1 << 31}])
    expect(call, zc.ERR_ALIGNMENT, [{"logits": F + 2}, {"ids": F + 2}, {"loss": F + 1}, {"counts": F + 2}, {"slope": F + 2},
                                    {"ws": F + 8}])
    expect(call, zc.ERR_WORKSPACE, [{"ws_bytes": need - 1}])


def test_balance_backward():
    def call(dloss=F, logits=F, dtype=0, tokens=12, experts=8, score=1, sequences=3, slope=F, out=F):
        return zc.load().zc_moe_balance_backward(dloss, logits, dtype, 8, tokens, experts, score, sequences, None, slope, out,
                                                 None)

    expect(call, zc.ERR_INVALID_ARG, [{"dloss": None}, {"logits": None}, {"dtype": -1}, {"experts": 0}, {"score": 7},
                                      {"sequences": 0}, {"sequences": 7}, {"slope": None}, {"out": None}])
    expect(call, zc.ERR_TOO_LARGE, [{"experts": 2000}, {"tokens": 3 << 30}])
    expect(call, zc.ERR_ALIGNMENT, [{"dloss": F + 2}, {"logits": F + 1}, {"slope": F + 2}, {"out": F + 1}])


def test_dropout():
    def call(x=F, dtype=0, stride=16, residual=F, rstride=16, tokens=4, width=16, p=0.5, rng=F, out=F):
        return zc.load().zc_dropout(x, dtype, stride, residual, rstride, 1.0, tokens, width, p, rng, 0, out, None)

    expect(call, zc.ERR_INVALID_ARG, [{"x": None}, {"dtype": 4}, {"width": 0}, {"p": -0.1}, {"p": 1.001},
                                      {"p": float("nan")}, {"rng": None}, {"out": None}])
    expect(call, zc.ERR_TOO_LARGE, [{"width": 1 << 31}, {"tokens": 1 << 32}, {"stride": 1 << 41}, {"rstride": 1 << 41}])
    expect(call, zc.ERR_ALIGNMENT, [{"x": F + 1}, {"residual": F + 1}, {"rng": F + 4}, {"out": F + 1}])
    assert call(tokens=0, x=None, rng=None, out=None, residual=None) == zc.OK


def test_layer_norm():
    def call(**kw):
        a = LayerNormArgs(y=F, x=F, y_stride=16, x_stride=16, tokens=4, weight=F, bias=F, rng=F, p=0.1, hidden=16,
                          dtype=0, params_f32=1, residual_scale=1, eps=1e-5, x_new=F, h=F, stats=F)
        for k, v in kw.items():
            setattr(a, k, v)
        return zc.load().zc_layer_norm(ctypes.byref(a), None)

    expect(call, zc.ERR_INVALID_ARG, [{"x": None}, {"dtype": 3}, {"hidden": 0}, {"weight": None}, {"h": None}, {"x_new": None},
                                      {"y": None}, {"rng": None}, {"p": 1.5}, {"y": None, "x_new": None}])
    expect(call, zc.ERR_TOO_LARGE, [{"hidden": norm.MAX_HIDDEN + 1}, {"tokens": 1 << 31}, {"x_stride": 1 << 41}])
    expect(call, zc.ERR_ALIGNMENT, [{"x": F + 1}, {"y": F + 1}, {"weight": F + 2}, {"bias": F + 2}, {"x_new": F + 1},
                                    {"h": F + 1}, {"stats": F + 4}, {"rng": F + 4}])
    assert zc.load().zc_layer_norm(None, None) == zc.ERR_INVALID_ARG
    assert call(tokens=0, x=None, h=None) == zc.OK


def test_layer_norm_backward():
    need = norm.workspace_size(4, 16)

    def call(**kw):
        a = LayerNormBackwardArgs(dx_new=F, dh=F, x_new=F, dx_new_stride=16, dh_stride=16, x_new_stride=16, tokens=4,
                                  stats=F, weight=F, rng=F, p=0.1, hidden=16, dtype=0, params_f32=1, residual_scale=1,
                                  dy=F, dx=F, dweight=F, dbias=F, ws=F, ws_bytes=need)
        for k, v in kw.items():
            setattr(a, k, v)
        return zc.load().zc_layer_norm_backward(ctypes.byref(a), None)

    expect(call, zc.ERR_INVALID_ARG, [{"dh": None}, {"x_new": None}, {"stats": None}, {"weight": None}, {"dx": None},
                                      {"dweight": None}, {"ws": None}, {"dy": None}, {"rng": None}, {"p": -1},
                                      {"dtype": 5}, {"hidden": 0}])
    expect(call, zc.ERR_TOO_LARGE, [{"hidden": norm.MAX_HIDDEN + 1}, {"tokens": 1 << 31}, {"dh_stride": 1 << 41}])
    expect(call, zc.ERR_ALIGNMENT, [{"dx_new": F + 1}, {"dh": F + 1}, {"x_new": F + 1}, {"stats": F + 4}, {"weight": F + 2},
                                    {"dy": F + 1}, {"dx": F + 1}, {"dweight": F + 2}, {"dbias": F + 2}, {"ws": F + 8}])
    expect(call, zc.ERR_WORKSPACE, [{"ws_bytes": need - 1}])


def test_embedding():
    def call(ids=F, wide=1, tokens=4, table=F, dtype=0, f32=0, stride=16, vocab=10, hidden=16, out=F, status=F):
        return zc.load().zc_embedding(ids, wide, tokens, table, dtype, f32, stride, vocab, hidden, 1.0, out, status, None)

    expect(call, zc.ERR_INVALID_ARG, [{"ids": None}, {"table": None}, {"dtype": 3}, {"hidden": 0}, {"out": None},
                                      {"status": None}])
    expect(call, zc.ERR_TOO_LARGE, [{"tokens": 1 << 31}, {"vocab": 1 << 31}, {"hidden": 1 << 31}, {"stride": 1 << 41}])
    expect(call, zc.ERR_ALIGNMENT, [{"ids": F + 4}, {"ids": F + 2, "wide": 0}, {"table": F + 1}, {"table": F + 2, "f32": 1},
                                    {"out": F + 1}, {"status": F + 2}])


def test_embedding_backward():
    need = embedding.workspace_size(4, 10, 16)

    def call(dout=F, dtype=0, stride=16, ids=F, wide=1, tokens=4, vocab=10, hidden=16, f32=0, out=F, ws=F, ws_bytes=need,
             status=F):
        return zc.load().zc_embedding_backward(dout, dtype, stride, ids, wide, tokens, vocab, hidden, 1.0, f32, 0, out, ws,
                                               ws_bytes, status, None)

    expect(call, zc.ERR_INVALID_ARG, [{"dout": None}, {"ids": None}, {"dtype": 3}, {"hidden": 0}, {"out": None}, {"ws": None},
                                      {"status": None}])
    expect(call, zc.ERR_TOO_LARGE, [{"tokens": 1 << 31}, {"vocab": 1 << 31}, {"hidden": 1 << 31}, {"stride": 1 << 41}])
    expect(call, zc.ERR_ALIGNMENT, [{"dout": F + 1}, {"ids": F + 4}, {"out": F + 1}, {"out": F + 2, "f32": 1}, {"ws": F + 8},
                                    {"status": F + 2}])
    expect(call, zc.ERR_WORKSPACE, [{"ws_bytes": need - 1}])


def test_workspace_sizes():
    for size, args in ((moe.balance_workspace_size, [(5, 0, 1), (5, 8, 0), (5, 8, 2)]),
                       (embedding.workspace_size, [(5, 8, 0)])):
        for a in args:
            with pytest.raises(zc.ZcError) as e:
                size(*a)
            assert e.value.code == zc.ERR_INVALID_ARG
    for size, a in ((moe.balance_workspace_size, (5, 1025, 1)), (moe.balance_workspace_size, (1 << 31, 8, 1)),
                    (embedding.workspace_size, (1 << 31, 8, 8)), (embedding.workspace_size, (5, 1 << 31, 8))):
        with pytest.raises(zc.ZcError) as e:
            size(*a)
        assert e.value.code == zc.ERR_TOO_LARGE
    assert embedding.workspace_size(100, 10, 8) <= embedding.workspace_size(101, 11, 9)


# ------------------------------------------------------------------ the Python entry points
TOKENS, EXPERTS, HIDDEN, VOCAB = 6, 4, 32, 10


def tensors(device):
    def empty(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device=device)

    return {"logits": empty(TOKENS, EXPERTS), "experts": empty(TOKENS, 2, dtype=torch.int32), "loss": empty(),
            "slope": empty(3, EXPERTS), "mask": empty(TOKENS, dtype=torch.bool), "dlogits": empty(TOKENS, EXPERTS),
            "x": empty(TOKENS, HIDDEN), "y": empty(TOKENS, HIDDEN), "dout": empty(TOKENS, HIDDEN), "out": empty(TOKENS, HIDDEN),
            "h": empty(TOKENS, HIDDEN), "stats": empty(TOKENS, 2), "w": empty(HIDDEN), "b": empty(HIDDEN),
            "rng": empty(2, dtype=torch.int64), "ids": empty(TOKENS, dtype=torch.int64), "table": empty(VOCAB, HIDDEN),
            "dtable": empty(VOCAB, HIDDEN), "status": empty(1, dtype=torch.int32), "ws": empty(1 << 16, dtype=torch.uint8)}


CALLS = {
    "balance_loss": (lambda t: moe.balance_loss(t["logits"], t["experts"], t["ws"], sequences=3, mask=t["mask"]),
                     ("logits", "experts", "ws", "mask")),
    "balance_loss_backward": (lambda t: moe.balance_loss_backward(t["loss"], t["logits"], t["slope"], mask=t["mask"],
                                                                  dlogits=t["dlogits"]),
                              ("loss", "logits", "slope", "mask", "dlogits")),
    "dropout": (lambda t: dropout.dropout(t["x"], 0.5, t["rng"], residual=t["y"], out=t["out"]), ("x", "rng", "y", "out")),
    "dropout_backward": (lambda t: dropout.dropout_backward(t["x"], 0.5, t["rng"], out=t["out"]), ("x", "rng", "out")),
    "layer_norm": (lambda t: norm.layer_norm(t["x"], t["w"], t["b"], out=t["out"]), ("x", "w", "b", "out")),
    "add_layer_norm": (lambda t: norm.add_layer_norm(t["y"], t["x"], t["w"], t["b"], p=0.5, rng=t["rng"], x_new=t["out"],
                                                     h=t["h"]), ("y", "x", "w", "b", "rng", "out", "h")),
    "layer_norm_backward": (lambda t: norm.layer_norm_backward(t["dout"], t["x"], t["stats"], t["w"], t["ws"],
                                                               dresidual=t["y"]), ("dout", "x", "stats", "w", "ws", "y")),
    "add_layer_norm_backward": (lambda t: norm.add_layer_norm_backward(t["y"], t["dout"], t["x"], t["stats"], t["w"], t["ws"],
                                                                       p=0.5, rng=t["rng"]),
                                ("y", "dout", "x", "stats", "w", "ws", "rng")),
    "lookup": (lambda t: embedding.lookup(t["ids"], t["table"], t["status"], out=t["out"]), ("ids", "table", "status", "out")),
    "lookup_backward": (lambda t: embedding.lookup_backward(t["dout"], t["ids"], VOCAB, t["ws"], t["status"],
                                                            dtable=t["dtable"]), ("dout", "ids", "ws", "status", "dtable")),
}


@pytest.fixture
def fake(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)  # or fake tensors first try the device they name
    with FakeTensorMode():
        yield


@pytest.mark.parametrize("call,names,other", [(c, n, o) for c, n in CALLS.values() for o in n],
                         ids=[f"{c}-{o}" for c, (_, n) in CALLS.items() for o in n])
def test_a_tensor_on_another_device(fake, call, names, other):
    here, there = tensors("cuda:0"), tensors("cuda:1")
    with pytest.raises(ValueError, match="device"):
        call({**here, other: there[other]})


WRONG = [("balance_loss", {"experts": (TOKENS, 2, torch.int64)}), ("balance_loss", {"experts": (TOKENS, torch.int32)}),
         ("balance_loss", {"logits": (TOKENS + 1, EXPERTS, torch.float32)}), ("balance_loss", {"mask": (TOKENS, torch.float32)}),
         ("balance_loss", {"mask": (TOKENS, 1, torch.bool)}), ("balance_loss", {"logits": (TOKENS, EXPERTS, torch.float64)}),
         ("balance_loss_backward", {"loss": (2, torch.float32)}), ("balance_loss_backward", {"loss": (1, torch.float64)}),
         ("balance_loss_backward", {"slope": (4, EXPERTS, torch.float32)}),
         ("balance_loss_backward", {"slope": (3, EXPERTS + 1, torch.float32)}),
         ("dropout", {"x": (TOKENS, HIDDEN, torch.int32)}), ("dropout", {"rng": (2, torch.int32)}),
         ("dropout", {"rng": (3, torch.int64)}), ("dropout", {"y": (TOKENS, HIDDEN, torch.bfloat16)}),
         ("dropout", {"x": (TOKENS, 2, HIDDEN, torch.float32)}),
         ("layer_norm", {"w": (HIDDEN + 1, torch.float32)}), ("layer_norm", {"w": (HIDDEN, torch.bfloat16)}),
         ("layer_norm", {"b": (HIDDEN, torch.bfloat16)}), 
         ("add_layer_norm", {"y": (TOKENS + 1, HIDDEN, torch.float32)}),
         ("layer_norm_backward", {"stats": (TOKENS, 1, torch.float32)}),
         ("layer_norm_backward", {"stats": (TOKENS, 2, torch.float64)}),
         ("add_layer_norm_backward", {"dout": (TOKENS, HIDDEN, torch.bfloat16)}),
         ("lookup", {"ids": (TOKENS, torch.int16)}), ("lookup", {"ids": (2, 3, torch.int64)}),
         ("lookup", {"table": (VOCAB, HIDDEN, torch.float64)}), 
         ("lookup_backward", {"ids": (TOKENS + 1, torch.int64)}),
         ("lookup_backward", {"dtable": (VOCAB, HIDDEN, torch.bfloat16)})]


WRONG_OUTPUTS = [("dropout", {"out": (TOKENS, HIDDEN + 1, torch.float32)}), ("dropout", {"out": (TOKENS, HIDDEN, torch.float16)}),
                 ("layer_norm", {"x": (TOKENS, HIDDEN, torch.float16)}),
                 ("add_layer_norm", {"h": (TOKENS, HIDDEN, torch.bfloat16)}),
                 ("add_layer_norm", {"out": (TOKENS + 1, HIDDEN, torch.float32)}),
                 ("balance_loss_backward", {"dlogits": (TOKENS, EXPERTS, torch.float16)}),
                 ("lookup", {"out": (TOKENS, HIDDEN, torch.float16)}),
                 ("lookup_backward", {"dtable": (VOCAB + 1, HIDDEN, torch.float32)})]


@pytest.mark.gpu
@pytest.mark.parametrize("name,wrong", WRONG_OUTPUTS, ids=[f"{n}-{i}" for i, (n, _) in enumerate(WRONG_OUTPUTS)])
def test_wrong_outputs(zc, name, wrong):
    t = tensors("cuda:0")
    for k, (*shape, dtype) in wrong.items():
        t[k] = torch.empty(shape, dtype=dtype, device="cuda:0")
    with pytest.raises(ValueError):
        CALLS[name][0](t)


@pytest.mark.parametrize("name,wrong", WRONG, ids=[f"{n}-{i}" for i, (n, _) in enumerate(WRONG)])
def test_wrong_tensors(fake, name, wrong):
    t = tensors("cuda:0")
    for k, (*shape, dtype) in wrong.items():
        t[k] = torch.empty(shape, dtype=dtype, device="cuda:0")
    with pytest.raises(ValueError):
        CALLS[name][0](t)


def test_wrong_values(fake):
    t = tensors("cuda:0")
    for p in (-0.5, 1.5, float("nan")):
        with pytest.raises(ValueError, match="probability"):
            dropout.dropout(t["x"], p, t["rng"])
    for call in (-1, 1 << 32):
        with pytest.raises(ValueError, match="32 bits"):
            dropout.dropout(t["x"], 0.5, t["rng"], call)
    for bad in (lambda: dropout.dropout(t["x"], 0.5, None), lambda: norm.add_layer_norm(t["y"], t["x"], t["w"], p=0.5),
                lambda: moe.balance_loss(t["logits"], t["experts"], t["ws"], sequences=4),
                lambda: moe.balance_loss(t["logits"], t["experts"], t["ws"], sequences=0),
                lambda: moe.balance_loss(t["logits"], t["experts"], t["ws"], score="tanh"),
                lambda: embedding.lookup(t["ids"], t["table"], t["status"], dtype=torch.int32),
                lambda: embedding.lookup(t["ids"], t["table"].t(), t["status"]),
                lambda: embedding.lookup_backward(t["dout"], t["ids"], -1, t["ws"], t["status"]),
                lambda: embedding.lookup_backward(t["dout"], t["ids"], VOCAB, t["ws"], t["status"], accumulate=True)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        norm.layer_norm(t["x"], None)
    with pytest.raises(zc.ZcError):
        embedding.lookup_backward(t["dout"], t["ids"], 1 << 31, t["ws"], t["status"])


SCALES_OF_ONE = [1 + 2**-40, 2**0.5 * 0.5**0.5, 0.99999999]  # 1 as float32, which is what the kernels take


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("scale,own", [*((s, False) for s in SCALES_OF_ONE), (1.0, False), (1 + 2**-22, True), (0.5, True)])
def test_a_scale_of_one_after_rounding_has_one_gradient(fake, bias, scale, own):
    """The operator's list as the native call makes it: dy is dx where the scale that the kernel gets is 1."""
    from lossless_bf16_exponent_zc_gb300 import torch_ops  # noqa: F401
    t = tensors("cuda:0")
    got = torch.ops.zc.layer_norm_backward(None, t["dout"], t["x"], t["stats"], t["w"], bias, None, 0.0, 0, scale)
    assert [g.shape for g in got] == [t["x"].shape, t["w"].shape] + [t["x"].shape] * own + [t["w"].shape] * bias


@pytest.mark.parametrize("experts", [8, 256, 512, 513, 1024])
def test_a_balance_workspace_holds_every_smaller_batch(experts):
    """Up to so many tokens in up to so many sequences: also where the chunks of a sequence have reached their most."""
    sizes = [1, 63, 64, 65, 1024, 38911, 38912, 38913, 40000, 60000, 77823, 77824, 77825, 81920, 90112, 155648, 155649,
             1 << 20, (1 << 20) + 1, 2**31 - 1]
    need = [moe.balance_workspace_size(t, experts) for t in sizes]
    assert need == sorted(need)
    length = 4096                                                       # sequences of one length
    need = [moe.balance_workspace_size(n * length, experts, n) for n in (1, 2, 7, 19, 20, 304, 608, 609, 1000, 1216, 1217, 5000)]
    assert need == sorted(need)
    need = [moe.balance_workspace_size(1 << 20, experts, 1 << n) for n in range(21)]
    assert need == sorted(need)


class Unclear:
    """What has no truth value, like an array of several numbers."""

    def __bool__(self):
        raise ArithmeticError("ambiguous")


def test_flags_without_a_truth_value(fake):
    t = tensors("cuda:0")
    for call in (lambda: moe.route(t["logits"], 2, renormalize=Unclear()),
                 lambda: moe.route_backward(t["logits"][:, :2].contiguous(), t["logits"], t["experts"], renormalize=Unclear()),
                 lambda: norm.layer_norm(t["x"], t["w"], save=Unclear()),
                 lambda: norm.add_layer_norm(t["y"], t["x"], t["w"], save=Unclear()),
                 lambda: norm.layer_norm_backward(t["dout"], t["x"], t["stats"], t["w"], t["ws"], bias=Unclear()),
                 lambda: embedding.lookup_backward(t["dout"], t["ids"], VOCAB, t["ws"], t["status"], dtable=t["dtable"],
                                                   accumulate=Unclear())):
        with pytest.raises(ArithmeticError, match="ambiguous"):
            call()
