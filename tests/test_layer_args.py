"""Argument checks of the operators around an expert-parallel exchange (C ABI; nothing is launched, no GPU)."""
import ctypes

import pytest

from lossless_bf16_exponent_zc_gb300 import moe, norm, zc

class NormArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("y", "x")] + [(n, ctypes.c_uint64) for n in
                ("y_stride", "x_stride", "tokens")] + [(n, ctypes.c_void_p) for n in
                ("weight", "gate", "next_weight")] + [("gate_rows", ctypes.c_uint64), ("hidden", ctypes.c_uint32),
                ("dtype", ctypes.c_int32), ("gate_wide", ctypes.c_int32), ("params_f32", ctypes.c_int32),
                ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float), ("x_new", ctypes.c_void_p),
                ("h", ctypes.c_void_p)]


class NormBackwardArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dx_new", "dh", "y", "x_new")] + [(n, ctypes.c_uint64) for n in
                ("dx_new_stride", "dh_stride", "y_stride", "x_new_stride", "tokens")] + [(n, ctypes.c_void_p) for n in
                ("weight", "gate", "next_weight")] + [("gate_rows", ctypes.c_uint64), ("hidden", ctypes.c_uint32),
                ("dtype", ctypes.c_int32), ("gate_wide", ctypes.c_int32), ("params_f32", ctypes.c_int32),
                ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)] + [(n, ctypes.c_void_p) for n in
                ("dy", "dx", "dweight", "dgate", "dnext_weight", "ws")] + [("ws_bytes", ctypes.c_uint64)]


@pytest.fixture(scope="module", autouse=True)
def prototypes():
    lib = zc.load()
    vp, u64, u32, i32, f32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int, ctypes.c_float
    lib.zc_moe_route.argtypes = [vp, i32, u64, u64, u32, u32, i32, vp, i32, f32, vp, vp, vp]
    lib.zc_moe_route_backward.argtypes = [vp, vp, i32, u64, u64, u32, u32, vp, i32, i32, f32, vp, vp]
    lib.zc_moe_dispatch.argtypes = [vp, i32, u64, u64, u32, vp, i32, u32, u32, vp, vp, vp, vp, vp, u64, vp]
    lib.zc_moe_combine.argtypes = [vp, i32, u64, u64, vp, vp, u64, u32, u32, vp, vp, vp]
    lib.zc_moe_combine_backward.argtypes = [vp, i32, u64, vp, u64, u64, vp, vp, u64, u32, u32, vp, vp, vp, vp]
    lib.zc_norm.argtypes = [ctypes.POINTER(NormArgs), vp]
    lib.zc_norm_backward.argtypes = [ctypes.POINTER(NormBackwardArgs), vp]


F = 0x10000  # an aligned address that is never dereferenced: every call below is refused first


def code(name, *args):
    return getattr(zc.load(), name)(*args)


def test_route():
    def call(logits=F, dtype=0, stride=8, tokens=4, experts=8, k=2, score=0, bias=None, weights=F, ids=F):
        return code("zc_moe_route", logits, dtype, stride, tokens, experts, k, score, bias, 1, 1.0, weights, ids, None)

    for kw in ({"logits": None}, {"dtype": 3}, {"dtype": -1}, {"experts": 0}, {"k": 0}, {"k": 9}, {"score": 2},
               {"bias": F}, {"weights": None}, {"ids": None}):
        assert call(**kw) == zc.ERR_INVALID_ARG, kw
    for kw in ({"k": 33, "experts": 64}, {"experts": 1025}, {"tokens": 1 << 30}, {"stride": 1 << 41}):
        assert call(**kw) == zc.ERR_TOO_LARGE, kw
    for kw in ({"logits": F + 1}, {"weights": F + 2}, {"ids": F + 2}, {"bias": F + 2, "score": 1}):
        assert call(**kw) == zc.ERR_ALIGNMENT, kw


def test_route_backward():
    def call(dweights=F, logits=F, dtype=2, tokens=4, experts=8, k=2, ids=F, score=1, out=F):
        return code("zc_moe_route_backward", dweights, logits, dtype, 8, tokens, experts, k, ids, score, 1, 1.0, out,
                    None)

    for kw in ({"dweights": None}, {"logits": None}, {"ids": None}, {"out": None}, {"score": 5}, {"k": 0}, {"dtype": 9}):
        assert call(**kw) == zc.ERR_INVALID_ARG, kw
    for kw in ({"dweights": F + 1}, {"logits": F + 2}, {"ids": F + 1}, {"out": F + 2}):
        assert call(**kw) == zc.ERR_ALIGNMENT, kw


def test_dispatch():
    need = moe.workspace_size(4, 2, 8)

    def call(x=F, dtype=0, tokens=4, hidden=16, ids=F, wide=0, k=2, experts=8, rows=F, pos=F, slots=F, offsets=F, ws=F,
             ws_bytes=need):
        return code("zc_moe_dispatch", x, dtype, 16, tokens, hidden, ids, wide, k, experts, rows, pos, slots, offsets,
                    ws, ws_bytes, None)

    for kw in ({"x": None}, {"dtype": 7}, {"hidden": 0}, {"ids": None}, {"k": 0}, {"experts": 0}, {"rows": None},
               {"pos": None}, {"slots": None}, {"offsets": None}, {"ws": None}):
        assert call(**kw) == zc.ERR_INVALID_ARG, kw
    for kw in ({"hidden": 1 << 31}, {"k": 33}, {"experts": 1025}, {"tokens": 1 << 31}):
        assert call(**kw) == zc.ERR_TOO_LARGE, kw
    for kw in ({"x": F + 1}, {"ids": F + 4, "wide": 1}, {"ids": F + 2}, {"rows": F + 1}, {"pos": F + 2},
               {"slots": F + 1}, {"offsets": F + 2}, {"ws": F + 2}):
        assert call(**kw) == zc.ERR_ALIGNMENT, kw
    assert call(ws_bytes=need - 1) == zc.ERR_WORKSPACE


@pytest.mark.parametrize("backward", [False, True])
def test_combine(backward):
    def call(rows=F, dtype=1, n_rows=8, weights=F, pos=F, tokens=4, k=2, hidden=16, out=F, status=F, dout=F, dweights=F):
        if backward:
            return code("zc_moe_combine_backward", dout, dtype, 16, rows, 16, n_rows, weights, pos, tokens, k, hidden,
                        out, dweights, status, None)
        return code("zc_moe_combine", rows, dtype, 16, n_rows, weights, pos, tokens, k, hidden, out, status, None)

    for kw in ({"rows": None}, {"dtype": 4}, {"pos": None}, {"k": 0}, {"hidden": 0}, {"out": None}, {"status": None}) + (
            ({"dout": None}, {"dweights": None}, {"weights": None}) if backward else ()):
        assert call(**kw) == zc.ERR_INVALID_ARG, kw
    for kw in ({"k": 40}, {"tokens": 1 << 31}, {"hidden": 1 << 31}):
        assert call(**kw) == zc.ERR_TOO_LARGE, kw
    for kw in ({"rows": F + 1}, {"weights": F + 2}, {"pos": F + 1}, {"out": F + 1}, {"status": F + 2}):
        assert call(**kw) == zc.ERR_ALIGNMENT, kw


def norm_args(cls, **kw):
    a = cls()
    for n in ("y", "weight", "next_weight", "x_new", "x", "h", "dx_new", "dh", "dy", "dx", "dweight", "dnext_weight",
              "ws"):
        if hasattr(cls, n):
            setattr(a, n, F)
    a.tokens, a.hidden, a.eps = 4, 16, 1e-6
    for name, _ in cls._fields_:
        if name.endswith("_stride"):
            setattr(a, name, 16)
    if hasattr(cls, "ws_bytes"):
        a.ws_bytes = norm.workspace_size(4, 16)
    for n, v in kw.items():
        setattr(a, n, v)
    return ctypes.byref(a)


COMMON = [({"dtype": 3}, "INVALID_ARG"), ({"hidden": 0}, "INVALID_ARG"), ({"eps": -1.0}, "INVALID_ARG"),
          ({"eps": float("nan")}, "INVALID_ARG"), ({"weight": None}, "INVALID_ARG"), ({"y": None}, "INVALID_ARG"),
          ({"gate": F, "gate_rows": 3, "dgate": F}, "INVALID_ARG"), ({"gate": F, "dgate": F}, "INVALID_ARG"),
          ({"hidden": 16385}, "TOO_LARGE"), ({"tokens": 1 << 31}, "TOO_LARGE"), ({"y_stride": 1 << 41}, "TOO_LARGE"),
          ({"y": F + 1}, "ALIGNMENT"), ({"weight": F + 1}, "ALIGNMENT"), ({"next_weight": F + 2, "params_f32": 1},
                                                                          "ALIGNMENT")]


def test_norm():
    lib = zc.load()
    assert lib.zc_norm(None, None) == zc.ERR_INVALID_ARG
    own = [({"x": None}, "INVALID_ARG"), ({"x_new": None}, "INVALID_ARG"), ({"h": None}, "INVALID_ARG"),
           ({"next_weight": None}, "INVALID_ARG"), ({"h": F + 1}, "ALIGNMENT"), ({"x_new": F + 1}, "ALIGNMENT")]
    for kw, want in COMMON + own:
        kw = {n: v for n, v in kw.items() if n != "dgate"}
        assert lib.zc_norm(norm_args(NormArgs, **kw), None) == getattr(zc, "ERR_" + want), kw
    assert lib.zc_norm(norm_args(NormArgs, tokens=0, x=None), None) == zc.OK


def test_norm_backward():
    lib = zc.load()
    assert lib.zc_norm_backward(None, None) == zc.ERR_INVALID_ARG
    own = [({"x_new": None}, "INVALID_ARG"), ({"dh": None}, "INVALID_ARG"), ({"dx": None}, "INVALID_ARG"),
           ({"dy": None}, "INVALID_ARG"), ({"dweight": None}, "INVALID_ARG"), ({"dgate": F}, "INVALID_ARG"),
           ({"dnext_weight": None}, "INVALID_ARG"), ({"ws": None}, "INVALID_ARG"), ({"ws": F + 2}, "ALIGNMENT"),
           ({"dx": F + 1}, "ALIGNMENT"), ({"ws_bytes": norm.workspace_size(4, 16) - 1}, "WORKSPACE"),
           ({"dh": None, "next_weight": None, "dnext_weight": None, "dx_new": None}, "INVALID_ARG")]
    for kw, want in COMMON + own:
        assert lib.zc_norm_backward(norm_args(NormBackwardArgs, **kw), None) == getattr(zc, "ERR_" + want), kw


def test_sizes():
    assert 0 < moe.workspace_size(0, 1, 1) <= moe.workspace_size(16384, 8, 256) <= moe.workspace_size(1 << 20, 8, 256)
    assert norm.workspace_size(10, 64) == 4 * (3 * 10 * 64 + 10)
    for f, args, want in ((moe.workspace_size, (4, 0, 2), "INVALID_ARG"), (moe.workspace_size, (4, 33, 2), "TOO_LARGE"),
                          (norm.workspace_size, (4, 0), "INVALID_ARG"), (norm.workspace_size, (4, 16385), "TOO_LARGE")):
        with pytest.raises(zc.ZcError) as e:
            f(*args)
        assert e.value.code == getattr(zc, "ERR_" + want)
