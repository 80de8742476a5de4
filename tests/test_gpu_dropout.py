"""Dropout from a counter-based generator against the same formula in numpy: which values stay exactly, the values to
their rounding; both directions, strides, in place, replayed from a graph.

Tolerance: x f and a r + x f take at most three fp32 roundings of at most |a r| + |x f|, then one of the output's type:
half a step of the value, or of the smallest subnormal.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def drop(zc):
    from lossless_bf16_exponent_zc_gb300 import dropout
    return dropout


def philox(counter, key):
    """Philox-4x32-10 over arrays of counters [n, 4]."""
    c = [counter[:, i].astype(np.uint64) for i in range(4)]
    mask, k = np.uint64(0xFFFFFFFF), [int(key[0]), int(key[1])]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & mask, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]),
             a & mask]
        k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
    return np.stack(c, 1).astype(np.uint32)


def kept(rows, width, p, seed, offset, call):
    groups = -(-width // 8)
    at = np.stack(np.broadcast_arrays(np.arange(groups)[None, :], np.arange(rows)[:, None], call, offset % 2**32), -1)
    words = philox(at.reshape(-1, 4), (seed % 2**32, seed >> 32))
    bits = np.stack([words & 0xFFFF, words >> 16], 2).reshape(rows, groups * 8)[:, :width]
    limit = math.floor(p * 65536 + 0.5)
    return torch.from_numpy(bits >= limit).cuda(), 65536 / (65536 - limit) if limit < 65536 else 0.0


def check(got, x, keep, factor, residual=None, scale=1.0):
    t = got.dtype
    want = torch.where(keep, x.double() * factor, 0.0)
    size = want.abs()
    if residual is not None:
        size = size + (scale * residual.double()).abs()
        want = want + scale * residual.double()
    room = 3 * 2**-24 * size + torch.finfo(t).eps / 2 * want.abs() + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    assert bool(((got.double() - want).abs() <= room).all())
    if residual is None:
        assert torch.equal(got != 0, keep & (want != 0))


def test_published_vectors():
    """The known answers printed with the method: all zeros, all ones, and digits of pi."""
    zero = philox(np.zeros((1, 4), np.uint32), (0, 0))
    assert [hex(v) for v in zero[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    ones = philox(np.full((1, 4), 0xFFFFFFFF, np.uint32), (0xFFFFFFFF, 0xFFFFFFFF))
    assert [hex(v) for v in ones[0]] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]
    pi = philox(np.array([[0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344]], np.uint32), (0xA4093822, 0x299F31D0))
    assert [hex(v) for v in pi[0]] == ["0xd16cfe09", "0x94fdcceb", "0x5001e420", "0x24126ea1"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (2, 8), (5, 9), (1, 12), (4, 20), (33, 31), (7, 64), (3, 250),
                                        (2, 255), (9, 1021), (300, 264), (2, 4096), (1, 20011)])
def test_values(drop, dtype, rows, width):
    seed, offset, call, p = 0x1234_5678_9ABC_DEF, 2**32 + 7, 0xFFFF_FFF0, 0.3
    g = torch.Generator(device="cuda").manual_seed(width)
    x, r = (torch.randn((rows, width), device="cuda", generator=g).to(dtype) for _ in range(2))
    rng = drop.new_rng(seed, offset)
    keep, factor = kept(rows, width, p, seed, offset, call)
    check(drop.dropout(x, p, rng, call), x, keep, factor)
    check(drop.dropout(x, p, rng, call, residual=r, residual_scale=-0.75), x, keep, factor, r, -0.75)
    assert torch.equal(drop.dropout_backward(r, p, rng, call), drop.dropout(r, p, rng, call))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [5, 16, 129, 1024])
@pytest.mark.parametrize("lead,rlead", [(1, 0), (0, 1), (3, 5), (1, 1)])
def test_strides_and_alignment(drop, dtype, width, lead, rlead):
    """Rows of wider matrices, off 16 bytes by different amounts, one row for all, and an output off 16 bytes."""
    rows, p = 37, 0.5
    wide = torch.randn((rows, width + 11), device="cuda").to(dtype)
    x, r = wide[:, lead:lead + width], torch.randn((rows, width + 6), device="cuda").to(dtype)[:, rlead:rlead + width]
    one = torch.randn((1, width), device="cuda").to(dtype).expand(rows, width)
    rng = drop.new_rng(3)
    keep, factor = kept(rows, width, p, 3, 0, 1)
    check(drop.dropout(x, p, rng, 1, residual=r), x, keep, factor, r)
    check(drop.dropout(one, p, rng, 1, residual=x), one, keep, factor, x)
    room = torch.full((rows * width + 16,), 7.0, device="cuda").to(dtype)
    out = room[lead:lead + rows * width].view(rows, width)
    assert drop.dropout(x, p, rng, 1, out=out) is out
    check(out, x, keep, factor)
    assert bool((room[:lead] == 7).all()) and bool((room[lead + rows * width:] == 7).all())


@pytest.mark.parametrize("width", [64, 77])
def test_in_place(drop, width):
    x, r = (torch.randn((50, width), device="cuda").bfloat16() for _ in range(2))
    rng = drop.new_rng(11)
    want = drop.dropout(x, 0.4, rng, residual=r)
    a, b = x.clone(), r.clone()
    assert torch.equal(drop.dropout(a, 0.4, rng, residual=r, out=a), want)
    assert torch.equal(drop.dropout(x, 0.4, rng, residual=b, out=b), want)


@pytest.mark.parametrize("width", [64, 1000, 1021])
def test_a_row_for_all_tokens(drop, width):
    x = torch.randn((1, width), device="cuda").bfloat16().expand(300, width)
    r = torch.randn((300, width), device="cuda").bfloat16()
    keep, factor = kept(300, width, 0.3, 17, 0, 2)
    check(drop.dropout(x, 0.3, drop.new_rng(17), 2, residual=r), x, keep, factor, r)
    check(drop.dropout(r, 0.3, drop.new_rng(17), 2, residual=x), r, keep, factor, x)
    check(drop.dropout(x, 0.3, drop.new_rng(17), 2), x, keep, factor)


@pytest.mark.parametrize("dtype", TYPES)
def test_none_and_all(drop, dtype):
    x = torch.randn((6, 40), device="cuda").to(dtype)
    rng = drop.new_rng(1)
    assert torch.equal(drop.dropout(x, 0.0, rng), x)
    assert torch.equal(drop.dropout(x, 1e-7, rng), x)                  # rounds to no step
    assert not drop.dropout(x, 1.0, rng).any()
    assert torch.equal(drop.dropout(x, 1.0, rng, residual=x), x)
    assert drop.dropout(x[:0], 0.5, rng).shape == (0, 40)


def test_dropped_infinities_and_nans_leave_nothing(drop):
    x = torch.full((64, 64), math.nan, device="cuda")
    x[::2] = math.inf
    keep, _ = kept(64, 64, 0.5, 5, 0, 0)
    out = drop.dropout(x, 0.5, drop.new_rng(5))
    assert torch.equal(out == 0, ~keep) and torch.equal(torch.isnan(out), keep & torch.isnan(x))


def test_calls_offsets_and_seeds_draw_apart(drop):
    """A million values: the rate to five standard deviations, and masks of different counters share as many values as
    independent ones."""
    n, p = 1 << 20, 0.1
    x = torch.ones((256, n // 256), device="cuda")
    masks = [drop.dropout(x, p, drop.new_rng(s, o), c) != 0 for s, o, c in
             [(1, 0, 0), (2, 0, 0), (1, 1, 0), (1, 0, 1), (1 + 2**32, 0, 0)]]
    q = 1 - math.floor(p * 65536 + 0.5) / 65536
    for m in masks:
        assert abs(int(m.sum()) - n * q) < 5 * math.sqrt(n * q * (1 - q))
    for i, a in enumerate(masks):
        for b in masks[:i]:
            assert abs(int((a & b).sum()) - n * q * q) < 5 * math.sqrt(n * q * q * (1 - q * q))


def test_a_row_beyond_2_31_values(drop):
    """Offsets that pass 32 bits: the last row's values against the formula."""
    rows, width = 70000, 32768                                          # 2^31.1 values
    x = torch.ones((1, width), device="cuda").bfloat16().expand(rows, width)
    out = drop.dropout(x, 0.25, drop.new_rng(9), 2)
    words = philox(np.stack(np.broadcast_arrays(np.arange(width // 8), rows - 1, 2, 0), -1), (9, 0))
    bits = np.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)
    assert torch.equal(out[-1] != 0, torch.from_numpy(bits >= 16384).cuda())


def test_a_graph_draws_anew(drop):
    """The state is read when the graph runs: each replay gives what an ordinary call with that state gives."""
    x, rng = torch.randn((40, 96), device="cuda"), drop.new_rng(4)
    drop.dropout(x, 0.5, rng)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = drop.dropout(x, 0.5, rng, 3)
        rng[1] += 1
    rng[1] = 0
    seen = []
    for step in range(3):
        graph.replay()
        assert torch.equal(out, drop.dropout(x, 0.5, drop.new_rng(4, step), 3))
        seen.append(out.clone())
    assert not torch.equal(seen[0], seen[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(8200, 1032), (1030, 8208), (33000, 256)])
def test_many_values_with_a_residual(drop, dtype, rows, width):
    """More than 2^20 groups of eight columns, which 16-bit rows take four a thread: contiguous ones that end within a CTA's,
    rows of wider matrices, in place, and a last row written up to its end."""
    g = torch.Generator(device="cuda").manual_seed(width)
    wide, other = (torch.randn((rows, width + w), device="cuda", generator=g).to(dtype) for w in (8, 16))
    rng, p = drop.new_rng(21, 3), 0.3
    keep, factor = kept(rows, width, p, 21, 3, 6)
    x, r = wide[:, :width].contiguous(), other[:, :width].contiguous()
    room = torch.full((rows * width + 16,), 7.0, device="cuda").to(dtype)
    out = room[8:-8].view(rows, width)
    check(drop.dropout(x, p, rng, 6, residual=r, residual_scale=-0.75, out=out), x, keep, factor, r, -0.75)
    assert bool((room[:8] == 7).all()) and bool((room[-8:] == 7).all())
    want = drop.dropout(x, p, rng, 6, residual=r)
    check(want, x, keep, factor, r)
    for a, b in ((wide[:, :width], r), (x, other[:, :width]), (wide[:, :width], other[:, :width])):
        assert torch.equal(drop.dropout(a, p, rng, 6, residual=b), want)
    x, r = wide[:, 8:], other[:, 8:8 + width]                           # rows that start within the matrices'
    check(drop.dropout(x, p, rng, 6, residual=r), x, keep, factor, r)
    a = r.contiguous()
    assert torch.equal(drop.dropout(x, p, rng, 6, residual=a, out=a), drop.dropout(x, p, rng, 6, residual=r))
