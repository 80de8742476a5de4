"""The codec's calls on a stream that is given (``stream=``): their outputs come from that stream's memory.

A block of the caching allocator may be written only on the stream it was allocated for: its last reader there may still
be queued.
"""
import pytest
import torch

import oracle
import workloads

pytestmark = pytest.mark.gpu

N = 5 * 4096 + 77
CYCLES = 30_000_000  # about 15 ms of a sleeping kernel in front of a queued reader


@pytest.fixture(scope="module")
def calls(zc):
    """name -> call(**kw) of every function that makes its outputs, those in a list."""
    x = workloads.gaussian_on_device(N, 1e-3, seed=3)
    f8 = torch.randint(0, 256, (N,), device="cuda", dtype=torch.uint8)
    cb = zc.codebook_to_device(oracle.codebook_from_sigma(1e-3))
    ws, st, pws = zc.workspace(N), zc.new_status(), zc.pipeline_workspace(8192)
    main, esc = zc.compress(x, cb, ws, st)
    table = zc.zq_table_from_histogram(torch.bincount(f8.long(), minlength=256).cpu().numpy())
    zq = zc.zq_compress(f8, table, ws, st)

    def pipeline(stream=None):
        streams = None if stream is None else (stream, torch.cuda.Stream(), torch.cuda.Stream())
        return [zc.pipelined_transfer(x, cb, 8192, pws, st, streams=streams)]

    def used(zm):  # what the stream holds; the rest of its buffer is not written
        return zm[:zc.zq_stream_bytes(zm)]

    table_of = {
        "histogram_topk": lambda **kw: [zc.histogram_topk(x, ws, st, **kw)[0]],
        "compress": lambda **kw: [zc.compress(x, cb, ws, st, **kw)[0]],
        "compress_adaptive": lambda **kw: [zc.compress_adaptive(x, cb, ws, st, **kw)[0]],
        "decompress": lambda **kw: [zc.decompress(main, esc, N, st, **kw)],
        "decompress_reduce": lambda **kw: list(zc.decompress_reduce([main] * 2, [esc] * 2, N, st, out_cb=cb, ws=ws,
                                                                    **kw)[:2]),
        "pipelined_transfer": pipeline,
        "zq_compress": lambda **kw: [zc.zq_compress(f8, table, ws, st, **kw)],
        "zq_decompress": lambda **kw: [zc.zq_decompress(zq, N, st, **kw)],
    }
    torch.cuda.synchronize()
    return table_of, st, {"zq_compress": used}


NAMES = ["histogram_topk", "compress", "compress_adaptive", "decompress", "decompress_reduce", "pipelined_transfer",
         "zq_compress", "zq_decompress"]


def pool_of(t):
    """The stream that the allocator keeps a tensor's block for."""
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= t.data_ptr() < segment["address"] + segment["total_size"]:
            return segment["stream"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_belong_to_the_given_stream(zc, calls, name):
    table, st, part = calls
    part = part.get(name, lambda t: t)
    want = table[name]()
    assert [pool_of(t) for t in want] == [torch.cuda.current_stream().cuda_stream] * len(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = table[name](stream=side)
    assert torch.cuda.current_stream() != side
    assert [pool_of(t) for t in got] == [side.cuda_stream] * len(got)
    torch.cuda.synchronize()
    assert zc.status_value(st) == 0
    for a, b in zip(got, want):
        assert torch.equal(part(a), part(b))


def test_a_block_with_a_queued_reader_is_left_alone(zc, calls):
    table, st, _ = calls
    want = table["decompress"]()[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = torch.full_like(want, 7)
    torch.cuda._sleep(CYCLES)
    seen = old.clone()
    del old
    out = table["decompress"](stream=side)[0]
    side.synchronize()
    assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert torch.equal(seen, torch.full_like(want, 7)) and zc.status_value(st) == 0


def test_a_handle_alone(zc, calls):
    """Anything with a cuda_stream is a stream."""
    table, st, _ = calls
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    class Handle:
        cuda_stream = side.cuda_stream

    out = table["decompress"](stream=Handle())[0]
    assert pool_of(out) == side.cuda_stream
    torch.cuda.synchronize()
    assert torch.equal(out, table["decompress"]()[0]) and zc.status_value(st) == 0
