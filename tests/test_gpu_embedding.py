"""Embedding rows and the table's gradient against plain indexing: rows bit for bit (one product, one rounding), the
gradient to (number of the id's tokens + 2) roundings of fp32 over the magnitudes it adds, and its last rounding."""
import pytest
import torch

pytestmark = pytest.mark.gpu
KINDS = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32), (torch.float32, torch.float32)]
U = 2.0**-24


@pytest.fixture(scope="module")
def emb(zc):
    from lossless_bf16_exponent_zc_gb300 import embedding
    return embedding


def check_rows(zc, emb, ids, table, dtype, scale=1.0, **kw):
    st = zc.new_status()
    got = emb.lookup(ids, table, st, scale=scale, dtype=dtype, **kw)
    there = (ids >= 0) & (ids < table.shape[0])
    want = torch.zeros((ids.numel(), table.shape[1]), device="cuda")
    want[there] = table[ids[there].long()].float() * torch.tensor(scale, device="cuda")
    assert torch.equal(got, want.to(dtype)) and got.dtype == dtype
    assert zc.status_value(st) == (zc.ERR_BAD_INDEX if bool((ids >= table.shape[0]).any()) else 0)
    return got


def check_gradient(zc, emb, dout, ids, vocab, dtype, scale=1.0, dtable=None, accumulate=False):
    st = zc.new_status()
    ws = emb.workspace(ids.numel(), vocab, dout.shape[1])
    ws.fill_(0xA5)                                                      # needs no initialisation
    old = dtable.clone() if accumulate else None
    got = emb.lookup_backward(dout, ids, vocab, ws, st, scale=scale, dtype=dtype, dtable=dtable, accumulate=accumulate)
    assert dtable is None or got is dtable
    there = (ids >= 0) & (ids < vocab)
    at, rows = ids[there].long(), dout[there].double()
    want, size = (torch.zeros((vocab, dout.shape[1]), dtype=torch.float64, device="cuda") for _ in range(2))
    want.index_add_(0, at, rows)
    size.index_add_(0, at, rows.abs())
    n = torch.bincount(at, minlength=vocab)[:, None] if vocab else torch.zeros((0, 1), device="cuda")
    want, size = want * scale, size * abs(scale)
    if accumulate:
        assert torch.equal(got[n[:, 0] == 0], old[n[:, 0] == 0])
        want, size = want + old.double(), size + old.double().abs()
    f = torch.finfo(dtype)
    room = (n + 3) * U * size + f.eps / 2 * want.abs() + f.smallest_normal * f.eps
    bad = ~((got.double() - want).abs() <= room)
    assert not bool(bad.any()), (int(bad.sum()), torch.nonzero(bad)[:4].tolist())
    assert zc.status_value(st) == (zc.ERR_BAD_INDEX if bool((ids >= vocab).any()) else 0)
    if not accumulate:
        again = emb.lookup_backward(dout, ids, vocab, ws, st, scale=scale, dtype=dtype)
        assert torch.equal(got, again)
    return got


def make(tokens, vocab, seed=0, itype=torch.int64, padded=0.1, skew=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = torch.rand(tokens, device="cuda", generator=g)
    ids = ((r ** 3 if skew else r) * vocab).long().clamp(max=vocab - 1)
    pad = torch.rand(tokens, device="cuda", generator=g) < padded
    return torch.where(pad, -1 - ids, ids).to(itype)


def rows_of(tokens, width, dtype, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((tokens, width), device="cuda", generator=g).to(dtype)


@pytest.mark.parametrize("dtype,ttype", KINDS)
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,vocab,width", [(1, 1, 1), (5, 3, 7), (8, 100, 8), (33, 50, 31), (100, 1000, 64), (65, 17, 129),
                                                (400, 300, 256), (70, 5000, 264), (3, 40, 1021), (500, 1025, 1000),
                                                (2, 9, 4096), (300, 70, 4099)])
def test_values(zc, emb, dtype, ttype, itype, tokens, vocab, width):
    ids, table = make(tokens, vocab, tokens, itype), rows_of(vocab, width, ttype)
    check_rows(zc, emb, ids, table, dtype, 1.7)
    check_gradient(zc, emb, rows_of(tokens, width, dtype), ids, vocab, ttype, 1.7)
    old = rows_of(vocab, width, ttype, 9)
    check_gradient(zc, emb, rows_of(tokens, width, dtype), ids, vocab, ttype, -0.3, old, True)


@pytest.mark.parametrize("tokens,vocab", [(1000, 1), (5000, 2), (4097, 30), (20000, 1 << 10), (20000, (1 << 10) - 1),
                                          (70000, 1 << 20), (70001, (1 << 20) + 3), (65536, 300), (65537, 40000),
                                          (200000, 100)])
def test_runs_of_tokens(zc, emb, tokens, vocab):
    """Ids with more tokens than a warp, a CTA or a chunk of the sort takes, and tables of one to three digits."""
    for skew in (True, False):
        check_gradient(zc, emb, rows_of(tokens, 24, torch.float32), make(tokens, vocab, 3, skew=skew), vocab, torch.float32)


@pytest.mark.parametrize("tokens", [1023, 1024, 1025, 4096, 8193, 32767, 32768, 32769])
@pytest.mark.parametrize("vocab", [511, 512, 140000])
def test_sizes_of_the_sort(zc, emb, tokens, vocab):
    """One CTA, a cluster with every number of keys a thread, and the launches beyond; tables of one to two digits."""
    check_gradient(zc, emb, rows_of(tokens, 8, torch.float32), make(tokens, vocab, tokens, torch.int32), vocab, torch.float32)


@pytest.mark.parametrize("vocab", [1, 100, 2000, 70000])
@pytest.mark.parametrize("width", [8, 4096, 20000])
def test_tables_of_any_size_are_zeroed_once(zc, emb, vocab, width):
    """The rows without a token are cut over the CTAs beside the sort and those after it: none is left out."""
    if vocab * width > 1 << 29:
        pytest.skip("covered by the smaller ones")
    ids = torch.tensor([0, vocab - 1, vocab // 2], device="cuda")
    for tokens in (3, 1500):
        many = ids.repeat(tokens // 3)
        dout = rows_of(len(many), width, torch.bfloat16)
        room = torch.full((vocab * width + 64,), 7.0, device="cuda").bfloat16()
        got = emb.lookup_backward(dout, many, vocab, emb.workspace(len(many), vocab, width), zc.new_status(),
                                  dtable=room[32:-32].view(vocab, width))
        used = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        used[ids] = True
        assert not got[~used].any() and bool(got[used].any(1).all())
        assert bool((room[:32] == 7).all()) and bool((room[-32:] == 7).all())


@pytest.mark.parametrize("tokens", [31, 32, 33, 64, 95, 97])
def test_runs_that_end_where_a_warp_does(zc, emb, tokens):
    for counts in ([tokens], [1, tokens - 1], [tokens - 1, 1], [16, 16, tokens - 32] if tokens > 32 else [tokens],
                   [1] * tokens):
        ids = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts)).cuda()
        ids = ids[torch.randperm(tokens, generator=torch.Generator().manual_seed(tokens)).cuda()]
        check_gradient(zc, emb, rows_of(tokens, 40, torch.bfloat16), ids, len(counts) + 2, torch.float32)


@pytest.mark.parametrize("dtype,ttype", KINDS)
@pytest.mark.parametrize("width", [16, 77, 300])
@pytest.mark.parametrize("lead", [1, 2, 3])
def test_strides_and_alignment(zc, emb, dtype, ttype, width, lead):
    tokens, vocab = 90, 40
    ids = make(tokens, vocab)
    table = rows_of(vocab, width + 9, ttype)[:, lead:lead + width]
    check_rows(zc, emb, ids, table, dtype, 0.5)
    room = torch.full((tokens * width + 8,), 7.0, device="cuda").to(dtype)
    out = room[lead:lead + tokens * width].view(tokens, width)
    assert check_rows(zc, emb, ids, table, dtype, 0.5, out=out) is out
    assert bool((room[:lead] == 7).all()) and bool((room[lead + tokens * width:] == 7).all())
    dout = rows_of(tokens, width + 5, dtype)[:, lead:lead + width]
    room = torch.full((vocab * width + 8,), 7.0, device="cuda").to(ttype)
    for accumulate in (False, True):
        check_gradient(zc, emb, dout, ids, vocab, ttype, 1.0, room[lead:lead + vocab * width].view(vocab, width), accumulate)
        assert bool((room[:lead] == 7).all()) and bool((room[lead + vocab * width:] == 7).all())
    one = rows_of(1, width, dtype).expand(tokens, width)
    check_gradient(zc, emb, one, ids, vocab, ttype)


def test_bad_ids(zc, emb):
    ids = torch.tensor([3, 10, -1, 2**40, -2**40, 9, 2**31, -2**31 + 1, 0], device="cuda")
    table = rows_of(10, 24, torch.float32)
    check_rows(zc, emb, ids, table, torch.float32)
    check_gradient(zc, emb, rows_of(9, 24, torch.float32), ids, 10, torch.float32)
    all_out = torch.full((50,), -1, device="cuda")
    check_rows(zc, emb, all_out, table, torch.float32)
    check_gradient(zc, emb, rows_of(50, 24, torch.float32), all_out, 10, torch.float32)


@pytest.mark.parametrize("tokens", [600, 5000, 40000])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_ids_at_the_ends_of_their_type(zc, emb, tokens, itype):
    ids, ends = make(tokens, 700, tokens, itype), torch.iinfo(itype)
    ids[::7], ids[3::7] = ends.min, ends.min + 1
    check_gradient(zc, emb, rows_of(tokens, 24, torch.bfloat16), ids, 700, torch.float32)
    ids[5::7] = ends.max
    check_rows(zc, emb, ids, rows_of(700, 24, torch.bfloat16), torch.bfloat16)
    check_gradient(zc, emb, rows_of(tokens, 24, torch.bfloat16), ids, 700, torch.bfloat16)


@pytest.mark.parametrize("width", [24, 1000, 1021])
def test_a_row_for_all_tokens(zc, emb, width):
    one = rows_of(1, width, torch.bfloat16).expand(900, width)
    check_gradient(zc, emb, one, make(900, 50), 50, torch.float32)
    ids = make(900, 50)
    check_rows(zc, emb, ids, rows_of(1, width, torch.float32).expand(50, width), torch.bfloat16)


def test_nothing(zc, emb):
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert emb.lookup(none, rows_of(5, 8, torch.float32), zc.new_status()).shape == (0, 8)
    check_gradient(zc, emb, rows_of(0, 24, torch.bfloat16), none, 7, torch.bfloat16)
    check_gradient(zc, emb, rows_of(0, 24, torch.bfloat16), none, 7, torch.float32, 1.0, rows_of(7, 24, torch.float32), True)
    empty = torch.zeros((0, 8), device="cuda")
    check_rows(zc, emb, torch.tensor([-1, 0, 5], device="cuda"), empty, torch.float32)
    check_gradient(zc, emb, rows_of(3, 8, torch.float32), torch.tensor([-1, 0, 5], device="cuda"), 0, torch.float32)


def test_rows_of_tokens_without_an_id_are_not_read(zc, emb):
    ids = make(200, 30)
    dout = rows_of(200, 32, torch.float32)
    want = check_gradient(zc, emb, dout, ids, 30, torch.float32)
    dout = torch.where((ids < 0)[:, None], float("nan"), dout)
    assert torch.equal(emb.lookup_backward(dout, ids, 30, emb.workspace(200, 30, 32), zc.new_status()), want)


def test_a_table_beyond_2_32_bytes(zc, emb):
    vocab, width = 1_100_000, 2048                                      # 2^31.07 values, 4.5 GB
    table = torch.zeros((vocab, width), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 5, vocab - 1, vocab // 2 + 1], device="cuda")
    table[ids] = rows_of(4, width, torch.bfloat16)
    check_rows(zc, emb, ids, table, torch.bfloat16)
    st, ws, dout = zc.new_status(), emb.workspace(4, vocab, width), rows_of(4, width, torch.bfloat16)
    got = emb.lookup_backward(dout, ids, vocab, ws, st, dtable=table)
    assert torch.equal(got[5], dout[1]) and torch.equal(got[ids[3]], dout[3])
    assert torch.equal(got[-1], (dout[0].float() + dout[2].float()).bfloat16())
    assert int(got.view(torch.int16).any(1).sum()) == 3 and zc.status_value(st) == 0


def test_captured_and_replayed(zc, emb):
    ids, dout, table = make(3000, 500), rows_of(3000, 72, torch.bfloat16), rows_of(500, 72, torch.bfloat16)
    st, ws = zc.new_status(), emb.workspace(3000, 500, 72)
    emb.lookup_backward(dout, ids, 500, ws, st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows, d = emb.lookup(ids, table, st), emb.lookup_backward(dout, ids, 500, ws, st)
    for seed in range(3):
        ids.copy_(make(3000, 500, seed))
        ws.fill_(seed * 77)
        graph.replay()
        assert torch.equal(d, emb.lookup_backward(dout, ids, 500, emb.workspace(3000, 500, 72), st))
        assert torch.equal(rows, emb.lookup(ids, table, st))


@pytest.mark.parametrize("dtype,ttype", KINDS)
@pytest.mark.parametrize("tokens,width", [(40, 24), (4000, 504), (2000, 1000), (40, 1021)])
@pytest.mark.parametrize("scale", [-2.0, float("inf"), float("nan")])
def test_no_token_is_a_row_of_zeros_whatever_the_scale(zc, emb, dtype, ttype, tokens, width, scale):
    ids = make(tokens, 30)
    ids[::5], ids[1::5] = -1, 30                                        # beyond the table: reported, and none too
    rows = emb.lookup(ids, rows_of(30, width, ttype), zc.new_status(), scale=scale, dtype=dtype)
    none = (ids < 0) | (ids >= 30)
    assert torch.equal(rows[none].float().view(torch.int32), torch.zeros((int(none.sum()), width), dtype=torch.int32, device="cuda"))
    assert bool((rows[~none] != 0).any(1).all())


@pytest.mark.parametrize("dtype,ttype", KINDS)
@pytest.mark.parametrize("tokens,width", [(2001, 1024), (2001, 1000), (2001, 4104), (1203, 2048), (20001, 264), (20001, 136)])
def test_many_wide_rows(zc, emb, dtype, ttype, tokens, width):
    """Every token a row of its own: rows of one warp's share, of a part of one and of several, the last partly filled, and
    narrow ones by pieces; negative ids and ids beyond the table, rows apart from one another."""
    vocab = 3000
    ids = make(tokens, vocab, width, torch.int32 if width % 3 else torch.int64, skew=False)
    table = rows_of(vocab, width, ttype)
    check_rows(zc, emb, ids, table, dtype, 1.7)
    ids[7::50] = vocab + torch.arange(len(ids[7::50]), device="cuda").to(ids.dtype)
    check_rows(zc, emb, ids, rows_of(vocab, width + 16, ttype, 2)[:, 8:8 + width], dtype, -0.6)
    room = torch.full((tokens * width + 16,), 7.0, device="cuda").to(dtype)
    check_rows(zc, emb, ids, table, dtype, 1.0, out=room[8:8 + tokens * width].view(tokens, width))
    assert bool((room[:8] == 7).all()) and bool((room[8 + tokens * width:] == 7).all())


@pytest.mark.parametrize("dtype,ttype", KINDS)
@pytest.mark.parametrize("tokens,vocab,width", [(5000, 2, 264), (5000, 2, 301), (9000, 40, 77), (40000, 3, 24), (40000, 900, 33)])
def test_long_runs_written_and_added(zc, emb, dtype, ttype, tokens, vocab, width):
    """Ids whose tokens lie in many runs, of several slabs, on 16 bytes and off them, in a table of their own and added to one."""
    ids, dout = make(tokens, vocab, tokens), rows_of(tokens, width, dtype)
    check_gradient(zc, emb, dout, ids, vocab + 5, ttype, 0.7)
    check_gradient(zc, emb, dout, ids, vocab + 5, ttype, 0.7, rows_of(vocab + 5, width, ttype, 9), True)
