"""The embedding, layer norm, dropout and balance loss together as a model's step uses them, as torch operators, on given
streams and from captured graphs."""
import math

import pytest
import torch

from lossless_bf16_exponent_zc_gb300 import torch_ops  # noqa: F401  (registers torch.ops.zc)
from test_gpu_dropout import kept
from test_gpu_layer_streams import pool_of

pytestmark = pytest.mark.gpu
ops = torch.ops.zc


def leaf(*shape, dtype=torch.float32, grad=True):
    return torch.randn(shape, device="cuda").to(dtype).requires_grad_(grad)


def op_calls(tokens, dtype):
    """name -> (op, arguments)"""
    ids = torch.randint(-1, 10, (tokens,), device="cuda")
    experts = torch.randint(-1, 9, (tokens, 2), device="cuda", dtype=torch.int32)
    mask = torch.arange(tokens, device="cuda") % 3 != 1
    rng = torch.tensor([7, 1], device="cuda")

    def act():
        return leaf(tokens, 24, dtype=dtype)

    return {"balance": (ops.moe_balance_loss, (leaf(tokens, 9, dtype=dtype), experts, None, "softmax", 1)),
            "balance_masked": (ops.moe_balance_loss, (leaf(tokens, 9, dtype=dtype), experts, mask, "sigmoid", 2)),
            "dropout": (ops.dropout, (act(), rng, None, 0.5, 3, 1.0)),
            "dropout_residual": (ops.dropout, (act(), rng, act(), 0.5, 3, 0.5)),
            "dropout_residual_1": (ops.dropout, (act(), rng, act(), 0.5, 3, 1.0)),
            "layer_norm": (ops.layer_norm, (act(), leaf(24), None, 1e-5)),
            "layer_norm_bias": (ops.layer_norm, (act(), leaf(24), leaf(24), 1e-5)),
            "add_layer_norm": (ops.add_layer_norm, (act(), act(), leaf(24), None, None, 0.0, 0, 1.0, 1e-5)),
            "add_layer_norm_scaled": (ops.add_layer_norm, (act(), act(), leaf(24), leaf(24), None, 0.0, 0, 0.5, 1e-5)),
            "add_layer_norm_drop": (ops.add_layer_norm, (act(), act(), leaf(24), leaf(24), rng, 0.25, 2, 1.0, 1e-5)),
            "embedding": (ops.embedding, (ids, leaf(10, 24, dtype=dtype), 2.0, None)),
            "embedding_f32": (ops.embedding, (ids, leaf(10, 24), 1.0, torch.bfloat16))}


OPS = ["balance", "balance_masked", "dropout", "dropout_residual", "dropout_residual_1", "layer_norm", "layer_norm_bias",
       "add_layer_norm", "add_layer_norm_scaled", "add_layer_norm_drop", "embedding", "embedding_f32"]


@pytest.mark.parametrize("name", OPS)
@pytest.mark.parametrize("tokens,dtype", [(6, torch.bfloat16), (0, torch.float32)])
def test_opcheck(zc, name, tokens, dtype):
    op, args = op_calls(tokens, dtype)[name]
    torch.library.opcheck(op, args)


@pytest.mark.parametrize("name", OPS)
def test_gradients_of_an_empty_batch(zc, name):
    op, args = op_calls(0, torch.bfloat16)[name]
    out = op(*args)
    out = out if isinstance(out, tuple) else (out,)
    sum(o.float().sum() for o in out if o.requires_grad).backward()
    for a in args:
        if isinstance(a, torch.Tensor) and a.requires_grad:
            assert a.grad.shape == a.shape and not a.grad.any()


def test_partly_used_outputs(zc):
    """Gradients that reach one of two outputs alone, and ones with strides of their own."""
    y, x, w, b = leaf(10, 24), leaf(10, 24), leaf(24), leaf(24)
    rng = torch.tensor([3, 0], device="cuda")
    keep, factor = kept(10, 24, 0.5, 3, 0, 0)
    a, _, _ = ops.add_layer_norm(y, x, w, b, rng, 0.5, 0, 0.5, 1e-5)
    a.t().contiguous().sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 0.5)) and torch.equal(y.grad, keep * factor) and w.grad is None
    x.grad = y.grad = None
    _, h, _ = ops.add_layer_norm(y, x, w, b, rng, 0.5, 0, 0.5, 1e-5)
    (h.t() @ torch.ones((10, 1), device="cuda")).sum().backward()        # a transposed gradient
    assert torch.equal(b.grad, torch.full_like(b, 10.0)) and y.grad is not None
    ops.dropout(y, rng, x, 0.5, 1, 1.0).sum().backward()                 # an expanded one
    table = leaf(5, 24)
    rows, _ = ops.embedding(torch.tensor([1, 1, -1], device="cuda"), table, 2.0, None)
    rows.sum().backward()
    want = torch.zeros_like(table)
    want[1] = 4.0
    assert torch.equal(table.grad, want)


def test_a_state_that_moved_on_is_noticed(zc):
    x, rng = leaf(4, 24), torch.tensor([3, 0], device="cuda")
    out = ops.dropout(x, rng, None, 0.5, 0, 1.0)
    rng[1] += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_step_of_a_model(zc, score):
    """Embedding, layer norm, a router with its balance loss and experts, dropout into the stream, the next norm and a
    dropout of its own, against automatic differentiation of the plain formulas in 64 bits.  As in a block of the other
    norms: fp32 sums of up to 48 terms through the operators, each good to about 2^-20 of its terms, the norms passing on
    the relative error of their input: 2^-14 of a tensor's largest gradient leaves a wide margin."""
    torch.manual_seed(3)
    tokens, hidden, n, k, vocab, p = 60, 48, 6, 2, 17, 0.2
    ids = torch.randint(-1, vocab, (tokens,), device="cuda")
    shapes = {"table": (vocab, hidden), "w0": (hidden,), "b0": (hidden,), "router": (hidden, n), "up": (n, hidden, hidden),
              "w1": (hidden,), "b1": (hidden,)}
    v = {name: torch.randn(s, device="cuda") * (hidden**-0.5 if len(s) == 3 else 1) for name, s in shapes.items()}
    mine = {name: t.clone().requires_grad_(True) for name, t in v.items()}
    rng = torch.tensor([11, 4], device="cuda")
    mask = ids >= 0

    x, st = ops.embedding(ids, mine["table"], hidden**0.5, None)
    h, _ = ops.layer_norm(x, mine["w0"], mine["b0"], 1e-5)
    logits = h @ mine["router"]
    weights, experts = ops.moe_route(logits, None, k, score, True, 1.0)
    experts = torch.where(mask[:, None], experts, -1)
    loss, counts, _ = ops.moe_balance_loss(logits, experts, mask, score, 3)
    rows, positions, _, offsets = ops.moe_dispatch(h, experts, n)
    at = offsets.tolist()
    out = torch.cat([rows[at[e]:at[e + 1]] @ mine["up"][e] for e in range(n)] + [rows[at[n]:]])
    y, _ = ops.moe_combine(out, weights, positions)
    a, b, _ = ops.add_layer_norm(y, x, mine["w1"], mine["b1"], rng, p, 0, 0.8, 1e-5)
    c = ops.dropout(b, rng, a, p, 1, 0.5)
    assert zc.status_value(st) == 0 and int(counts.sum()) == k * int(mask.sum())

    e = {name: t.double().requires_grad_(True) for name, t in v.items()}

    def normed(z, w, bias):
        z = z - z.mean(1, keepdim=True)
        return z * torch.rsqrt(z.square().mean(1, keepdim=True) + 1e-5) * w + bias

    def dropped(z, call):
        keep, factor = kept(tokens, hidden, p, 11, 4, call)
        return torch.where(keep, z * factor, 0.0)

    ex = torch.where(mask[:, None], e["table"][ids.clamp(min=0)] * hidden**0.5, 0.0)
    eh = normed(ex, e["w0"], e["b0"])
    el = eh @ e["router"]
    prob = torch.softmax(el, 1) if score == "softmax" else torch.sigmoid(el)
    picked = torch.gather(prob, 1, experts.clamp(min=0).long()) * (experts >= 0)
    ew = picked / (picked.sum(1, keepdim=True) + 1e-20)
    ey = sum(ew[:, j:j + 1] * torch.einsum("td,tde->te", eh, e["up"][experts[:, j].clamp(min=0).long()]) for j in range(k))
    ea = 0.8 * ex + dropped(ey, 0)
    eb = normed(ea, e["w1"], e["b1"])
    ec = 0.5 * ea + dropped(eb, 1)
    q = prob / prob.sum(1, keepdim=True) * mask[:, None]
    want_loss = 0.0
    for s in range(3):
        part = slice(s * tokens // 3, (s + 1) * tokens // 3)
        t = int(mask[part].sum())
        used = experts[part][experts[part] >= 0].long()
        f = torch.bincount(used, minlength=n).double() / (k * t)
        want_loss = want_loss + n / 3 * (f * q[part].sum(0) / t).sum()
    co = torch.randn_like(c)
    ((c * co).sum() + 50 * loss).backward()
    ((ec * co.double()).sum() + 50 * want_loss).backward()
    assert abs(loss.item() - want_loss.item()) < 2**-18 * want_loss.item()
    for g, w in ((a, ea), (b, eb), (c, ec)):
        assert float((g.detach().double() - w.detach()).abs().max()) < 2**-14 * float(w.abs().max())
    for name in v:
        d, w = mine[name].grad.double(), e[name].grad
        assert float((d - w).abs().max()) < 2**-14 * float(w.abs().max()), name


TOKENS, HIDDEN, VOCAB, EXPERTS = 700, 264, 90, 12
NAMES = ["balance_loss", "balance_loss_backward", "dropout", "dropout_backward", "layer_norm", "add_layer_norm",
         "layer_norm_backward", "add_layer_norm_backward", "lookup", "lookup_backward", "no_tokens"]


@pytest.fixture(scope="module")
def calls(zc):
    """name -> call(stream=...) of every function, its tensor outputs in a list; and the tensors they read."""
    from lossless_bf16_exponent_zc_gb300 import dropout, embedding, moe, norm
    g = torch.Generator(device="cuda").manual_seed(6)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    x, y, gx = (randn(TOKENS, HIDDEN).bfloat16() for _ in range(3))
    w, b, logits, table = randn(HIDDEN), randn(HIDDEN), randn(TOKENS, EXPERTS), randn(VOCAB, HIDDEN)
    ids = torch.randint(-1, VOCAB, (TOKENS,), device="cuda", generator=g)
    experts = torch.randint(-1, EXPERTS, (TOKENS, 2), device="cuda", generator=g, dtype=torch.int32)
    rng, st, one = dropout.new_rng(1), zc.new_status(), torch.ones((), device="cuda")
    bws, nws = moe.balance_workspace(TOKENS, EXPERTS, 2), norm.workspace(TOKENS, HIDDEN)
    ews = embedding.workspace(TOKENS, VOCAB, HIDDEN)
    slope = moe.balance_loss(logits, experts, bws, sequences=2).slope
    stats = norm.layer_norm(x, w, save=True)[1]
    none = x[:0]

    def flat(r):
        if torch.is_tensor(r):
            return [r]
        return [t for part in r if part is not None for t in flat(part)]

    table_of = {
        "balance_loss": lambda **kw: moe.balance_loss(logits, experts, bws, sequences=2, **kw),
        "balance_loss_backward": lambda **kw: moe.balance_loss_backward(one, logits, slope, **kw),
        "dropout": lambda **kw: dropout.dropout(x, 0.3, rng, residual=y, **kw),
        "dropout_backward": lambda **kw: dropout.dropout_backward(x, 0.3, rng, **kw),
        "layer_norm": lambda **kw: norm.layer_norm(x, w, b, save=True, **kw),
        "add_layer_norm": lambda **kw: norm.add_layer_norm(y, x, w, b, p=0.3, rng=rng, save=True, **kw),
        "layer_norm_backward": lambda **kw: norm.layer_norm_backward(gx, x, stats, w, nws, dresidual=y, **kw),
        "add_layer_norm_backward": lambda **kw: norm.add_layer_norm_backward(y, gx, x, stats, w, nws, p=0.3, rng=rng, **kw),
        "lookup": lambda **kw: embedding.lookup(ids, table, st, dtype=torch.bfloat16, **kw),
        "lookup_backward": lambda **kw: embedding.lookup_backward(gx, ids, VOCAB, ews, st, dtype=torch.float32, **kw),
        "no_tokens": lambda **kw: norm.layer_norm_backward(none, none, stats[:0], w, nws, **kw),
    }
    torch.cuda.synchronize()
    made = {name: (lambda stream=None, f=f: flat(f(stream=stream))) for name, f in table_of.items()}
    made["inputs"] = [x, y, gx, logits, table]
    return made


@pytest.mark.parametrize("name", NAMES)
def test_outputs_belong_to_the_given_stream(calls, name):
    want = calls[name]()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = calls[name](stream=side)
    assert torch.cuda.current_stream() != side
    for t in got:
        assert t.numel() == 0 or pool_of(t) == side.cuda_stream
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(calls, name):
    """A graph's replay on inputs that changed gives what an ordinary call on them gives, several times over."""
    calls[name]()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls[name]()
    for _ in range(3):
        for t in calls["inputs"]:
            t.copy_(t.roll(1, 0))
        graph.replay()
        got = [t.clone() for t in out]
        for a, b in zip(got, calls[name]()):
            assert torch.equal(a, b)


def test_back_to_back_in_one_workspace(zc):
    """Calls of different sizes share a workspace in stream order, with no wait in between."""
    from lossless_bf16_exponent_zc_gb300 import embedding, moe
    ws, bws, st = embedding.workspace(20000, 5000, 64), moe.balance_workspace(20000, 64), zc.new_status()
    sizes = [(20000, 5000), (17, 3), (3000, 4999), (1, 1), (9000, 31), (20000, 2)] * 3
    made, losses = [], []
    for i, (tokens, vocab) in enumerate(sizes):
        g = torch.Generator(device="cuda").manual_seed(i)
        ids = torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
        dout = torch.randint(-8, 8, (tokens, 64), device="cuda", generator=g).float()
        made.append((ids, dout, vocab))
        experts = (ids % 64).to(torch.int32)[:, None]
        losses.append((experts, torch.zeros((tokens, 64), device="cuda")))
    torch.cuda.synchronize()
    got = [embedding.lookup_backward(dout, ids, vocab, ws, st) for ids, dout, vocab in made]
    counts = [moe.balance_loss(logits, experts, bws) for experts, logits in losses]
    for (ids, dout, vocab), d in zip(made, got):
        assert torch.equal(d, torch.zeros((vocab, 64), device="cuda").index_add_(0, ids, dout))  # whole numbers: exact
    for (experts, _), c in zip(losses, counts):
        assert torch.equal(c.counts[0], torch.bincount(experts[:, 0], minlength=64).int())
        assert math.isclose(float(c.loss), 1.0, rel_tol=1e-3)
    assert zc.status_value(st) == 0


def test_two_graphs_with_a_workspace_each(zc):
    """Graphs replayed side by side on two streams give what each gives by itself."""
    from lossless_bf16_exponent_zc_gb300 import embedding, moe, norm
    made = []
    for seed in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids = torch.randint(0, 700, (9000,), device="cuda", generator=g)
        dout = torch.randn((9000, 136), device="cuda", generator=g)
        logits = torch.randn((9000, 40), device="cuda", generator=g)
        experts = torch.randint(0, 40, (9000, 3), device="cuda", generator=g, dtype=torch.int32)
        w = torch.rand(136, device="cuda", generator=g)
        st, ews = zc.new_status(), embedding.workspace(9000, 700, 136)
        bws, nws = moe.balance_workspace(9000, 40), norm.workspace(9000, 136)
        stats = norm.layer_norm(dout, w, save=True)[1]

        def call(ids=ids, dout=dout, logits=logits, experts=experts, w=w, st=st, ews=ews, bws=bws, nws=nws, stats=stats):
            return [embedding.lookup_backward(dout, ids, 700, ews, st), *moe.balance_loss(logits, experts, bws),
                    *norm.layer_norm_backward(dout, dout, stats, w, nws)]

        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        made.append((graph, out, want, torch.cuda.Stream(), call))  # the call keeps what the graph reads
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, _, _, stream, _ in made:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, _, _ in made:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_from_several_threads(zc):
    import threading

    from lossless_bf16_exponent_zc_gb300 import dropout, embedding, moe, norm

    def step(seed, rounds, out):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids = torch.randint(0, 90, (500,), device="cuda", generator=g)
        table = torch.randn((90, 72), device="cuda", generator=g)
        logits, experts = torch.randn((500, 8), device="cuda", generator=g), (ids % 8).to(torch.int32)[:, None]
        w, rng, st = torch.ones(72, device="cuda"), dropout.new_rng(seed), zc.new_status()
        ews, bws, nws = embedding.workspace(500, 90, 72), moe.balance_workspace(500, 8), norm.workspace(500, 72)
        for i in range(rounds):
            x = embedding.lookup(ids, table, st)
            y = dropout.dropout(x, 0.2, rng, 1, residual=x)
            x_new, h, stats = norm.add_layer_norm(y, x, w, p=0.2, rng=rng, save=True)
            back = norm.add_layer_norm_backward(y, x, x_new, stats, w, nws, p=0.2, rng=rng)
            out.append([y, x_new, h, back.dy, back.dx, back.dweight, *moe.balance_loss(logits, experts, bws),
                        embedding.lookup_backward(back.dx, ids, 90, ews, st)])
        torch.cuda.current_stream().synchronize()

    want, got, errors = [[], []], [[], []], []
    for seed in (0, 1):
        step(seed, 1, want[seed])

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
            assert all(torch.equal(a, b) for a, b in zip(run, want[seed][0]))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("scale", [1 + 2**-40, 2**0.5 * 0.5**0.5, 0.99999999])
def test_a_residual_scale_that_is_one_in_fp32(zc, bias, scale):
    """The kernels take the scale as fp32: gradients like those of a scale of 1, which has one tensor for dy and dx."""
    args = (leaf(10, 24), leaf(10, 24), leaf(24), leaf(24) if bias else None, None, 0.0, 0)
    torch.library.opcheck(ops.add_layer_norm, (*args, scale, 1e-5))
    gx, gh = torch.randn((10, 24), device="cuda"), torch.randn((10, 24), device="cuda")
    made = []
    for s in (scale, 1.0):
        for a in args[:4]:
            if a is not None:
                a.grad = None
        x_new, h, _ = ops.add_layer_norm(*args, s, 1e-5)
        torch.autograd.backward([x_new, h], [gx, gh])
        made.append([x_new, h, *(a.grad for a in args[:4] if a is not None)])
    assert all(torch.equal(a, b) for a, b in zip(*made))
