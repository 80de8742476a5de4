"""The rest of a training step's way through a block, as measured cases: embedding, layer norm, dropout, balance loss.

perf/operators.py measures what stands around an expert-parallel exchange: routing, dispatch, combine and the block
norms.  These are the operators next to them in the same models.  The residual stream starts with the rows of an
embedding table (embedding.lookup), whose gradient adds up the tokens of every id; a block's output is dropped out and
added to the stream (dropout.dropout), where the model has layer norms instead of root-mean-square ones in the same
pass as the next block's norm (norm.layer_norm, norm.add_layer_norm); and the router's load is kept even by a loss over
its probabilities and the experts' counts (moe.balance_loss).  Every one has a gradient.

Where `own` is false run() computes them from elementary torch operations in 32 bits; where it is true it calls
the package.  exact() computes the same from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # a micro-batch's router: small enough that latency is all that counts
        {"name": "balance_small_train", "op": "balance", "tokens": 512, "experts": 64, "k": 4, "dtype": "f32",
         "score": "softmax", "sequences": 1, "masked": 0.0, "padded": 0.0},
        # a training step's router over the payload's tokens: sigmoid scores, a loss for each of eight sequences
        {"name": "balance_payload_train", "op": "balance", "tokens": 16384, "experts": 256, "k": 8, "dtype": "f32",
         "score": "sigmoid", "sequences": 8, "masked": 0.0, "padded": 0.0},
        # an odd number of experts, most of them masked out for some tokens, padding tokens whose logits are anything
        {"name": "balance_ragged_train", "op": "balance", "tokens": 5003, "experts": 61, "k": 6, "dtype": "bf16",
         "score": "softmax", "sequences": 1, "masked": 0.5, "padded": 0.2},
        # decoding: the residual addition and the next block's layer norm for a small batch
        {"name": "layer_norm_decode", "op": "layer_norm", "mode": "forward", "tokens": 8, "hidden": 4096,
         "dtype": "bf16", "params": "bf16", "branch": True, "bias": True, "p": 0.0},
        # the payload's tokens in training: dropout, residual and layer norm in one pass, both directions
        {"name": "layer_norm_payload_train", "op": "layer_norm", "mode": "train", "tokens": 16384, "hidden": 4096,
         "dtype": "bf16", "params": "f32", "branch": True, "bias": True, "p": 0.1},
        # a norm by itself, an odd width, all in 32 bits
        {"name": "layer_norm_ragged_train", "op": "layer_norm", "mode": "train", "tokens": 2331, "hidden": 1531,
         "dtype": "f32", "params": "f32", "branch": False, "bias": True, "p": 0.0},
        # a micro-batch's block output dropped out and added to the residual stream
        {"name": "dropout_small_train", "op": "dropout", "tokens": 256, "hidden": 1024, "dtype": "bf16",
         "residual": True, "p": 0.1},
        # the same over the payload's tokens
        {"name": "dropout_payload_train", "op": "dropout", "tokens": 16384, "hidden": 4096, "dtype": "bf16",
         "residual": True, "p": 0.1},
        # activations of an odd width, without a residual
        {"name": "dropout_ragged_train", "op": "dropout", "tokens": 2051, "hidden": 1021, "dtype": "f16",
         "residual": False, "p": 0.25},
        # decoding: a handful of tokens' rows of a large table
        {"name": "embedding_decode", "op": "embedding", "mode": "forward", "tokens": 8, "vocab": 131072,
         "hidden": 4096, "dtype": "bf16", "params": "bf16", "padded": 0.0, "skew": 1.0, "ids": "int64"},
        # the payload's tokens in training: their rows, and the gradient of the whole table
        {"name": "embedding_payload_train", "op": "embedding", "mode": "train", "tokens": 16384, "vocab": 131072,
         "hidden": 4096, "dtype": "bf16", "params": "bf16", "padded": 0.0, "skew": 1.0, "ids": "int64"},
        # padding among the tokens, an odd table, its gradient kept in 32 bits
        {"name": "embedding_ragged_train", "op": "embedding", "mode": "train", "tokens": 5003, "vocab": 50021,
         "hidden": 1021, "dtype": "f16", "params": "f32", "padded": 0.2, "skew": 1.0, "ids": "int32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "layer_norm", "dropout", "embedding"])
    c = {"op": op, "tokens": _log(rng, 1, 16384), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op == "balance":
        c["k"] = rng.choice([1, 2, 4, 6, 8])
        c["experts"] = max(c["k"], _log(rng, 4, 512))
        c["score"] = rng.choice(["softmax", "sigmoid"])
        c["sequences"] = min(c["tokens"], rng.choice([1, 1, 2, 7, 16]))
        c["tokens"] -= c["tokens"] % c["sequences"]
        c["masked"] = rng.choice([0.0, 0.0, 0.3, 0.9])
        c["padded"] = rng.choice([0.0, 0.1, 0.5])
    else:
        width = _log(rng, 64, 8192)
        c["hidden"] = width // 64 * 64 if rng.random() < 0.6 else width | 1
    if op == "layer_norm":
        c["mode"] = rng.choice(["forward", "train"])
        c["params"] = rng.choice([c["dtype"], "f32"])
        c["branch"] = rng.random() < 0.7
        c["bias"] = rng.random() < 0.7
        c["p"] = rng.choice([0.0, 0.1, 0.3]) if c["branch"] else 0.0
    elif op == "dropout":
        c["residual"] = rng.random() < 0.6
        c["p"] = rng.choice([0.05, 0.1, 0.25, 0.5])
    elif op == "embedding":
        c["mode"] = rng.choice(["forward", "train"])
        c["vocab"] = _log(rng, 256, 131072)
        c["params"] = rng.choice([c["dtype"], "f32"])
        c["padded"] = rng.choice([0.0, 0.0, 0.2, 0.6])
        c["skew"] = rng.choice([0.0, 0.6, 1.0, 1.4])
        c["ids"] = rng.choice(["int32", "int64"])
    groups = c.get("sequences", 1)
    most = max(work(x)["bytes"] for x in listed() if x["op"] == op)
    while work(c)["bytes"] > most:  # no dearer than the operator's largest listed case
        if op == "embedding" and c["tokens"] * 8 < c["vocab"]:
            c["vocab"] //= 2
        else:
            c["tokens"] = max(groups, c["tokens"] // 2 // groups * groups)
    return c


def _popularity(case):
    """Of a table's rows, by rank: 1 / rank^skew."""
    p = np.arange(1, case["vocab"] + 1, dtype=np.float64) ** -case["skew"]
    return p / p.sum()


def _distinct(case):
    """Expected number of table rows that the tokens ask for."""
    p = _popularity(case)
    return int((1 - np.exp(case["tokens"] * (1 - case["padded"]) * np.log1p(-np.minimum(p, 1 - 1e-12)))).sum())


def work(case):
    t, size = case["tokens"], 4 if case["dtype"] == "f32" else 2
    if case["op"] == "balance":
        e, k, s = case["experts"], case["k"], case["sequences"]
        # forward: logits, ids and mask in, counts and slopes out; backward: logits, slopes and mask in, gradient out
        return {"bytes": 3 * size * t * e + 4 * t * k + 2 * t + 12 * s * e + 8, "flops": 12 * t * e}
    d = case["hidden"]
    if case["op"] == "dropout":
        # in (and the residual) and out; backward: the output's gradient in, the input's out
        n = size * t * d * (3 if case["residual"] else 2) + size * t * d * 2
        return {"bytes": n, "flops": t * d * (5 if case["residual"] else 3)}
    p = 4 if case["params"] == "f32" else 2
    train = case["mode"] == "train"
    if case["op"] == "layer_norm":
        params = d * (2 if case["bias"] else 1)
        n = size * t * d * (4 if case["branch"] else 2) + p * params
        flops = t * d * (11 if case["branch"] else 8)
        if train:
            # statistics out and in; the gradients of both outputs and the saved stream in; those of the branch, the
            # stream and the parameters out
            n += 16 * t + size * t * d * (5 if case["branch"] else 4) + p * (params + d)
            flops += t * d * 14
        return {"bytes": n, "flops": flops}
    ids = t * (8 if case["ids"] == "int64" else 4)
    n = ids + p * _distinct(case) * d + size * t * d
    if train:  # the rows' gradient in, the whole table's out
        n += ids + size * t * d + p * case["vocab"] * d
    return {"bytes": n, "flops": t * d * (2 if train else 1)}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _gradient(g, dtype, *shape):
    """Of an output; scaled, like the loss, where 16 bits would make it subnormal."""
    return (_randn(g, *shape) * (1.0 if dtype == "f16" else 1e-3)).to(DTYPES[dtype])


def prepare(case, seed):
    g = _generator(seed)
    op, t = case["op"], case["tokens"]
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "balance":
        e, k = case["experts"], case["k"]
        logits = _randn(g, t, e) * 1.5
        masked = torch.rand((t, e), device="cuda", generator=g) < case["masked"]
        masked[0] = False  # others may lose all their experts
        logits = torch.where(masked, -math.inf, logits)
        order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
        s["experts"] = torch.where(masked.gather(1, order), -1, order).to(torch.int32).contiguous()
        s["mask"] = None
        if case["padded"]:
            pad = torch.rand(t, device="cuda", generator=g) < case["padded"]
            pad[0] = False
            s["mask"] = ~pad
            rubbish = torch.where(torch.rand((t, 1), device="cuda", generator=g) < 0.5, math.nan, math.inf)
            logits = torch.where(pad[:, None], rubbish, logits)
        s["logits"] = logits.to(dt)
        # scaled losses keep 16-bit gradients away from the subnormals
        s["dloss"] = torch.full((), (10.0 if case["dtype"] == "f16" else 0.01) * t, device="cuda")
        if own:
            from lossless_bf16_exponent_zc_gb300 import moe
            s["ws"] = moe.balance_workspace(t, e, case["sequences"])
        return s
    d = case["hidden"]
    if op == "dropout":
        s["x"] = _randn(g, t, d).to(dt)
        s["residual"] = (_randn(g, t, d) * 2).to(dt) if case["residual"] else None
        s["dout"] = _gradient(g, case["dtype"], t, d)
        s["rng"] = torch.tensor([seed * 0x9E3779B97F4A7C15 % 2**63, seed % 1000], device="cuda")
        s["call"] = 5
    elif op == "layer_norm":
        pt = DTYPES[case["params"]]
        s["x"] = (_randn(g, t, d) * 2 + _randn(g, t, 1)).to(dt)
        s["y"] = _randn(g, t, d).to(dt) if case["branch"] else None
        s["weight"] = (1 + 0.1 * _randn(g, d)).to(pt)
        s["bias"] = (0.1 * _randn(g, d)).to(pt) if case["bias"] else None
        s["residual_scale"] = 1.0
        s["rng"] = torch.tensor([seed * 0x9E3779B97F4A7C15 % 2**63, seed % 1000], device="cuda") if case["p"] else None
        s["call"] = 2
        if case["mode"] == "train":
            # what the backward pass finds: the saved stream and its statistics, and the gradients of the outputs
            s["saved"] = (_randn(g, t, d) * 2 + _randn(g, t, 1)).to(dt) if case["branch"] else s["x"]
            z = s["saved"].double()
            mean = z.mean(1, keepdim=True)
            root = 1 / torch.sqrt((z - mean).square().mean(1, keepdim=True) + EPS)
            s["stats"] = torch.cat([mean, root], 1).float()
            s["dh"] = _gradient(g, case["dtype"], t, d)
            s["dpast"] = _gradient(g, case["dtype"], t, d)
            if own:
                from lossless_bf16_exponent_zc_gb300 import norm
                s["ws"] = norm.workspace(t, d)
    else:
        v = case["vocab"]
        s["table"] = (_randn(g, v, d) * 0.02).to(DTYPES[case["params"]])
        upto = torch.from_numpy(np.cumsum(_popularity(case))).cuda()  # added up on the host, where the order is fixed
        rank = torch.searchsorted(upto, torch.rand(t, device="cuda", generator=g).double()).clamp(max=v - 1)
        ids = torch.randperm(v, device="cuda", generator=g)[rank]
        pad = torch.rand(t, device="cuda", generator=g) < case["padded"]
        s["ids"] = torch.where(pad, -1, ids).to(torch.int32 if case["ids"] == "int32" else torch.int64)
        s["scale"] = math.sqrt(d)
        if case["mode"] == "train":
            s["drows"] = _gradient(g, case["dtype"], t, d)
        if own:
            from lossless_bf16_exponent_zc_gb300 import embedding, zc
            s["status"] = zc.new_status()
            if case["mode"] == "train":
                s["ws"] = embedding.workspace(t, v, d)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"balance": _balance, "layer_norm": _layer_norm, "dropout": _dropout, "embedding": _embedding}[op](state)
    return {"balance": _plain_balance, "layer_norm": _plain_layer_norm, "dropout": _plain_dropout,
            "embedding": _plain_embedding}[op](state)


def _balance(s):
    from lossless_bf16_exponent_zc_gb300 import moe
    c = s["case"]
    b = moe.balance_loss(s["logits"], s["experts"], s["ws"], score=c["score"], sequences=c["sequences"], mask=s["mask"])
    dlogits = moe.balance_loss_backward(s["dloss"], s["logits"], b.slope, score=c["score"], mask=s["mask"])
    return {"loss": b.loss, "counts": b.counts, "slope": b.slope, "dlogits": dlogits}


def _layer_norm(s):
    from lossless_bf16_exponent_zc_gb300 import norm
    c = s["case"]
    train = c["mode"] == "train"
    if not c["branch"]:
        h, stats = norm.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, save=train)
        out = {"h": h, "stats": stats}
        if train:
            out["dx"], out["dweight"], out["dbias"] = norm.layer_norm_backward(
                s["dh"], s["saved"], s["stats"], s["weight"], s["ws"], bias=c["bias"], dresidual=s["dpast"])
        return out
    drop = {"p": c["p"], "rng": s["rng"], "call": s["call"]} if c["p"] else {}
    x_new, h, stats = norm.add_layer_norm(s["y"], s["x"], s["weight"], s["bias"], eps=EPS, save=train,
                                          residual_scale=s["residual_scale"], **drop)
    out = {"x_new": x_new, "h": h, "stats": stats}
    if train:
        b = norm.add_layer_norm_backward(s["dpast"], s["dh"], s["saved"], s["stats"], s["weight"], s["ws"],
                                         bias=c["bias"], residual_scale=s["residual_scale"], **drop)
        out.update(dy=b.dy, dx=b.dx, dweight=b.dweight, dbias=b.dbias)
    return out


def _dropout(s):
    from lossless_bf16_exponent_zc_gb300 import dropout
    p = s["case"]["p"]
    return {"out": dropout.dropout(s["x"], p, s["rng"], s["call"], residual=s["residual"]),
            "dx": dropout.dropout_backward(s["dout"], p, s["rng"], s["call"])}


def _embedding(s):
    from lossless_bf16_exponent_zc_gb300 import embedding
    c = s["case"]
    out = {"rows": embedding.lookup(s["ids"], s["table"], s["status"], scale=s["scale"], dtype=DTYPES[c["dtype"]])}
    if c["mode"] == "train":
        out["dtable"] = embedding.lookup_backward(s["drows"], s["ids"], c["vocab"], s["ws"], s["status"],
                                                  scale=s["scale"], dtype=DTYPES[c["params"]])
    return out


# ------------------------------------------------------------------ plain forms, 32 bits
def _plain_balance(s):
    c, k, e, seqs = s["case"], s["case"]["k"], s["case"]["experts"], s["case"]["sequences"]
    logits = s["logits"].float()
    open_ = logits != -math.inf
    if s["mask"] is not None:
        open_ = open_ & s["mask"][:, None]
    counted = open_.any(1)
    logits = torch.where(open_, logits, -math.inf)
    if c["score"] == "softmax":
        top = torch.where(counted[:, None], logits.amax(1, keepdim=True), 0)
        raw = torch.where(open_, torch.exp(logits - top), 0)
        total = torch.where(counted[:, None], raw.sum(1, keepdim=True), 1)
    else:
        raw = torch.where(open_, 1 / (1 + torch.exp(-logits)), 0)
        total = raw.sum(1, keepdim=True) + 1e-20
    p = raw / total
    per = lambda m: m.reshape(seqs, -1, *m.shape[1:])  # noqa: E731
    tokens = per(counted).sum(1).float()[:, None]
    chosen = torch.where(counted[:, None], s["experts"], -1)
    counts = torch.zeros((seqs, e), dtype=torch.int32, device=logits.device)
    for j in range(k):
        counts += (per(chosen[:, j])[:, :, None] == torch.arange(e, device=logits.device)).sum(1).to(torch.int32)
    slope = torch.where(tokens > 0, counts.float() * e / (seqs * k * tokens.clamp(min=1) ** 2), 0)
    loss = (slope * per(p).sum(1)).sum()
    # dp of token t is the slope of its sequence
    dp = s["dloss"] * slope.repeat_interleave(logits.shape[0] // seqs, 0)
    inner = dp - (dp * p).sum(1, keepdim=True)
    dlogits = p * inner if c["score"] == "softmax" else raw * (1 - raw) * inner / total
    return {"loss": loss, "counts": counts, "slope": slope, "dlogits": dlogits.to(s["logits"].dtype)}


_M32 = 0xFFFFFFFF


def _plain_keep(rng, call, p, tokens, width, device):
    """Which values stay, bool [tokens, width]: the 16 bits that Philox-4x32-10 (Salmon et al., 2011) has for a value,
    eight values a counter, against p in steps of 2^-16.  And the factor that makes up for the others."""
    limit = math.floor(p * 65536 + 0.5)
    groups = (width + 7) // 8
    c0 = torch.arange(groups, device=device).expand(tokens, groups)
    c1 = torch.arange(tokens, device=device)[:, None].expand(tokens, groups)
    c2 = torch.full((1, 1), call, device=device, dtype=torch.int64).expand(tokens, groups)
    c3 = (rng[1] & _M32).expand(tokens, groups)
    k0, k1 = rng[0] & _M32, (rng[0] >> 32) & _M32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # the products modulo 2^64
        c0, c1, c2, c3 = ((b >> 32) & _M32) ^ c1 ^ k0, b & _M32, ((a >> 32) & _M32) ^ c3 ^ k1, a & _M32
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    bits = torch.stack([h for w in (c0, c1, c2, c3) for h in (w & 0xFFFF, w >> 16)], 2)
    keep = bits.reshape(tokens, groups * 8)[:, :width] >= limit
    return keep, 65536 / (65536 - limit) if limit < 65536 else 0.0


def _plain_dropout(s):
    x = s["x"]
    keep, factor = _plain_keep(s["rng"], s["call"], s["case"]["p"], *x.shape, x.device)
    out = torch.where(keep, x.float() * factor, 0)
    if s["residual"] is not None:
        out = s["residual"].float() + out
    return {"out": out.to(x.dtype), "dx": torch.where(keep, s["dout"].float() * factor, 0).to(x.dtype)}


def _plain_layer_norm(s):
    c, x, dt = s["case"], s["x"].float(), s["x"].dtype
    w = s["weight"].float()
    out, keep = {}, None
    if c["branch"]:
        y = s["y"].float()
        if c["p"]:
            keep, factor = _plain_keep(s["rng"], s["call"], c["p"], *x.shape, x.device)
            y = torch.where(keep, y * factor, 0)
        x = s["residual_scale"] * x + y
        out["x_new"] = x.to(dt)
    mean = x.mean(1, keepdim=True)
    root = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    h = (x - mean) * root * w
    out["h"] = (h + s["bias"].float() if c["bias"] else h).to(dt)
    out["stats"] = torch.cat([mean, root], 1) if c["mode"] == "train" else None
    if c["mode"] == "train":
        dh, pt = s["dh"].float(), s["weight"].dtype
        mean, root = s["stats"][:, :1], s["stats"][:, 1:]
        n, u = (s["saved"].float() - mean) * root, dh * w
        g = s["dpast"].float() + root * (u - u.mean(1, keepdim=True) - n * (u * n).mean(1, keepdim=True))
        if c["branch"]:
            out["dy"] = (torch.where(keep, g * factor, 0) if c["p"] else g).to(dt)
            g = s["residual_scale"] * g
        out["dx"] = g.to(dt)
        out["dweight"] = (dh * n).sum(0).to(pt)
        out["dbias"] = dh.sum(0).to(pt) if c["bias"] else None
    return out


def _plain_embedding(s):
    c, ids = s["case"], s["ids"].long()
    there = ids >= 0
    rows = s["table"][ids.clamp(min=0)].float() * s["scale"]
    out = {"rows": torch.where(there[:, None], rows, 0).to(DTYPES[c["dtype"]])}
    if c["mode"] == "train":
        # an extra row takes the padding
        total = torch.zeros((c["vocab"] + 1, c["hidden"]), device=ids.device)
        total.index_add_(0, torch.where(there, ids, c["vocab"]), s["drows"].float())
        out["dtable"] = (total[:-1] * s["scale"]).to(s["table"].dtype)
    return out


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False  # the inputs alone: no handles of the package
    s = prepare(case, seed)
    globals()["own"] = was
    return {"balance": _exact_balance, "layer_norm": _exact_layer_norm, "dropout": _exact_dropout,
            "embedding": _exact_embedding}[case["op"]](s)


def _exact_balance(s):
    """Sequence by sequence; the gradient by automatic differentiation of the loss, its counts fixed."""
    c, k, e, seqs = s["case"], s["case"]["k"], s["case"]["experts"], s["case"]["sequences"]
    logits = s["logits"].double()
    valid = torch.ones(logits.shape[0], dtype=torch.bool, device=logits.device) if s["mask"] is None else s["mask"]
    valid = valid & ~(logits == -math.inf).all(1)
    leaf = torch.where(valid[:, None], logits, 0.0).requires_grad_(True)
    p = torch.sigmoid(leaf) if c["score"] == "sigmoid" else torch.softmax(leaf, 1)
    if c["score"] == "sigmoid":
        p = p / (p.sum(1, keepdim=True) + 1e-20)
    n = logits.shape[0] // seqs
    loss, slopes = torch.zeros((), dtype=torch.float64, device=logits.device), []
    for q in range(seqs):
        part = slice(q * n, q * n + n)
        v = valid[part]
        tokens = int(v.sum())
        ids = s["experts"][part][v].reshape(-1)
        f = torch.bincount(ids[ids >= 0].long(), minlength=e).double() / (k * max(tokens, 1))
        mean = (p[part] * v[:, None]).sum(0) / max(tokens, 1)
        loss = loss + e * (f * mean).sum() / seqs
        slopes.append(e * f / (seqs * max(tokens, 1)))
    dlogits, = torch.autograd.grad(loss, leaf, s["dloss"].double())
    return {"loss": loss.detach(), "counts": None, "slope": torch.stack(slopes), "dlogits": dlogits}


def _exact_keep(s, tokens, width):
    """The generator in numpy's 64-bit words, a round at a time over all counters."""
    word = np.uint64
    low, half = word(0xFFFFFFFF), word(32)
    seed, offset = (int(v) for v in s["rng"].tolist())
    groups = -(-width // 8)
    at = np.arange(tokens * groups, dtype=np.uint64)
    x = [at % word(groups), at // word(groups), np.full_like(at, s["call"]), np.full_like(at, offset % 2**32)]
    key = [seed % 2**32, seed // 2**32 % 2**32]
    for step in range(10):
        first, second = x[0] * word(0xD2511F53), x[2] * word(0xCD9E8D57)
        k = [word((key[0] + step * 0x9E3779B9) % 2**32), word((key[1] + step * 0xBB67AE85) % 2**32)]
        x = [(second >> half) ^ x[1] ^ k[0], second & low, (first >> half) ^ x[3] ^ k[1], first & low]
    bits = np.stack(x, 1).astype(np.uint32).astype("<u4").view("<u2").reshape(tokens, groups * 8)[:, :width]
    limit = int(s["case"]["p"] * 65536 + 0.5)
    return torch.from_numpy(bits >= limit).cuda(), 1 / (1 - limit / 65536) if limit < 65536 else 0.0


def _exact_dropout(s):
    keep, factor = _exact_keep(s, *s["x"].shape)
    scaled = lambda z: z.double().masked_fill(~keep, 0.0) * factor  # noqa: E731
    out = scaled(s["x"])
    return {"out": out if s["residual"] is None else s["residual"].double() + out, "dx": scaled(s["dout"])}


def _exact_layer_norm(s):
    """Forward from the definition; backward by automatic differentiation of the norm at the saved stream."""
    c, d = s["case"], s["case"]["hidden"]
    w = s["weight"].double().requires_grad_(True)
    b = s["bias"].double().requires_grad_(True) if c["bias"] else None

    def normed(z):
        centred = z - z.sum(1, keepdim=True) / d
        root = torch.rsqrt(centred.square().sum(1, keepdim=True) / d + EPS)
        return centred * root * w + (0 if b is None else b), root

    x, out = s["x"].double(), {}
    if c["branch"]:
        y = s["y"].double()
        if c["p"]:
            keep, factor = _exact_keep(s, *y.shape)
            y = y * keep * factor
        x = out["x_new"] = s["residual_scale"] * x + y
    h, root = normed(x)
    out["h"], out["stats"] = h.detach(), None
    if c["mode"] == "train":
        out["stats"] = torch.cat([x.mean(1, keepdim=True), root.detach()], 1)
        leaf = s["saved"].double().requires_grad_(True)
        need = [leaf, w] + ([b] if c["bias"] else [])
        dx, dweight, *dbias = torch.autograd.grad(normed(leaf)[0], need, s["dh"].double())
        dx = dx + s["dpast"].double()
        if c["branch"]:
            out["dy"] = dx * keep * factor if c["p"] else dx
            dx = dx * s["residual_scale"]
        out.update(dx=dx, dweight=dweight, dbias=dbias[0] if dbias else None)
    return out


def _exact_embedding(s):
    c, ids = s["case"], s["ids"].long()
    rows = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device="cuda")
    at = torch.nonzero(ids >= 0)[:, 0]
    rows[at] = s["table"][ids[at]].double() * s["scale"]
    out = {"rows": rows}
    if c["mode"] == "train":
        # differences of the running sum over the tokens sorted by id would lose bits: a sum for every id
        table = torch.zeros((c["vocab"], c["hidden"]), dtype=torch.float64, device="cuda")
        order = at[torch.sort(ids[at], stable=True).indices]
        seen, count = torch.unique_consecutive(ids[order], return_counts=True)
        first = count.cumsum(0) - count
        for turn in range(0, int(count.max()) if len(count) else 0):  # the turn-th token of every id that has so many
            more = count > turn
            table[seen[more]] += s["drows"][order[first[more] + turn]].double()
        out["dtable"] = table * s["scale"]
    return out
