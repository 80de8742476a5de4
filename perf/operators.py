"""The operators around an expert-parallel layer, as measured cases: routing, dispatch, combine and the block norms.

The library moves the activations of mixture-of-experts layers compressed between ranks; these operators stand on
both sides of that exchange.  A block normalises its input (norm.pre_norm), picks experts for every token
(moe.route), sorts the tokens by expert into the contiguous pieces that are exchanged (moe.dispatch), brings the
experts' outputs back weighted (moe.combine) and joins them to the residual stream through the block's second
norm, its gate and its residual scale, with the next block's first norm in the same pass (norm.post_norm).  Every
one has a gradient.

Where `own` is false run() computes them from elementary torch operations in 32 bits; where it is true it calls
the package.  exact() computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    return [
        # one decoding step of a small batch: latency is all that counts
        {"name": "route_decode", "op": "route", "mode": "forward", "tokens": 8, "experts": 128, "k": 8,
         "dtype": "f32", "score": "softmax", "renormalize": True, "masked": 0.0},
        # a training step's router over the payload's tokens: sigmoid scores with a balancing bias, both directions
        {"name": "route_train", "op": "route", "mode": "train", "tokens": 16384, "experts": 256, "k": 8,
         "dtype": "f32", "score": "sigmoid", "renormalize": True, "masked": 0.0},
        # an odd number of experts, most of them masked out for some tokens (restricted groups), unnormalised weights
        {"name": "route_ragged_train", "op": "route", "mode": "train", "tokens": 5003, "experts": 61, "k": 6,
         "dtype": "bf16", "score": "softmax", "renormalize": False, "masked": 0.5},
        # decoding: a handful of tokens to their experts
        {"name": "dispatch_decode", "op": "dispatch", "mode": "forward", "tokens": 8, "experts": 128, "k": 8,
         "hidden": 4096, "dtype": "bf16", "dropped": 0.0, "skew": 1.2},
        # a prefill's tokens with padding among them, widths that no vector divides, both directions
        {"name": "dispatch_ragged_train", "op": "dispatch", "mode": "train", "tokens": 2051, "experts": 61, "k": 3,
         "hidden": 1021, "dtype": "f16", "dropped": 0.2, "skew": 0.6},
        # the 16384 x 4096 all-to-all payload, four experts a token, skewed like its destinations, both directions
        {"name": "dispatch_payload_train", "op": "dispatch", "mode": "train", "tokens": 16384, "experts": 64, "k": 4,
         "hidden": 4096, "dtype": "bf16", "dropped": 0.0, "skew": 1.2},
        # decoding: the experts' outputs of a handful of tokens back into token order
        {"name": "combine_decode", "op": "combine", "mode": "forward", "tokens": 8, "experts": 128, "k": 8,
         "hidden": 4096, "dtype": "bf16", "dropped": 0.0, "skew": 1.2},
        # the payload's way back, with the gradients of the experts' outputs and of the weights
        {"name": "combine_payload_train", "op": "combine", "mode": "train", "tokens": 16384, "experts": 64, "k": 4,
         "hidden": 4096, "dtype": "bf16", "dropped": 0.05, "skew": 1.2},
        # decoding: both norms around a block for a small batch
        {"name": "norm_decode", "op": "norm", "mode": "forward", "tokens": 8, "hidden": 4096, "dtype": "bf16",
         "params": "bf16", "gate": "channel", "sequences": 1, "next": True},
        # a prefill over the payload's tokens
        {"name": "norm_prefill", "op": "norm", "mode": "forward", "tokens": 16384, "hidden": 4096, "dtype": "bf16",
         "params": "bf16", "gate": "channel", "sequences": 1, "next": True},
        # its gradient in training, parameters kept in 32 bits
        {"name": "norm_payload_backward", "op": "norm", "mode": "backward", "tokens": 16384, "hidden": 4096,
         "dtype": "bf16", "params": "f32", "gate": "channel", "sequences": 1, "next": True},
        # one gate row for each of several sequences, an odd width, all in 32 bits
        {"name": "norm_ragged_backward", "op": "norm", "mode": "backward", "tokens": 2331, "hidden": 1531,
         "dtype": "f32", "params": "f32", "gate": "sequence", "sequences": 7, "next": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "norm"])
    c = {"op": op, "tokens": _log(rng, 1, 16384), "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op != "norm":
        c["k"] = rng.choice([1, 2, 3, 4, 6, 8])
        c["experts"] = max(c["k"], _log(rng, 4, 512))
    c["mode"] = rng.choice(["forward", "backward" if op == "norm" else "train"])
    if op == "route":
        c["score"] = rng.choice(["softmax", "sigmoid"])
        c["renormalize"] = c["k"] > 1 and rng.random() < 0.5  # one weight alone is 1, with no gradient
        c["masked"] = rng.choice([0.0, 0.0, 0.3, 0.9])
    else:
        width = _log(rng, 64, 8192)
        c["hidden"] = width // 64 * 64 if rng.random() < 0.6 else width | 1
    if op == "norm":
        c["params"] = rng.choice([c["dtype"], "f32"])
        c["gate"] = rng.choice(["none", "channel", "token", "sequence"])
        c["sequences"] = min(c["tokens"], rng.randint(2, 9)) if c["gate"] == "sequence" else 1
        c["next"] = rng.random() < 0.75
    elif op != "route":
        c["dropped"] = rng.choice([0.0, 0.0, 0.1, 0.5])
        c["skew"] = rng.choice([0.0, 0.6, 1.2])
    groups = c.get("sequences", 1)
    c["tokens"] -= c["tokens"] % groups
    most = max(work(x)["bytes"] for x in listed() if x["op"] == op)
    while work(c)["bytes"] > most:  # no dearer than the operator's largest listed case
        c["tokens"] = max(groups, c["tokens"] // 2 // groups * groups)
    return c


def work(case):
    t, size = case["tokens"], 4 if case["dtype"] == "f32" else 2
    train = case["mode"] == "train"
    if case["op"] == "route":
        e, k = case["experts"], case["k"]
        n = size * t * e + 8 * t * k + (4 * e if case["score"] == "sigmoid" else 0)
        if train:  # the weights' gradient in, the logits' gradient out
            n += 4 * t * k + size * t * e
        return {"bytes": n, "flops": t * e * (8 if train else 4) + 2 * t * e * k}
    d = case["hidden"]
    if case["op"] == "dispatch":
        e, k = case["experts"], case["k"]
        n = size * t * d * (1 + k) + 4 * t * k + 8 * t * k + 4 * (e + 1)
        if train:  # the rows' gradient in, the tokens' gradient out
            n += size * t * d * (1 + k)
        return {"bytes": n, "flops": t * k * d if train else 0}
    if case["op"] == "combine":
        k = case["k"]
        n = size * t * d * (1 + k) + 8 * t * k
        if train:  # the output's gradient in, the rows' and the weights' gradients out
            n += size * t * d * (1 + k) + 4 * t * k
        return {"bytes": n, "flops": 2 * t * k * d + (3 * t * k * d if train else 0)}
    p = 4 if case["params"] == "f32" else 2
    gate = {"none": 0, "channel": d, "token": t, "sequence": case["sequences"] * d}[case["gate"]]
    params = d + gate + (d if case["next"] else 0)
    if case["mode"] == "forward":  # y, x in; the new x and the next block's input out
        return {"bytes": size * t * d * (4 if case["next"] else 3) + p * params,
                "flops": t * d * (11 if case["next"] else 7)}
    # the gradients of both outputs, y and the new x in; the gradients of y, x and the parameters out
    return {"bytes": size * t * d * (6 if case["next"] else 4) + 2 * p * params,
            "flops": t * d * (28 if case["next"] else 16)}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _activations(g, dtype, *shape):
    """0.5 x Student-t with 4 degrees of freedom: the heavy tails of an MoE payload."""
    chi = torch.zeros(shape, device="cuda")
    for _ in range(4):
        z = _randn(g, *shape)
        chi += z * z
    return (_randn(g, *shape) * 0.5 / (chi / 4).sqrt()).to(DTYPES[dtype])


def _experts(g, case):
    """Expert ids int32 [tokens, k]: distinct within a token, popularity 1 / rank^skew; -1 where a slot is not routed
    (padding tokens lose all their slots, others single ones)."""
    t, e, k = case["tokens"], case["experts"], case["k"]
    popularity = -case["skew"] * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32))
    gumbel = -torch.log(-torch.log(torch.rand((t, e), device="cuda", generator=g).clamp(1e-7, 1 - 1e-7)))
    ids = torch.sort(popularity + gumbel, dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)
    lost = torch.rand((t, 1), device="cuda", generator=g) < case["dropped"] / 2
    lost = lost | (torch.rand((t, k), device="cuda", generator=g) < case["dropped"] / 2)
    return torch.where(lost, -1, ids).contiguous()


def _sorted(experts, num_experts):
    """positions, slots and offsets of the stable sort by expert; unrouted slots come last."""
    key = experts.reshape(-1)
    valid = (key >= 0) & (key < num_experts)
    key = torch.where(valid, key, num_experts)
    ordered, slots = torch.sort(key, stable=True)
    place = torch.empty_like(slots)
    place[slots] = torch.arange(slots.numel(), device=slots.device)
    positions = torch.where(valid, place, -1 - place).reshape(experts.shape).to(torch.int32)
    offsets = (ordered[None, :] < torch.arange(num_experts + 1, device=key.device)[:, None]).sum(1)
    return positions, slots.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    op, t = case["op"], case["tokens"]
    s = {"case": case}
    if op == "route":
        e, k = case["experts"], case["k"]
        logits = _randn(g, t, e) * 1.5
        masked = torch.rand((t, e), device="cuda", generator=g) < case["masked"]
        masked[0] = False  # others may lose all their experts
        s["logits"] = torch.where(masked, -math.inf, logits).to(DTYPES[case["dtype"]])
        s["bias"] = _randn(g, e) * 0.1 if case["score"] == "sigmoid" else None
        s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
        if case["mode"] == "train":
            s["dweights"] = _randn(g, t, k)
    elif op == "dispatch":
        s["x"] = _activations(g, case["dtype"], t, case["hidden"])
        s["experts"] = _experts(g, case)
        if case["mode"] == "train":
            s["drows"] = (_randn(g, t * case["k"], case["hidden"]) * 1e-3).to(DTYPES[case["dtype"]])
            if case["dtype"] == "f16":  # scaled losses keep 16-bit gradients away from the subnormals
                s["drows"] = (s["drows"] * 1024).contiguous()
        if own:
            from lossless_bf16_exponent_zc_gb300 import moe, zc
            s["ws"], s["status"] = moe.workspace(t, case["k"], case["experts"]), zc.new_status()
    elif op == "combine":
        s["rows"] = _activations(g, case["dtype"], t * case["k"], case["hidden"])
        s["positions"] = _sorted(_experts(g, case), case["experts"])[0]
        w = torch.rand((t, case["k"]), device="cuda", generator=g)
        s["weights"] = w / w.sum(1, keepdim=True)
        if case["mode"] == "train":
            s["dout"] = _randn(g, t, case["hidden"]).to(DTYPES[case["dtype"]])
        if own:
            from lossless_bf16_exponent_zc_gb300 import zc
            s["status"] = zc.new_status()
    else:
        d, dt, pt = case["hidden"], DTYPES[case["dtype"]], DTYPES[case["params"]]
        s["y"] = _activations(g, case["dtype"], t, d)
        s["x"] = (_randn(g, t, d) * 2).to(dt)  # the residual stream: the saved new one in the backward pass
        s["weight"] = (1 + 0.1 * _randn(g, d)).to(pt)
        s["next_weight"] = (1 + 0.1 * _randn(g, d)).to(pt) if case["next"] else None
        shape = {"none": None, "channel": (1, d), "token": (t, 1), "sequence": (case["sequences"], d)}[case["gate"]]
        s["gate"] = (0.5 * _randn(g, *shape)).to(pt) if shape else None
        s["residual_scale"] = 0.75
        if case["mode"] == "backward":
            s["dx_new"] = _randn(g, t, d).to(dt)
            s["dh"] = _randn(g, t, d).to(dt) if case["next"] else None
            if own:
                from lossless_bf16_exponent_zc_gb300 import norm
                s["ws"] = norm.workspace(t, d)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _route, "dispatch": _dispatch, "combine": _combine, "norm": _norm}[op](state)
    return {"route": _plain_route, "dispatch": _plain_dispatch, "combine": _plain_combine, "norm": _plain_norm}[op](state)


def _route(s):
    from lossless_bf16_exponent_zc_gb300 import moe
    c = s["case"]
    weights, experts = moe.route(s["logits"], c["k"], score=c["score"], bias=s["bias"],
                                 renormalize=c["renormalize"], scale=s["scale"])
    out = {"weights": weights, "experts": experts}
    if c["mode"] == "train":
        out["dlogits"] = moe.route_backward(s["dweights"], s["logits"], experts, score=c["score"],
                                            renormalize=c["renormalize"], scale=s["scale"])
    return out


def _dispatch(s):
    from lossless_bf16_exponent_zc_gb300 import moe
    c = s["case"]
    rows, plan = moe.dispatch(s["x"], s["experts"], c["experts"], s["ws"])
    out = {"rows": rows, "positions": plan.positions, "slots": plan.slots, "offsets": plan.offsets}
    if c["mode"] == "train":
        out["dx"] = moe.dispatch_backward(s["drows"], plan.positions, s["status"])
    return out


def _combine(s):
    from lossless_bf16_exponent_zc_gb300 import moe
    out = {"out": moe.combine(s["rows"], s["weights"], s["positions"], s["status"])}
    if s["case"]["mode"] == "train":
        out["drows"], out["dweights"] = moe.combine_backward(s["dout"], s["rows"], s["weights"], s["positions"],
                                                             s["status"])
    return out


def _norm(s):
    from lossless_bf16_exponent_zc_gb300 import norm
    if s["case"]["mode"] == "forward":
        x_new, h = norm.post_norm(s["y"], s["x"], s["weight"], gate=s["gate"], residual_scale=s["residual_scale"],
                                  next_weight=s["next_weight"], eps=EPS)
        return {"x_new": x_new, "h": h}
    g = norm.post_norm_backward(s["dx_new"], s["dh"], s["y"], s["x"], s["weight"], s["ws"], gate=s["gate"],
                                residual_scale=s["residual_scale"], next_weight=s["next_weight"], eps=EPS)
    return {"dy": g.dy, "dx": g.dx, "dweight": g.dweight, "dgate": g.dgate, "dnext_weight": g.dnext_weight}


# ------------------------------------------------------------------ plain forms, 32 bits
def _plain_route(s):
    c, k = s["case"], s["case"]["k"]
    logits = s["logits"].float()
    masked = logits == -math.inf
    scores = 1 / (1 + torch.exp(-logits)) if c["score"] == "sigmoid" else logits
    choice = torch.where(masked, -math.inf, scores + s["bias"]) if s["bias"] is not None else scores
    order = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    picked = ~masked.gather(1, order)
    if c["score"] == "softmax":
        top = logits.amax(1, keepdim=True)
        p = torch.where(masked, 0, torch.exp(logits - top))
        p = torch.where(masked, 0, p / p.sum(1, keepdim=True))
    else:
        p = torch.where(masked, 0, scores)
    chosen = torch.where(picked, p.gather(1, order), 0)
    total = chosen.sum(1, keepdim=True) + 1e-20
    weights = s["scale"] * (chosen / total if c["renormalize"] else chosen)
    out = {"weights": weights, "experts": torch.where(picked, order, -1).to(torch.int32)}
    if c["mode"] == "train":
        g = torch.where(picked, s["dweights"], 0) * s["scale"]
        if c["renormalize"]:
            g = torch.where(picked, (g - (g * chosen).sum(1, keepdim=True) / total) / total, 0)
        dp = torch.zeros_like(p).scatter_add(1, order, g)
        if c["score"] == "softmax":
            dlogits = p * (dp - (dp * p).sum(1, keepdim=True))
        else:
            dlogits = dp * p * (1 - p)
        out["dlogits"] = dlogits.to(s["logits"].dtype)
    return out


def _plain_dispatch(s):
    c, k = s["case"], s["case"]["k"]
    positions, slots, offsets = _sorted(s["experts"], c["experts"])
    routed = torch.arange(slots.numel(), device=slots.device) < offsets[-1]
    rows = torch.where(routed[:, None], s["x"][slots.long() // k], 0)
    out = {"rows": rows, "positions": positions, "slots": slots, "offsets": offsets}
    if c["mode"] == "train":
        there = positions >= 0
        g = s["drows"][positions.clamp(min=0).long()].float()
        out["dx"] = torch.where(there[:, :, None], g, 0).sum(1).to(s["x"].dtype)
    return out


def _plain_combine(s):
    rows, positions = s["rows"], s["positions"]
    there = positions >= 0
    at = positions.clamp(min=0).long()
    picked = torch.where(there[:, :, None], rows[at].float(), 0)
    out = {"out": (picked * s["weights"][:, :, None]).sum(1).to(rows.dtype)}
    if s["case"]["mode"] == "train":
        dout = s["dout"].float()
        drows = torch.where(there[:, :, None], s["weights"][:, :, None] * dout[:, None, :], 0)
        place = torch.where(there, positions, -1 - positions).reshape(-1).long()
        out["drows"] = torch.empty_like(rows)
        out["drows"][place] = drows.reshape(rows.shape).to(rows.dtype)
        out["dweights"] = (picked * dout[:, None, :]).sum(2)
    return out


def _gate_rows(gate, tokens):
    """The gate of each token, [tokens, hidden or 1]."""
    return gate.repeat_interleave(tokens // gate.shape[0], 0) if gate.shape[0] > 1 else gate


def _plain_norm(s):
    c, t = s["case"], s["case"]["tokens"]
    y, x, w = s["y"].float(), s["x"].float(), s["weight"].float()
    gate = _gate_rows(s["gate"].float(), t) if s["gate"] is not None else 1.0
    a, dt, pt = s["residual_scale"], s["y"].dtype, s["weight"].dtype
    r = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + EPS)
    n = y * r
    if c["mode"] == "forward":
        x_new, h = a * x + gate * (n * w), None
        if c["next"]:
            h = (x_new / torch.sqrt((x_new * x_new).mean(1, keepdim=True) + EPS) * s["next_weight"].float()).to(dt)
        return {"x_new": x_new.to(dt), "h": h}
    g, dnext = s["dx_new"].float(), None
    if c["next"]:
        dh, r2 = s["dh"].float(), 1 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
        n2, u = x * r2, dh * s["next_weight"].float()
        g = g + r2 * (u - n2 * (u * n2).mean(1, keepdim=True))
        dnext = (dh * n2).sum(0).to(pt)
    dgate = None
    if c["gate"] != "none":
        e = g * (n * w)
        e = e.sum(1, keepdim=True) if c["gate"] == "token" else e
        dgate = e.reshape(s["gate"].shape[0], -1, e.shape[1]).sum(1).to(pt)
    v = g * gate
    dweight = (v * n).sum(0).to(pt)
    v = v * w
    dy = r * (v - n * (v * n).mean(1, keepdim=True))
    return {"dy": dy.to(dt), "dx": (a * g).to(dt), "dweight": dweight, "dgate": dgate, "dnext_weight": dnext}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    was = globals()["own"]
    globals()["own"] = False  # the inputs alone: no handles of the package
    s = prepare(case, seed)
    globals()["own"] = was
    return {"route": _exact_route, "dispatch": _exact_dispatch, "combine": _exact_combine, "norm": _exact_norm}[
        case["op"]](s)


def _exact_route(s):
    """Weights and gradients for the experts of a selection made one at a time, largest first, lowest index on ties."""
    c, k = s["case"], s["case"]["k"]
    l32 = s["logits"].float()
    l = l32.double()
    choice = l32.clone() if c["score"] == "softmax" else 1 / (1 + torch.exp(-l32)) + s["bias"]
    choice[l32 == -math.inf] = -math.inf
    index = torch.arange(c["experts"], device=l.device).expand_as(l)
    chosen = torch.zeros_like(l, dtype=torch.bool)
    picks = []
    for _ in range(k):
        best = torch.where(chosen, -math.inf, choice).amax(1, keepdim=True)
        first = torch.where(~chosen & (choice == best), index, c["experts"]).amin(1, keepdim=True)
        first = torch.where(best == -math.inf, -1, first)
        picks.append(first)
        chosen = chosen | (index == first)
    p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    total = (p * chosen).sum(1, keepdim=True) + 1e-20
    f = p / total if c["renormalize"] else p
    at = torch.cat(picks, 1)
    take = lambda m: torch.where(at >= 0, m.gather(1, at.clamp(min=0)), 0.0)  # noqa: E731
    out = {"weights": s["scale"] * take(f), "experts": None}
    if c["mode"] == "train":
        # directional derivatives by the chain rule over the full score matrix, masked to the chosen experts
        g = torch.zeros_like(l)
        for j in range(k):
            g = g + (index == at[:, j:j + 1]) * s["dweights"][:, j:j + 1].double() * s["scale"]
        if c["renormalize"]:
            g = chosen * (g - (g * f).sum(1, keepdim=True)) / total
        slope = p * (1 - p) * g if c["score"] == "sigmoid" else p * g - p * (p * g).sum(1, keepdim=True)
        out["dlogits"] = slope
    return out


def _exact_place(experts, num_experts):
    """Row of every slot by counting: slots of smaller experts, then earlier slots of the same one."""
    key = torch.where((experts >= 0) & (experts < num_experts), experts, num_experts).reshape(-1).long().cpu()
    count = torch.zeros(num_experts + 2, dtype=torch.long)
    count[1:] = torch.bincount(key, minlength=num_experts + 1)
    start = count.cumsum(0)
    place = torch.empty_like(key)
    for e in range(num_experts + 1):
        of = torch.nonzero(key == e)[:, 0]
        place[of] = start[e] + torch.arange(of.numel())
    return place.cuda(), (key < num_experts).cuda()


def _exact_dispatch(s):
    c, k = s["case"], s["case"]["k"]
    t = c["tokens"]
    place, routed = _exact_place(s["experts"], c["experts"])
    x = s["x"].double()
    rows = torch.zeros((t * k, c["hidden"]), dtype=torch.float64, device="cuda")
    for j in range(k):
        rows[place.view(t, k)[:, j]] = x * routed.view(t, k)[:, j, None]
    out = {"rows": rows, "positions": None, "slots": None, "offsets": None}
    if c["mode"] == "train":
        dx = torch.zeros_like(x)
        for j in range(k):
            dx += s["drows"][place.view(t, k)[:, j]].double() * routed.view(t, k)[:, j, None]
        out["dx"] = dx
    return out


def _exact_combine(s):
    t, k, d = s["case"]["tokens"], s["case"]["k"], s["case"]["hidden"]
    out = torch.zeros((t, d), dtype=torch.float64, device="cuda")
    train = s["case"]["mode"] == "train"
    drows = torch.zeros((t * k, d), dtype=torch.float64, device="cuda") if train else None
    dweights = torch.zeros((t, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        token = torch.nonzero(s["positions"][:, j] >= 0)[:, 0]
        row = s["positions"][token, j].long()
        w, y = s["weights"][token, j].double()[:, None], s["rows"][row].double()
        out[token] += w * y
        if train:
            dout = s["dout"][token].double()
            drows[row] = w * dout
            dweights[token, j] = torch.einsum("td,td->t", dout, y)
    return {"out": out, "drows": drows, "dweights": dweights} if train else {"out": out}


def _exact_norm(s):
    """Forward from the definition; backward by automatic differentiation of the definition, in 64 bits."""
    c, t = s["case"], s["case"]["tokens"]
    d = c["hidden"]
    names = [n for n in ("y", "weight", "gate", "next_weight") if s[n] is not None]
    v = {n: s[n].double().requires_grad_(c["mode"] == "backward") for n in names}

    def rms(z):
        return z * torch.rsqrt(z.square().sum(1, keepdim=True) / d + EPS)

    branch = rms(v["y"]) * v["weight"]
    if "gate" in v:
        rows = v["gate"].shape[0]
        branch = (branch.view(rows, t // rows, d) * v["gate"].view(rows, 1, -1)).view(t, d)
    if c["mode"] == "forward":
        x_new = s["residual_scale"] * s["x"].double() + branch
        return {"x_new": x_new, "h": rms(x_new) * v["next_weight"] if c["next"] else None}
    # the new x is saved, so its own gradient comes from a leaf; the branch's follows from it
    leaf = s["x"].double().requires_grad_(True)
    g, dnext = s["dx_new"].double(), None
    if c["next"]:
        got = torch.autograd.grad(rms(leaf) * v["next_weight"], (leaf, v["next_weight"]), s["dh"].double())
        g, dnext = g + got[0], got[1]
    need = [n for n in names if n != "next_weight"]
    got = dict(zip(need, torch.autograd.grad(branch, [v[n] for n in need], g)))
    return {"dy": got["y"], "dx": s["residual_scale"] * g, "dweight": got["weight"], "dgate": got.get("gate"),
            "dnext_weight": dnext}
