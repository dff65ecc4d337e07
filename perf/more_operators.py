"""Cases of the operators around a mixture-of-experts block: the router (scores,
balance bias, expert groups, top-k, weights) and its gradient, the dispatch of
tokens' rows into the order of their experts, the weighted way back and its
gradient, and the norms after and before a block with its gate and residual
scale, forward and backward.

``run`` computes a case in plain torch operations, or with the library's
kernels where ``own`` is true.
"""
import math

import torch

own = False

E4M3_MAX = 448.0          # largest finite e4m3 value
SCALE_MIN = 2.0 ** -126   # smallest row scale: its reciprocal is finite
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZES = {"f32": 4, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------ cases ---

def _route(name, tokens, experts, k, scores, dtype, groups=1, top_groups=1, group_top=1,
           bias=False, renormalise=True, scale=1.0, masked=False, op="route"):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "k": k,
            "scores": scores, "dtype": dtype, "groups": groups, "top_groups": top_groups,
            "group_top": group_top, "bias": bias, "renormalise": renormalise, "scale": scale,
            "masked": masked}


def _dispatch(name, tokens, k, experts, hidden, dtype, capacity):
    return {"name": name, "op": "dispatch", "tokens": tokens, "k": k, "experts": experts,
            "hidden": hidden, "dtype": dtype, "capacity": capacity, "zipf": 0.6}


def _combine(name, tokens, k, hidden, dtype, shared, op="combine"):
    return {"name": name, "op": op, "tokens": tokens, "k": k, "experts": 64, "hidden": hidden,
            "dtype": dtype, "shared": shared, "capacity": False, "zipf": 0.6}


def _block(name, rows, hidden, dtype, out, post, gate, op="block_norm"):
    case = {"name": name, "op": op, "rows": rows, "hidden": hidden, "dtype": dtype,
            "post": post, "gate": gate, "residual_scale": 0.9, "block_scale": 0.25}
    if op == "block_norm":
        case["out"] = out
    return case


def listed():
    return [
        # one new token's router, softmax over a few experts: latency alone
        _route("route 1x64 bf16", 1, 64, 6, "softmax", "bf16"),
        # a prefill's 16384 tokens, sigmoid scores with a balance bias, experts in 8 groups
        _route("route 16384x256 f32 grouped", 16384, 256, 8, "sigmoid", "f32", 8, 4, 2, True,
               True, 2.5),
        # training: the softmax router's gradient over every expert, an odd number of them
        _route("route backward 16384x129 f32", 16384, 129, 4, "softmax", "f32",
               renormalise=False, op="route_backward"),
        # a decode batch of 8-bit rows to 64 experts, in capacity-padded buffers
        _dispatch("dispatch 128x7168 e4m3", 128, 8, 64, 7168, "e4m3", True),
        # a prefill's rows after the 8-bit norm, packed by expert
        _dispatch("dispatch 16384x7168 e4m3", 16384, 8, 256, 7168, "e4m3", False),
        # the way back of a small odd batch, with the shared expert's rows
        _combine("combine 509x1021 f32", 509, 3, 1021, "f32", True),
        # the way back of the prefill dispatch
        _combine("combine 16384x7168 bf16", 16384, 8, 7168, "bf16", False),
        # training: gradients of the rows and of the weights
        _combine("combine backward 16384x4096 bf16", 16384, 8, 4096, "bf16", False,
                 "combine_backward"),
        # one new token after the AllReduce of a block's output
        _block("block norm 1x4096 bf16", 1, 4096, "bf16", "bf16", True, "columns"),
        # a prefill's tokens, quantised for the 8-bit dispatch
        _block("block norm 16384x7168 bf16 to e4m3", 16384, 7168, "bf16", "e4m3", True,
               "columns"),
        # training step of the largest AllReduce size
        _block("block norm backward 32768x4096 bf16", 32768, 4096, "bf16", None, True,
               "columns", "block_norm_backward"),
        # an odd hidden size, a gate of its own for every row
        _block("block norm backward 1000x4099 f32", 1000, 4099, "f32", None, True, "rows",
               "block_norm_backward"),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v))


def _size(rng, lo, hi):
    """Log-uniform; two in three rounded to a multiple of 64, as model sizes are."""
    v = _log(rng, lo, hi)
    return max(64, (v + 32) // 64 * 64) if rng.random() < 2 / 3 else v


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "dispatch", "combine",
                     "combine_backward", "block_norm", "block_norm_backward"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        each = max(2, _log(rng, 4, 256) // groups)
        top_groups = rng.randint(1, groups)
        renormalise = rng.random() < 0.6
        # the one weight of a renormalised row is a constant: it has no gradient
        least = 2 if op == "route_backward" and renormalise else 1
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": each * groups,
                "k": rng.randint(least, min(10, each * top_groups)),
                "scores": rng.choice(["softmax", "sigmoid"]), "dtype": rng.choice(["f32", "bf16"]),
                "groups": groups, "top_groups": top_groups, "group_top": rng.choice([1, 2]),
                "bias": rng.random() < 0.6, "renormalise": renormalise,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.random() < 0.3}
    if op in ("dispatch", "combine", "combine_backward"):
        experts = _log(rng, 4, 256)
        case = {"op": op, "tokens": _log(rng, 1, 16384), "k": rng.randint(1, min(8, experts)),
                "experts": experts, "hidden": _size(rng, 64, 7168),
                "dtype": rng.choice(["f32", "bf16"] if op != "dispatch"
                                    else ["f32", "bf16", "e4m3", "e4m3"]),
                "capacity": rng.random() < 0.4, "zipf": rng.choice([0.0, 0.6, 1.2])}
        if op != "dispatch":
            case["shared"] = op == "combine" and rng.random() < 0.5
        # at most the bytes of the largest listed case of the operator
        most = 131072 * (7168 if op == "dispatch" else 14336 if op == "combine" else 8192)
        row = case["k"] * case["hidden"] * SIZES[case["dtype"]] * (2 if case["capacity"] else 1)
        case["tokens"] = max(1, min(case["tokens"], most // row))
        return case
    case = {"op": op, "rows": _log(rng, 1, 32768), "hidden": _size(rng, 64, 16384),
            "dtype": rng.choice(["f32", "bf16", "bf16"]), "post": rng.random() < 0.7,
            "gate": rng.choice(["none", "columns", "rows"]),
            "residual_scale": rng.choice([1.0, 0.9]), "block_scale": rng.choice([1.0, 0.25])}
    if op == "block_norm":
        case["out"] = rng.choice([case["dtype"], "e4m3"])
    # at most half the elements of the largest listed case, for f32 rows and gates a row
    case["rows"] = max(1, min(case["rows"], (1 << 25) // case["hidden"]))
    return case


# ----------------------------------------------------------------- inputs ---

def _router_inputs(case, s, g):
    tokens, experts, k = case["tokens"], case["experts"], case["k"]
    logits = torch.randn(tokens, experts, device="cuda", generator=g) * 1.5
    # a skew between experts, as the bias is there to even out
    logits += torch.randn(experts, device="cuda", generator=g) * 0.5
    if case["masked"]:      # experts out of service, and rows of padding
        at = torch.arange(experts, device="cuda")
        logits[:, at % 7 == 3] = -math.inf
        logits[torch.rand(tokens, device="cuda", generator=g) < 0.1] = -math.inf
    s["logits"] = logits.to(DTYPES[case["dtype"]])
    s["bias"] = None
    if case["bias"]:        # many steps of 0.001 up or down
        s["bias"] = torch.randint(-60, 61, (experts,), device="cuda", generator=g).float() * 1e-3
    if case["op"] == "route":
        s["weights"] = torch.empty(tokens, k, device="cuda")
        s["chosen"] = torch.empty(tokens, k, device="cuda", dtype=torch.int32)
    else:
        s["chosen"] = _choose(s)
        s["dweights"] = torch.randn(tokens, k, device="cuda", generator=g)
        s["dlogits"] = torch.empty_like(s["logits"])


def _slots(case, g):
    """tokens x k distinct experts a token, by Zipf weights, in a random order of experts."""
    experts = case["experts"]
    share = -case["zipf"] * torch.log(torch.arange(1.0, experts + 1, device="cuda"))
    share = share[torch.randperm(experts, device="cuda", generator=g)]
    noise = torch.rand(case["tokens"], experts, device="cuda", generator=g).clamp_min(1e-20)
    keys = share - torch.log(-torch.log(noise.clamp_max(1 - 1e-7)))
    return torch.topk(keys, case["k"], dim=1).indices.int()


def _capacity(case):
    """Slots an expert takes: a quarter more than an even share; 0: all, packed."""
    return math.ceil(1.25 * case["tokens"] * case["k"] / case["experts"]) if case["capacity"] else 0


def _order_rows(case):
    return case["experts"] * _capacity(case) if case["capacity"] else case["tokens"] * case["k"]


def _randn(g, rows, cols, dtype, scale=1.0):
    return (torch.randn(rows, cols, device="cuda", generator=g) * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]
    s = dict(case)
    if op in ("route", "route_backward"):
        _router_inputs(case, s, g)
    elif op == "dispatch":
        tokens, hidden, rows = case["tokens"], case["hidden"], _order_rows(case)
        s.update(capacity=_capacity(case), total_rows=rows, slots=_slots(case, g))
        s["x"] = _randn(g, tokens, hidden, dt, 40.0 if case["dtype"] == "e4m3" else 1.0)
        s["scales"] = s["out_scales"] = None
        if case["dtype"] == "e4m3":
            s["scales"] = 0.5 + torch.rand(tokens, device="cuda", generator=g)
            s["out_scales"] = torch.zeros(rows, device="cuda")
        s["place"] = torch.empty(tokens, case["k"], device="cuda", dtype=torch.int32)
        s["begin"] = torch.empty(case["experts"], device="cuda", dtype=torch.int64)
        s["count"] = torch.empty(case["experts"], device="cuda", dtype=torch.int64)
        s["out"] = torch.zeros(rows, hidden, device="cuda").to(dt)
    elif op in ("combine", "combine_backward"):
        tokens, hidden, k, rows = case["tokens"], case["hidden"], case["k"], _order_rows(case)
        place = _place(_slots(case, g), case["experts"], _capacity(case))[0]
        s.update(place=place, total_rows=rows, rows=_randn(g, rows, hidden, dt))
        s["weights"] = torch.rand(tokens, k, device="cuda", generator=g) / k
        if op == "combine":
            s["shared"] = _randn(g, tokens, hidden, dt) if case["shared"] else None
            s["y"] = torch.empty(tokens, hidden, device="cuda", dtype=dt)
        else:
            s["dy"] = _randn(g, tokens, hidden, dt)
            s["drows"] = torch.zeros(rows, hidden, device="cuda", dtype=dt)
            s["dweights"] = torch.empty(tokens, k, device="cuda")
    else:
        rows, hidden = case["rows"], case["hidden"]

        def vector():
            return (1 + 0.1 * torch.randn(hidden, device="cuda", generator=g)).to(dt)

        s.update(x=_randn(g, rows, hidden, dt), weight=vector(), post_weight=None, gate_values=None)
        if case["post"]:
            s["post_weight"] = vector()
        if case["gate"] == "columns":
            s["gate_values"] = vector()
        elif case["gate"] == "rows":
            s["gate_values"] = _randn(g, rows, hidden, dt)
        if op == "block_norm":
            s["residual"] = _randn(g, rows, hidden, dt, 2.0)
            s["total"] = torch.empty_like(s["x"])
            s["y"] = torch.empty(rows, hidden, device="cuda", dtype=DTYPES[case["out"]])
            s["scales"] = torch.empty(rows, device="cuda") if case["out"] == "e4m3" else None
        else:
            s.update(dy=_randn(g, rows, hidden, dt), dtotal=_randn(g, rows, hidden, dt),
                     total=_randn(g, rows, hidden, dt, 2.0))
            s["dx"], s["dresidual"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
            s["dweight"] = torch.empty(hidden, device="cuda")
            s["dpost_weight"] = torch.empty(hidden, device="cuda") if case["post"] else None
            s["dgate"] = None
            if case["gate"] == "columns":
                s["dgate"] = torch.empty(hidden, device="cuda")
            elif case["gate"] == "rows":
                s["dgate"] = torch.empty_like(s["x"])
    return s


# ------------------------------------------------------------- plain form ---

def _score(logits, kind):
    """Scores of every expert in the type of ``logits``; a row without an expert has zeros."""
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    top = logits.amax(1, keepdim=True).clamp_min(torch.finfo(logits.dtype).min)
    e = torch.exp(logits - top)
    return e / e.sum(1, keepdim=True).clamp_min(SCALE_MIN)


def _choose(s):
    """Chosen experts, descending, ties to the lowest index, -1 where there is none.
    In 64 bits: values that 32 would round together lie next to a border."""
    logits = s["logits"].double()
    tokens, experts = logits.shape
    choice = _score(logits, s["scores"])
    if s["bias"] is not None:
        choice = choice + s["bias"].double()
    choice = torch.where(logits == -math.inf, -math.inf, choice)
    if s["groups"] > 1:
        by_group = choice.view(tokens, s["groups"], -1)
        best = by_group.sort(dim=2, descending=True).values[:, :, :s["group_top"]]
        total = torch.where(best == -math.inf, 0.0, best).sum(2)
        total = torch.where(best[:, :, 0] == -math.inf, -math.inf, total)
        kept = total.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros_like(total, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(keep[:, :, None], by_group, -math.inf).view(tokens, experts)
    top = choice.sort(dim=1, descending=True, stable=True)
    chosen = torch.where(top.values == -math.inf, -1, top.indices)
    return chosen[:, :s["k"]].int()


def _plain_route(s):
    chosen = _choose(s)
    score = _score(s["logits"].float(), s["scores"])
    w = torch.where(chosen < 0, 0.0, score.gather(1, chosen.clamp_min(0).long()))
    if s["renormalise"]:
        w = w / w.sum(1, keepdim=True).clamp_min(SCALE_MIN)
    return {"weights": w * s["scale"], "experts": chosen}


def _plain_route_backward(s):
    score = _score(s["logits"].float(), s["scores"])
    real, at = s["chosen"] >= 0, s["chosen"].clamp_min(0).long()
    g = torch.where(real, s["dweights"] * s["scale"], 0.0)
    if s["renormalise"]:
        w = torch.where(real, score.gather(1, at), 0.0)
        total = w.sum(1, keepdim=True).clamp_min(SCALE_MIN)
        g = torch.where(real, (g - (g * w).sum(1, keepdim=True) / total) / total, 0.0)
    ds = torch.zeros_like(score).scatter_add_(1, at, g)
    if s["scores"] == "softmax":
        dl = score * (ds - (ds * score).sum(1, keepdim=True))
    else:
        dl = ds * score * (1 - score)
    return {"dlogits": dl.to(s["logits"].dtype)}


def _place(slots, experts, capacity):
    """Each slot's row in expert order (-1 past the capacity), first rows and counts."""
    flat = slots.reshape(-1).long()
    order = flat.sort(stable=True).indices
    count = (flat[:, None] == torch.arange(experts, device="cuda")).sum(0)
    first = count.cumsum(0) - count
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(flat.numel(), device="cuda") - first[flat[order]]
    if capacity:
        begin = torch.arange(experts, device="cuda") * capacity
        place = torch.where(rank < capacity, begin[flat] + rank, -1)
        return place.int().view_as(slots), begin, count.clamp_max(capacity)
    return (first[flat] + rank).int().view_as(slots), first, count


def _plain_dispatch(s):
    place, begin, count = _place(s["slots"], s["experts"], s["capacity"])
    rows = s["total_rows"]
    at = torch.where(place < 0, rows, place).long().view(-1)
    out = torch.zeros(rows + 1, s["hidden"], device="cuda")
    out[at] = s["x"].float().repeat_interleave(s["k"], 0)
    got = {"place": place, "begin": begin, "count": count, "out": out[:rows].to(s["x"].dtype)}
    if s["scales"] is not None:
        scales = torch.zeros(rows + 1, device="cuda")
        scales[at] = s["scales"].repeat_interleave(s["k"], 0)
        got["scales"] = scales[:rows]
    return got


def _plain_combine(s):
    real, at = s["place"] >= 0, s["place"].clamp_min(0).long()
    w = torch.where(real, s["weights"], 0.0)
    y = (s["rows"][at].float() * w[:, :, None]).sum(1)
    if s["shared"] is not None:
        y = y + s["shared"].float()
    return {"y": y.to(s["rows"].dtype)}


def _plain_combine_backward(s):
    real, at = s["place"] >= 0, s["place"].clamp_min(0).long()
    dy = s["dy"].float()[:, None, :]
    dw = torch.where(real, (s["rows"][at].float() * dy).sum(2), 0.0)
    rows = s["total_rows"]
    drows = torch.zeros(rows + 1, s["hidden"], device="cuda", dtype=s["rows"].dtype)
    drows[torch.where(real, at, rows)] = (s["weights"][:, :, None] * dy).to(drows.dtype)
    return {"drows": drows[:rows], "dweights": dw}


def _plain_block_norm(s):
    u = s["x"].float()
    if s["post_weight"] is not None:
        u = u * torch.rsqrt((u * u).mean(1, keepdim=True) + EPS) * s["post_weight"].float()
    if s["gate_values"] is not None:
        u = u * s["gate_values"].float()
    t = s["residual_scale"] * s["residual"].float() + s["block_scale"] * u
    y = t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * s["weight"].float()
    got = {"total": t.to(s["x"].dtype)}
    if s["out"] == "e4m3":
        scale = (y.abs().amax(1) / E4M3_MAX).clamp_min(SCALE_MIN)
        got["y"] = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        got["scales"] = scale
    else:
        got["y"] = y.to(DTYPES[s["out"]])
    return got


def _plain_block_norm_backward(s):
    x, t, dy = s["x"].float(), s["total"].float(), s["dy"].float()
    r = torch.rsqrt((t * t).mean(1, keepdim=True) + EPS)
    g = dy * s["weight"].float()
    dt = r * (g - t * (r * r * (g * t).mean(1, keepdim=True))) + s["dtotal"].float()
    got = {"dresidual": (s["residual_scale"] * dt).to(s["x"].dtype), "dweight": (dy * t * r).sum(0)}
    dv = s["block_scale"] * dt                     # of gate * u
    unit, q, post = x, None, None
    if s["post_weight"] is not None:
        q = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        unit, post = x * q, s["post_weight"].float()
    if s["gate_values"] is not None:
        dgate = dv * (unit if post is None else unit * post)
        got["dgate"] = dgate.sum(0) if s["gate"] == "columns" else dgate.to(s["x"].dtype)
        dv = dv * s["gate_values"].float()
    if post is not None:
        got["dpost_weight"] = (dv * unit).sum(0)
        dv = dv * post
        dv = q * (dv - unit * (dv * unit).mean(1, keepdim=True))
    got["dx"] = dv.to(s["x"].dtype)
    return got


# ---------------------------------------------------------- library calls ---

_context = []


def _library():
    """The package and one context on the current stream, as a program keeps them."""
    if not _context:
        import collective_datapath_atom_gb300 as purlin

        _context.append((purlin, purlin.purlin_init(8, torch.cuda.current_stream())))
    return _context[0]


def _code(purlin, dtype):
    return {"f32": purlin.PURLIN_F32, "bf16": purlin.PURLIN_BF16, "e4m3": purlin.PURLIN_E4M3}[dtype]


def _router(purlin, s):
    return purlin.purlin_router(
        experts=s["experts"], top_k=s["k"],
        scores=purlin.PURLIN_SOFTMAX if s["scores"] == "softmax" else purlin.PURLIN_SIGMOID,
        groups=s["groups"], top_groups=s["top_groups"], group_top=s["group_top"],
        renormalise=int(s["renormalise"]), scale=s["scale"])


def _own_route(s):
    purlin, ctx = _library()
    purlin.purlin_route(ctx, s["logits"], s["weights"], s["chosen"], s["tokens"],
                        _router(purlin, s), _code(purlin, s["dtype"]), bias=s["bias"])
    return {"weights": s["weights"], "experts": s["chosen"]}


def _own_route_backward(s):
    purlin, ctx = _library()
    purlin.purlin_route_backward(ctx, s["dweights"], s["logits"], s["chosen"], s["dlogits"],
                                 s["tokens"], _router(purlin, s), _code(purlin, s["dtype"]))
    return {"dlogits": s["dlogits"]}


def _own_dispatch(s):
    purlin, ctx = _library()
    purlin.purlin_expert_order(ctx, s["slots"], s["place"], s["begin"], s["count"],
                               s["tokens"] * s["k"], s["experts"], capacity=s["capacity"])
    purlin.purlin_dispatch_rows(ctx, s["x"], s["place"], s["out"], s["tokens"], s["k"],
                                s["hidden"], s["total_rows"], _code(purlin, s["dtype"]),
                                scales=s["scales"], out_scales=s["out_scales"])
    got = {"place": s["place"], "begin": s["begin"], "count": s["count"], "out": s["out"]}
    if s["scales"] is not None:
        got["scales"] = s["out_scales"]
    return got


def _own_combine(s):
    purlin, ctx = _library()
    purlin.purlin_combine_rows(ctx, s["rows"], s["place"], s["y"], s["tokens"], s["k"],
                               s["hidden"], s["total_rows"], _code(purlin, s["dtype"]),
                               weights=s["weights"], shared=s["shared"])
    return {"y": s["y"]}


def _own_combine_backward(s):
    purlin, ctx = _library()
    purlin.purlin_combine_rows_backward(ctx, s["dy"], s["rows"], s["place"], s["weights"],
                                        s["drows"], s["dweights"], s["tokens"], s["k"],
                                        s["hidden"], s["total_rows"], _code(purlin, s["dtype"]))
    return {"drows": s["drows"], "dweights": s["dweights"]}


def _gate_layout(purlin, s):
    return purlin.PURLIN_GATE_ROWS if s["gate"] == "rows" else purlin.PURLIN_GATE_COLUMNS


def _own_block_norm(s):
    purlin, ctx = _library()
    purlin.purlin_block_norm(ctx, s["x"], s["weight"], s["y"], s["rows"], s["hidden"], EPS,
                             _code(purlin, s["dtype"]), _code(purlin, s["out"]),
                             residual=s["residual"], post_weight=s["post_weight"],
                             gate=s["gate_values"], gate_layout=_gate_layout(purlin, s),
                             residual_scale=s["residual_scale"], block_scale=s["block_scale"],
                             total=s["total"], scales=s["scales"])
    got = {"total": s["total"], "y": s["y"]}
    if s["scales"] is not None:
        got["scales"] = s["scales"]
    return got


def _own_block_norm_backward(s):
    purlin, ctx = _library()
    purlin.purlin_block_norm_backward(ctx, s["dy"], s["x"], s["total"], s["weight"], s["dx"],
                                      s["dweight"], s["rows"], s["hidden"], EPS,
                                      _code(purlin, s["dtype"]), dtotal=s["dtotal"],
                                      post_weight=s["post_weight"], gate=s["gate_values"],
                                      gate_layout=_gate_layout(purlin, s),
                                      residual_scale=s["residual_scale"],
                                      block_scale=s["block_scale"], dresidual=s["dresidual"],
                                      dpost_weight=s["dpost_weight"], dgate=s["dgate"])
    got = {"dresidual": s["dresidual"], "dweight": s["dweight"], "dx": s["dx"]}
    if s["dgate"] is not None:
        got["dgate"] = s["dgate"]
    if s["dpost_weight"] is not None:
        got["dpost_weight"] = s["dpost_weight"]
    return got


_PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward,
          "dispatch": _plain_dispatch, "combine": _plain_combine,
          "combine_backward": _plain_combine_backward, "block_norm": _plain_block_norm,
          "block_norm_backward": _plain_block_norm_backward}
_OWN = {"route": _own_route, "route_backward": _own_route_backward, "dispatch": _own_dispatch,
        "combine": _own_combine, "combine_backward": _own_combine_backward,
        "block_norm": _own_block_norm, "block_norm_backward": _own_block_norm_backward}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ------------------------------------------------------------ work, exact ---

def work(case):
    e, op = SIZES[case["dtype"]], case["op"]
    if op in ("route", "route_backward"):
        cells, slots = case["tokens"] * case["experts"], case["tokens"] * case["k"]
        if op == "route":
            moved = cells * e + 8 * slots + (4 * case["experts"] if case["bias"] else 0)
            return {"bytes": moved, "flops": 4 * cells}
        # the chosen experts' logits alone where no other score counts
        all_scores = case["scores"] == "softmax" and not case["renormalise"]
        moved = cells * e + (cells if all_scores else slots) * e + 8 * slots
        return {"bytes": moved, "flops": 6 * cells if all_scores else 8 * slots}
    if op in ("dispatch", "combine", "combine_backward"):
        cells, slots = case["tokens"] * case["hidden"], case["tokens"] * case["k"]
        rows = min(slots, _order_rows(case)) * case["hidden"]
        if op == "dispatch":
            moved = 8 * slots + 16 * case["experts"] + e * (cells + rows)
            moved += 4 * (case["tokens"] + slots) if case["dtype"] == "e4m3" else 0
            return {"bytes": moved, "flops": 0}
        if op == "combine":
            moved = 8 * slots + e * (rows + cells * (2 if case["shared"] else 1))
            return {"bytes": moved, "flops": 2 * rows}
        return {"bytes": 12 * slots + e * (cells + 2 * rows), "flops": 3 * rows}
    cells, hidden = case["rows"] * case["hidden"], case["hidden"]
    vectors = 1 + case["post"] + (case["gate"] == "columns")
    if op == "block_norm":
        moved = cells * (3 * e + SIZES[case["out"]]) + vectors * hidden * e
        moved += cells * e if case["gate"] == "rows" else 0
        moved += 4 * case["rows"] if case["out"] == "e4m3" else 0
        return {"bytes": moved, "flops": 12 * cells}
    moved = cells * 6 * e + vectors * hidden * (e + 4)
    moved += 2 * cells * e if case["gate"] == "rows" else 0
    return {"bytes": moved, "flops": 26 * cells}


def _exact_chosen(case, s):
    """The router's choice row by row in numpy: (chosen, scores, chosen scores) in 64 bits."""
    import numpy as np

    logits = s["logits"].double().cpu().numpy()
    out = np.isneginf(logits)
    with np.errstate(invalid="ignore", over="ignore"):
        if case["scores"] == "sigmoid":
            score = np.where(logits >= 0, 1 / (1 + np.exp(-np.abs(logits))),
                             np.exp(-np.abs(logits)) / (1 + np.exp(-np.abs(logits))))
        else:
            high = logits.max(1, keepdims=True)
            score = np.exp(logits - np.where(np.isneginf(high), 0, high))
            score = score / np.maximum(score.sum(1, keepdims=True), SCALE_MIN)
    score[out] = 0
    key = score + (0 if s["bias"] is None else s["bias"].double().cpu().numpy())
    key[out] = -np.inf
    if case["groups"] > 1:
        each = case["experts"] // case["groups"]
        parts = -np.sort(-key.reshape(-1, case["groups"], each), axis=2)[:, :, :case["group_top"]]
        value = np.where(np.isneginf(parts), 0, parts).sum(2)
        value[np.isneginf(parts[:, :, 0])] = -np.inf
        rank = np.argsort(np.argsort(-value, axis=1, kind="stable"), axis=1)
        key[np.repeat(rank >= case["top_groups"], each, axis=1)] = -np.inf
    chosen = np.argsort(-key, axis=1, kind="stable")[:, :case["k"]]
    picked = np.take_along_axis(score, chosen, 1)
    none = np.isneginf(np.take_along_axis(key, chosen, 1))
    chosen[none], picked[none] = -1, 0
    return chosen, score, picked


def exact(case, seed):
    """The definitions in 64 bits, before any rounding of the outputs.  An e4m3
    output's values are y / scale; copies of rows have no error to measure."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_backward"):
        import numpy as np

        chosen, score, picked = _exact_chosen(case, s)
        total = np.maximum(picked.sum(1, keepdims=True), SCALE_MIN)
        if op == "route":
            w = picked / total if case["renormalise"] else picked
            return {"weights": torch.from_numpy(w * case["scale"]),
                    "experts": torch.from_numpy(chosen.astype(np.int32))}
        real = chosen >= 0
        g = np.where(real, s["dweights"].double().cpu().numpy() * case["scale"], 0)
        row, col = np.nonzero(real)
        at = chosen[row, col]
        dl = np.zeros_like(score)
        if case["renormalise"]:
            p = picked / total
            v = p * (g - (g * p).sum(1, keepdims=True))
            dl[row, at] = v[row, col] * (1 if case["scores"] == "softmax" else 1 - picked[row, col])
        elif case["scores"] == "softmax":
            dl = -score * (g * picked).sum(1, keepdims=True)
            dl[row, at] += (g * picked)[row, col]
        else:
            dl[row, at] = (g * picked * (1 - picked))[row, col]
        return {"dlogits": torch.from_numpy(dl)}
    if op == "dispatch":
        return None
    if op in ("combine", "combine_backward"):
        place, w = s["place"].long(), s["weights"].double()
        rows, tokens, hidden = s["total_rows"], case["tokens"], case["hidden"]
        if op == "combine":
            y = torch.zeros(tokens, hidden, device="cuda", dtype=torch.float64)
            if s["shared"] is not None:
                y += s["shared"].double()
            for j in range(case["k"]):
                t = torch.nonzero(place[:, j] >= 0).view(-1)
                y[t] += s["rows"][place[t, j]].double() * w[t, j].unsqueeze(1)
            return {"y": y}
        dy = s["dy"].double()
        drows = torch.zeros(rows, hidden, device="cuda", dtype=torch.float64)
        dw = torch.zeros(tokens, case["k"], device="cuda", dtype=torch.float64)
        for j in range(case["k"]):
            t = torch.nonzero(place[:, j] >= 0).view(-1)
            drows[place[t, j]] = dy[t] * w[t, j].unsqueeze(1)
            dw[t, j] = torch.einsum("th,th->t", dy[t], s["rows"][place[t, j]].double())
        return {"drows": drows, "dweights": dw}
    hidden = case["hidden"]
    a, b = case["residual_scale"], case["block_scale"]

    def root(v):
        return (v.pow(2).sum(1, keepdim=True) / hidden + EPS).sqrt()

    x, w = s["x"].double(), s["weight"].double()
    gate = 1.0 if s["gate_values"] is None else s["gate_values"].double()
    post = 1.0 if s["post_weight"] is None else s["post_weight"].double()
    unit = x / root(x) if case["post"] else x
    if op == "block_norm":
        t = a * s["residual"].double() + b * gate * (unit * post)
        y = t / root(t) * w
        got = {"total": t}
        if case["out"] == "e4m3":
            got["scales"] = torch.clamp(y.abs().max(1).values / E4M3_MAX, min=SCALE_MIN)
            y = y / got["scales"].unsqueeze(1)
        got["y"] = y
        return got
    t, dy = s["total"].double(), s["dy"].double()
    n = t / root(t)
    dt = (dy * w - n * (dy * w * n).sum(1, keepdim=True) / hidden) / root(t) + s["dtotal"].double()
    got = {"dresidual": a * dt, "dweight": (dy * n).sum(0)}
    if case["gate"] == "columns":
        got["dgate"] = (b * dt * unit * post).sum(0)
    elif case["gate"] == "rows":
        got["dgate"] = b * dt * unit * post
    dv = b * dt * gate
    if case["post"]:
        got["dpost_weight"] = (dv * unit).sum(0)
        dv = dv * post
        dv = (dv - unit * (dv * unit).sum(1, keepdim=True) / hidden) / root(x)
    got["dx"] = dv
    return got
