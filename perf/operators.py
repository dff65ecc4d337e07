"""Cases of the layer operators that stand beside the collectives: the RMS norm
with the residual's addition (bf16, f32 or e4m3 output) and its backward pass,
and the matrix products grouped by expert (bf16 or e4m3) and their backward
pass.  The first consumes an AllReduce's output, the second what an AllToAllV
dispatch delivers.

``run`` computes a case in plain torch operations, or with the library's
kernels where ``own`` is true.
"""
import torch

own = False

E4M3_MAX = 448.0          # largest finite e4m3 value
SCALE_MIN = 2.0 ** -126   # smallest row scale: its reciprocal is finite
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ------------------------------------------------------------------ cases ---

def _norm(name, rows, hidden, dtype, out, residual):
    return {"name": name, "op": "norm", "rows": rows, "hidden": hidden, "dtype": dtype,
            "out": out, "residual": residual}


def _norm_backward(name, rows, hidden, dtype, residual):
    return {"name": name, "op": "norm_backward", "rows": rows, "hidden": hidden, "dtype": dtype,
            "residual": residual}


def _experts(name, rows, groups, k, n, dtype, zipf, capacity, op="experts"):
    return {"name": name, "op": op, "rows": rows, "groups": groups, "k": k, "n": n,
            "dtype": dtype, "zipf": zipf, "capacity": capacity}


def listed():
    return [
        # one new token after the AllReduce of a tensor-parallel layer
        _norm("norm 1x4096 bf16", 1, 4096, "bf16", "bf16", True),
        # a decode batch, quantised for an 8-bit dispatch to the experts
        _norm("norm 128x7168 bf16 to e4m3", 128, 7168, "bf16", "e4m3", True),
        # a prefill's 16384 tokens, quantised for the dispatch
        _norm("norm 16384x7168 bf16 to e4m3", 16384, 7168, "bf16", "e4m3", True),
        # a hidden size whose rows start on no 16-byte boundary, without a residual stream
        _norm("norm 1000x4099 f32", 1000, 4099, "f32", "f32", False),
        # backward pass of the largest AllReduce size, with the residual stream's gradient
        _norm_backward("norm backward 32768x4096 bf16", 32768, 4096, "bf16", True),
        # a small odd backward pass: the weight gradient's join is most of it
        _norm_backward("norm backward 509x1021 f32", 509, 1021, "f32", False),
        # decode: 8 tokens' rows on 8 experts, some of them empty; the weights' bytes count
        _experts("experts 8 rows bf16", 8, 8, 7168, 2048, "bf16", 1.2, False),
        # decode batch on many small experts, 8-bit, in capacity-padded dispatch buffers
        _experts("experts 128 rows on 64 e4m3", 128, 64, 4096, 1024, "e4m3", 0.6, True),
        # prefill dispatch of 16384 tokens x 7168 with Zipf destinations
        _experts("experts 16384 rows bf16", 16384, 8, 7168, 2048, "bf16", 1.2, False),
        # the same dispatch in 8 bits, gate and up projections in one product
        _experts("experts 16384 rows e4m3", 16384, 8, 7168, 4096, "e4m3", 1.2, False),
        # training step of the prefill product: data and weight gradients
        _experts("experts backward 16384 rows", 16384, 8, 7168, 2048, "bf16", 1.2, False,
                 "experts_backward"),
        # odd sizes in capacity-padded buffers: ragged tiles on every axis
        _experts("experts backward 1003 rows odd", 1003, 5, 1001, 517, "bf16", 0.6, True,
                 "experts_backward"),
    ]


def _log(rng, lo, hi):
    import math
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v))
    return v + 1 if v == 3072 else v


def _size(rng, lo, hi):
    """Log-uniform; two in three rounded to a multiple of 64, as model sizes are."""
    v = _log(rng, lo, hi)
    if rng.random() < 2 / 3:
        v = max(64, (v + 32) // 64 * 64)
    return v + 8 if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "experts", "experts", "experts_backward"])
    if op in ("norm", "norm_backward"):
        case = {"op": op, "rows": _log(rng, 1, 32768), "hidden": _size(rng, 64, 16384),
                "dtype": rng.choice(["f32", "bf16", "bf16"]), "residual": rng.random() < 0.7}
        if op == "norm":
            case["out"] = rng.choice([case["dtype"], "e4m3"])
        # at most the elements of the largest listed case
        case["rows"] = max(1, min(case["rows"], (1 << 26) // case["hidden"]))
        return case
    case = {"op": op, "rows": _log(rng, 1, 16384), "groups": _log(rng, 1, 64),
            "k": _size(rng, 64, 7168), "n": _size(rng, 64, 4096),
            "dtype": "bf16" if op == "experts_backward" else rng.choice(["bf16", "e4m3"]),
            "zipf": rng.choice([0.0, 0.6, 1.2]), "capacity": rng.random() < 0.4}
    # at most the weights and the padded rows of the largest listed cases
    while case["groups"] * case["n"] * case["k"] > 8 * 4096 * 7168:
        case["groups"] = (case["groups"] + 1) // 2
    most = 8 * 7030 * 7168 * (2048 if op == "experts_backward" else 4096)
    while case["rows"] > 1 and \
            case["groups"] * max(_counts(case)) * case["n"] * case["k"] > most:
        case["rows"] = (case["rows"] + 1) // 2
    return case


def _counts(case):
    """Rows of each group by falling Zipf weights, largest remainders first."""
    rows, groups = case["rows"], case["groups"]
    p = [(g + 1) ** -case["zipf"] for g in range(groups)]
    exact_share = [rows * v / sum(p) for v in p]
    counts = [int(v) for v in exact_share]
    order = sorted(range(groups), key=lambda g: (counts[g] - exact_share[g], g))
    for g in order[:rows - sum(counts)]:
        counts[g] += 1
    return counts


# ----------------------------------------------------------------- inputs ---

def _pitch(cols, dtype):
    """Row pitch in elements: rows of the products start on 16-byte boundaries."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return (cols + per - 1) // per * per


def _rows_of(g, rows, cols, dtype, scale=1.0):
    """A rows x cols view of a pitched buffer of N(0, scale^2) values."""
    t = torch.zeros(rows, _pitch(cols, dtype), device="cuda", dtype=dtype)
    t[:, :cols] = (torch.randn(rows, cols, device="cuda", generator=g) * scale).to(dtype)
    return t[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("norm", "norm_backward"):
        rows, hidden = case["rows"], case["hidden"]

        def mat(scale=1.0):
            return (torch.randn(rows, hidden, device="cuda", generator=g) * scale).to(dt)

        s = dict(case, x=mat(), y=None, scales=None, total=None)
        s["weight"] = (1 + 0.1 * torch.randn(hidden, device="cuda", generator=g)).to(dt)
        s["other"] = mat(2.0) if case["residual"] else None
        if case["op"] == "norm":
            s["y"] = torch.empty(rows, hidden, device="cuda", dtype=DTYPES[case["out"]])
            if case["out"] == "e4m3":
                s["scales"] = torch.empty(rows, device="cuda")
            if case["residual"]:
                s["total"] = torch.empty_like(s["x"])
        else:
            s["dy"] = mat()
            s["dx"] = torch.empty_like(s["x"])
            s["dweight"] = torch.empty(hidden, device="cuda")
        return s
    n, k, groups = case["n"], case["k"], case["groups"]
    counts = _counts(case)
    perm = torch.randperm(groups, generator=torch.Generator().manual_seed(seed)).tolist()
    counts = [counts[p] for p in perm]
    most = max(counts)
    if case["capacity"]:                      # each expert's rows at a fixed place
        begin, rows = [i * most for i in range(groups)], groups * most
    else:                                     # packed, in expert order
        begin, rows = [sum(counts[:i]) for i in range(groups)], case["rows"]
    s = dict(case, most=most, total_rows=rows,
             begin=torch.tensor(begin, device="cuda", dtype=torch.int64),
             count=torch.tensor(counts, device="cuda", dtype=torch.int64))
    s["x"] = _rows_of(g, rows, k, dt)
    pitch = _pitch(k, dt)
    w = torch.zeros(groups, n, pitch, device="cuda", dtype=dt)
    w[:, :, :k] = (torch.randn(groups, n, k, device="cuda", generator=g) * k ** -0.5
                   * (16.0 if case["dtype"] == "e4m3" else 1.0)).to(dt)
    s["w"] = w[:, :, :k]
    s["x_scales"] = s["w_scales"] = None
    if case["dtype"] == "e4m3":
        s["x_scales"] = 0.5 + torch.rand(rows, device="cuda", generator=g)
        s["w_scales"] = (0.5 + torch.rand(groups, n, device="cuda", generator=g)) / 16
    if case["op"] == "experts":
        s["y"] = torch.zeros(rows, n, device="cuda", dtype=torch.bfloat16)
    else:
        s["dy"] = _rows_of(g, rows, n, dt)
        s["dx"] = torch.zeros(rows, pitch, device="cuda", dtype=dt)[:, :k]
        s["dw"] = torch.empty(groups, n, pitch, device="cuda", dtype=dt)[:, :, :k]
    return s


# ------------------------------------------------------------- plain form ---

def _plain_norm(s):
    t = s["x"].float()
    if s["other"] is not None:
        t = t + s["other"].float()
    r = torch.rsqrt((t * t).mean(1, keepdim=True) + EPS)
    y = t * r * s["weight"].float()
    out = {}
    if s["out"] == "e4m3":
        scale = (y.abs().amax(1) / E4M3_MAX).clamp_min(SCALE_MIN)
        out["y"] = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        out["scales"] = scale
    else:
        out["y"] = y.to(DTYPES[s["out"]])
    if s["other"] is not None:
        out["total"] = t.to(s["x"].dtype)
    return out


def _plain_norm_backward(s):
    t, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((t * t).mean(1, keepdim=True) + EPS)
    g = dy * s["weight"].float()
    dx = r * (g - t * (r * r * (g * t).mean(1, keepdim=True)))
    if s["other"] is not None:
        dx = dx + s["other"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * t * r).sum(0)}


def _padded(s):
    """Rows of every group in a groups x most table: their indices, and which are real."""
    at = torch.arange(s["most"], device="cuda")
    real = at[None, :] < s["count"][:, None]
    index = torch.where(real, s["begin"][:, None] + at[None, :], 0)
    return index, real


def _take(t, index, real):
    return torch.where(real[:, :, None], t[index].float(), 0.0)


def _put(values, index, real, rows, dtype):
    """The table's real rows back in their places; other rows are zero."""
    out = torch.zeros(rows + 1, values.shape[2], device="cuda", dtype=dtype)
    out[torch.where(real, index, rows)] = values.to(dtype)
    return out[:rows]


def _plain_experts(s):
    index, real = _padded(s)
    x, w = s["x"].float(), s["w"].float()
    y = torch.bmm(_take(x, index, real), w.transpose(1, 2))
    if s["x_scales"] is not None:
        y = y * s["x_scales"][index][:, :, None] * s["w_scales"][:, None, :]
    return {"y": _put(y, index, real, s["total_rows"], torch.bfloat16)}


def _plain_experts_backward(s):
    index, real = _padded(s)
    x, dy, w = _take(s["x"], index, real), _take(s["dy"], index, real), s["w"].float()
    dx = torch.bmm(dy, w)
    dw = torch.bmm(dy.transpose(1, 2), x)
    return {"dx": _put(dx, index, real, s["total_rows"], s["x"].dtype),
            "dw": dw.to(s["w"].dtype)}


# ---------------------------------------------------------- library calls ---

_context = []


def _library():
    """The package and one context on the current stream, as a program keeps them."""
    if not _context:
        import collective_datapath_atom_gb300 as purlin

        _context.append((purlin, purlin.purlin_init(8, torch.cuda.current_stream())))
    return _context[0]


def _own_norm(s):
    purlin, ctx = _library()
    dt = purlin.PURLIN_F32 if s["dtype"] == "f32" else purlin.PURLIN_BF16
    quantised = s["out"] == "e4m3"
    purlin.purlin_rms_norm(ctx, s["x"], s["weight"], s["y"], s["rows"], s["hidden"], EPS, dt,
                           purlin.PURLIN_E4M3 if quantised else dt, residual=s["other"],
                           total=s["total"], scales=s["scales"])
    out = {"y": s["y"]}
    if quantised:
        out["scales"] = s["scales"]
    if s["total"] is not None:
        out["total"] = s["total"]
    return out


def _own_norm_backward(s):
    purlin, ctx = _library()
    dt = purlin.PURLIN_F32 if s["dtype"] == "f32" else purlin.PURLIN_BF16
    purlin.purlin_rms_norm_backward(ctx, s["dy"], s["x"], s["weight"], s["dx"], s["dweight"],
                                    s["rows"], s["hidden"], EPS, dt, dtotal=s["other"])
    return {"dx": s["dx"], "dweight": s["dweight"]}


def _own_experts(s):
    purlin, ctx = _library()
    purlin.purlin_grouped_matmul(
        ctx, s["x"], s["w"], s["y"], s["begin"], s["count"], s["groups"], s["total_rows"],
        s["n"], s["k"], purlin.PURLIN_BF16 if s["dtype"] == "bf16" else purlin.PURLIN_E4M3,
        x_scales=s["x_scales"], w_scales=s["w_scales"], ldx=s["x"].stride(0),
        ldw=s["w"].stride(1))
    return {"y": s["y"]}


def _own_experts_backward(s):
    purlin, ctx = _library()
    rows, n, k = s["total_rows"], s["n"], s["k"]
    ldx, lddy = s["x"].stride(0), s["dy"].stride(0)
    purlin.purlin_grouped_matmul(
        ctx, s["dy"], s["w"], s["dx"], s["begin"], s["count"], s["groups"], rows, k, n,
        purlin.PURLIN_BF16, layout=purlin.PURLIN_WEIGHTS_KN, ldx=lddy, ldw=s["w"].stride(1),
        ldy=s["dx"].stride(0))
    purlin.purlin_grouped_matmul_weight_grad(
        ctx, s["dy"], s["x"], s["dw"], s["begin"], s["count"], s["groups"], rows, n, k,
        purlin.PURLIN_BF16, lddy=lddy, ldx=ldx, lddw=s["dw"].stride(1))
    return {"dx": s["dx"], "dw": s["dw"]}


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward,
          "experts": _plain_experts, "experts_backward": _plain_experts_backward}
_OWN = {"norm": _own_norm, "norm_backward": _own_norm_backward,
        "experts": _own_experts, "experts_backward": _own_experts_backward}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ------------------------------------------------------------ work, exact ---

def work(case):
    size = {"f32": 4, "bf16": 2, "e4m3": 1}
    e = size[case["dtype"]]
    if case["op"] in ("norm", "norm_backward"):
        cells = case["rows"] * case["hidden"]
        if case["op"] == "norm":
            moved = cells * (e + size[case["out"]]) + e * case["hidden"]
            moved += 2 * cells * e if case["residual"] else 0
            moved += 4 * case["rows"] if case["out"] == "e4m3" else 0
            return {"bytes": moved, "flops": 6 * cells}
        moved = cells * e * (4 if case["residual"] else 3) + (4 + e) * case["hidden"]
        return {"bytes": moved, "flops": 12 * cells}
    rows, n, k, groups = case["rows"], case["n"], case["k"], case["groups"]
    busy = sum(c > 0 for c in _counts(case))
    tables = 16 * groups
    if case["op"] == "experts":
        moved = e * (rows * k + busy * n * k) + 2 * rows * n + tables
        moved += 4 * (rows + busy * n) if case["dtype"] == "e4m3" else 0
        return {"bytes": moved, "flops": 2 * rows * n * k}
    moved = e * (rows * k + rows * n + busy * n * k + rows * k + groups * n * k) + tables
    return {"bytes": moved, "flops": 4 * rows * n * k}


def exact(case, seed):
    """The definitions in 64 bits, before any rounding of the outputs, row group by
    row group.  An e4m3 output's values are y / scale."""
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_backward"):
        t, w = s["x"].double(), s["weight"].double()
        if case["op"] == "norm":
            if s["other"] is not None:
                t += s["other"].double()
            y = t / (t.pow(2).sum(1, keepdim=True) / case["hidden"] + EPS).sqrt() * w
            out = {}
            if case["out"] == "e4m3":
                out["scales"] = torch.clamp(y.abs().max(1).values / E4M3_MAX, min=SCALE_MIN)
                y = y / out["scales"].unsqueeze(1)
            out["y"] = y
            if s["other"] is not None:
                out["total"] = t
            return out
        dy = s["dy"].double()
        root = (t.pow(2).sum(1, keepdim=True) / case["hidden"] + EPS).sqrt()
        unit = t / root
        g = dy * w
        dx = (g - unit * (g * unit).sum(1, keepdim=True) / case["hidden"]) / root
        if s["other"] is not None:
            dx = dx + s["other"].double()
        return {"dx": dx, "dweight": (dy * unit).sum(0)}
    begin, count = s["begin"].tolist(), s["count"].tolist()
    rows, n, k = s["total_rows"], case["n"], case["k"]
    if case["op"] == "experts":
        y = torch.zeros(rows, n, device="cuda", dtype=torch.float64)
        for g in range(case["groups"]):
            at = slice(begin[g], begin[g] + count[g])
            x, w = s["x"][at].double(), s["w"][g].double()
            if s["x_scales"] is not None:
                x = x * s["x_scales"][at].double().unsqueeze(1)
                w = w * s["w_scales"][g].double().unsqueeze(1)
            y[at] = x @ w.t()
        return {"y": y}
    dx = torch.zeros(rows, k, device="cuda", dtype=torch.float64)
    dw = torch.zeros(case["groups"], n, k, device="cuda", dtype=torch.float64)
    for g in range(case["groups"]):
        at = slice(begin[g], begin[g] + count[g])
        dy = s["dy"][at].double()
        dx[at] = dy @ s["w"][g].double()
        dw[g] = dy.t() @ s["x"][at].double()
    return {"dx": dx, "dw": dw}
