"""The norms around a block with gate and residual scale, and their gradients, on a
GPU, against the definitions in 64 bits.

Tolerances.  With u = 2^-24: a sum over a row's `hidden` terms is off by at most S u
times the sum of their absolute values, S = hidden / 32 + 100 (a thread adds at most
hidden / 32 of them, the joins and the few products and roots at each end are in the
100).  Errors of a root and of what is built on it follow by first order, with the
absolute values of the terms that are added, and 5% for the second order; the
functions below carry them along.  Sums over rows have `rows` more terms.  An output
then has its own rounding: half a step, 2^-24 (f32), 2^-8 (bf16), 2^-4 or half of the
smallest step, 2^-10 (e4m3).
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
T = {0: torch.float32, 1: torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import __graft_entry__

    __graft_entry__.build()
    import collective_datapath_atom_gb300 as mod

    torch.cuda.set_device(0)
    return mod


@pytest.fixture(scope="module")
def ctx(P):
    c = P.purlin_init(1, torch.cuda.current_stream())
    yield c
    c.close()


def randn(*shape, seed, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def near(got, want, err):
    half = HALF[got.dtype]
    bad = ~((got.double() - want).abs() <= err * 1.05 + (want.abs() + err) * half * 1.01 + 1e-37)
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} off, e.g. {got[bad][0]} for {want[bad][0]} "
        f"within {err.expand_as(want)[bad][0]}")


def mean(v):
    return v.mean(1, keepdim=True)


def forward64(x, res, post, gate, w, a, b, eps=EPS):
    """(t, its error, v, its error)."""
    S = (x.shape[1] / 32 + 100) * U
    u = b * x.double()
    if gate is not None:
        u = u * gate.double()
    rel = 8 * U
    if post is not None:
        u = u * post.double() / torch.sqrt(mean(x.double().square()) + eps)
        rel += S
    t = u if res is None else u + a * res.double()
    et = u.abs() * rel + (0 if res is None else (a * res.double()).abs() * 4 * U) + t.abs() * U
    if w is None:
        return t, et, None, None
    r = 1 / torch.sqrt(mean(t.square()) + eps)
    er = mean(t.abs() * et) * r * r + S
    v = t * r * w.double()
    ev = (r * w.double()).abs() * (et + t.abs() * (er + 4 * U))
    return t, et, v, ev


def inputs(rows, hidden, dtype, post, gate, residual, seed=1, pitch=0, offset=0):
    dt = T[dtype]

    def mat(s, scale=1.0):
        return randn(rows, hidden + pitch + offset, seed=seed + s, dtype=dt, scale=scale)[:, offset:offset + hidden]

    return dict(x=mat(0), residual=mat(1, 2.0) if residual else None,
                post_weight=randn(hidden, seed=seed + 2, dtype=dt) if post else None,
                gate=None if gate is None else randn(hidden, seed=seed + 3, dtype=dt) if gate == "columns"
                else mat(4), weight=randn(hidden, seed=seed + 5, dtype=dt))


def run(P, ctx, i, dtype, a, b, out=None, total=True, y=True, gate_rows=False, eps=EPS):
    rows, hidden = i["x"].shape
    kind = T[dtype] if out is None else torch.float8_e4m3fn
    yy = torch.full((rows, hidden), 9.0, device="cuda").to(kind) if y else None
    tt = torch.full((rows, hidden), 9.0, device="cuda", dtype=T[dtype]) if total else None
    scales = torch.full((rows,), -1.0, device="cuda") if out is not None else None
    ld = lambda t: t.stride(0) if t is not None and t.dim() == 2 else 0  # noqa: E731
    P.purlin_block_norm(ctx, i["x"], i["weight"] if y else None, yy, rows, hidden, eps, dtype,
                        P.PURLIN_E4M3 if out is not None else dtype, residual=i["residual"],
                        post_weight=i["post_weight"], gate=i["gate"],
                        gate_layout=P.PURLIN_GATE_ROWS if gate_rows else P.PURLIN_GATE_COLUMNS,
                        residual_scale=a, block_scale=b, total=tt, scales=scales, ldx=ld(i["x"]),
                        ldg=ld(i["gate"]), ldr=ld(i["residual"]))
    P.purlin_check(ctx)
    return yy, tt, scales


# one row and many; short rows, odd ones, rows past the registers
SHAPES = [(1, 1), (3, 7), (1, 64), (1300, 64), (5, 200), (130, 1000), (33, 1021), (1, 4096), (700, 1024),
          (19, 4099), (7, 7168), (400, 2048), (3, 16384), (2, 33000)]


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("post", [False, True], ids=["", "post"])
@pytest.mark.parametrize("gate", [None, "columns", "rows"])
def test_forward(P, ctx, dtype, rows, hidden, post, gate):
    residual = rows != 5
    i = inputs(rows, hidden, dtype, post, gate, residual)
    y, t, _ = run(P, ctx, i, dtype, 0.9, 0.25, gate_rows=gate == "rows")
    t64, et, v, ev = forward64(i["x"], i["residual"], i["post_weight"], i["gate"], i["weight"], 0.9, 0.25)
    near(t, t64, et)
    near(y, v, ev)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("gate", ["columns", "rows"])
def test_forward_e4m3(P, ctx, dtype, rows, hidden, gate):
    i = inputs(rows, hidden, dtype, True, gate, True, seed=30)
    y, t, scales = run(P, ctx, i, dtype, 1.0, 0.5, out="e4m3", total=hidden % 2 == 0,
                       gate_rows=gate == "rows")
    t64, et, v, ev = forward64(i["x"], i["residual"], i["post_weight"], i["gate"], i["weight"], 1.0, 0.5)
    want = (v.abs().amax(1) / 448).clamp_min(2.0 ** -126)
    es = ev.amax(1) / 448 + want * 4 * U
    near(scales, want, es)
    q = v / want[:, None]
    eq = ev / want[:, None] + q.abs() * (es / want)[:, None] + q.abs() * 4 * U
    half = torch.maximum(q.abs() * 2.0 ** -4, torch.full_like(q, 2.0 ** -10))
    assert bool(((y.float().double() - q).abs() <= (half + eq) * 1.05).all())
    assert float(y.float().abs().max()) == 448.0
    if t is not None:
        near(t, t64, et)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("pitch,offset", [(3, 0), (8, 8), (1, 1)])
def test_forward_views(P, ctx, dtype, pitch, offset):
    for rows, hidden in ((40, 1000), (500, 1024), (9, 4096)):
        i = inputs(rows, hidden, dtype, True, "rows", True, 50, pitch, offset)
        y, t, _ = run(P, ctx, i, dtype, 1.1, -0.5, gate_rows=True)
        t64, et, v, ev = forward64(i["x"], i["residual"], i["post_weight"], i["gate"], i["weight"], 1.1, -0.5)
        near(t, t64, et)
        near(y, v, ev)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", [(4, 96), (9, 1021), (700, 2048), (2, 40000)])
def test_total_alone_and_in_place(P, ctx, dtype, rows, hidden):
    i = inputs(rows, hidden, dtype, True, "columns", True, 60)
    y, t, _ = run(P, ctx, i, dtype, 0.9, 0.25)
    _, only, _ = run(P, ctx, i, dtype, 0.9, 0.25, y=False)
    assert torch.equal(only, t)
    y2, none, _ = run(P, ctx, i, dtype, 0.9, 0.25, total=False)
    assert torch.equal(y2, y) and none is None
    x, res = i["x"].clone(), i["residual"].clone()
    P.purlin_block_norm(ctx, x, i["weight"], x, rows, hidden, EPS, dtype, residual=res,
                        post_weight=i["post_weight"], gate=i["gate"], residual_scale=0.9,
                        block_scale=0.25, total=res)
    P.purlin_check(ctx)
    assert torch.equal(x, y) and torch.equal(res, t)
    x, res = i["x"].clone(), i["residual"].clone()
    P.purlin_block_norm(ctx, x, i["weight"], res, rows, hidden, EPS, dtype, residual=res,
                        post_weight=i["post_weight"], gate=i["gate"], residual_scale=0.9,
                        block_scale=0.25, total=x)
    P.purlin_check(ctx)
    assert torch.equal(res, y) and torch.equal(x, t)


def test_specials(P, ctx):
    rows, hidden = 6, 256
    i = inputs(rows, hidden, 0, True, "columns", True, 70)
    i["x"][0] = 0.0                       # t is the residual alone
    i["x"][1], i["residual"][1] = 0.0, 0.0
    i["x"][2, 7] = math.inf               # q is 0: 0 * inf at that place
    i["residual"][3, 9] = math.nan
    i["x"][4] *= 1e-25
    y, t, scales = run(P, ctx, i, 0, 0.9, 0.25, out="e4m3")
    yf = y.float()
    assert torch.equal(t[0], i["residual"][0] * 0.9)
    assert not bool(yf[1].any()) and float(scales[1]) == 2.0 ** -126 and not bool(t[1].any())
    assert bool(torch.isnan(t[2, 7])) and bool(torch.isnan(yf[2]).all())
    assert bool(torch.isnan(t[3, 9])) and int(torch.isnan(t[3]).sum()) == 1
    assert bool(torch.isnan(yf[3]).all())
    assert bool(torch.isfinite(t[4:]).all()) and bool(torch.isfinite(yf[4:]).all())


# ---------------------------------------------------------------- backward ---

def backward64(i, dy, dtotal, total, a, b, eps=EPS):
    """Gradients by autograd in 64 bits, with t moved to `total` by a constant."""
    leaf = {k: None if v is None else v.double().requires_grad_(True) for k, v in i.items()}
    u = leaf["x"]
    if leaf["post_weight"] is not None:
        u = u / torch.sqrt(mean(u.square()) + eps) * leaf["post_weight"]
    if leaf["gate"] is not None:
        u = u * leaf["gate"]
    t = b * u + (a * leaf["residual"] if leaf["residual"] is not None else 0)
    if total is not None:
        t = t + (total.double() - t).detach()
    loss = 0
    if dy is not None:
        loss = (t / torch.sqrt(mean(t.square()) + eps) * leaf["weight"] * dy.double()).sum()
    if dtotal is not None:
        loss = loss + (t * dtotal.double()).sum()
    loss.backward()
    return {k: None if v is None else v.grad for k, v in leaf.items()}


def backward_errors(i, dy, dtotal, total, a, b, gate_rows, eps=EPS):
    rows, hidden = i["x"].shape
    S = (hidden / 32 + 100) * U
    x = i["x"].double()
    zero = torch.zeros_like(x)
    dt, edt, unit, r = zero, zero, None, None
    if dy is not None:
        n, t = (dy.double() * i["weight"].double()), total.double()
        r = 1 / torch.sqrt(mean(t.square()) + eps)
        size = r * (n.abs() + t.abs() * r * r * mean((n * t).abs()))
        dt = r * (n - t * r * r * mean(n * t))
        edt = size * 3 * S
    if dtotal is not None:
        dt = dt + dtotal.double()
        edt = edt + dt.abs() * 2 * U
    g = 1.0 if i["gate"] is None else i["gate"].double()
    p = 1.0 if i["post_weight"] is None else i["post_weight"].double()
    q = 1.0 if i["post_weight"] is None else 1 / torch.sqrt(mean(x.square()) + eps)
    f = b * g * p * torch.ones_like(x)
    h, eh = f * dt, (f.abs() * edt + (f * dt).abs() * 8 * U)
    e = {"dresidual": abs(a) * (edt + dt.abs() * 2 * U)}
    if i["post_weight"] is None:
        e["dx"] = eh
    else:
        e["dx"] = q * (eh + x.abs() * q * q * (mean(eh * x.abs()) + 4 * S * mean((h * x).abs()))
                       + (h.abs() + x.abs() * q * q * mean((h * x).abs())) * S)
    more = S + (rows + 10) * U
    if dy is not None:
        e["dweight"] = ((dy.double() * total.double() * r).abs() * more).sum(0)
    s = b * (x * q * g).abs()
    e["dpost_weight"] = (s * edt + s * dt.abs() * more).sum(0)
    d = abs(b) * (x * q * p).abs()
    d = d * edt + d * dt.abs() * more
    e["dgate"] = d if gate_rows else d.sum(0)
    return e


def run_backward(P, ctx, i, dy, dtotal, total, dtype, a, b, gate_rows, dresidual=True, out=None):
    rows, hidden = i["x"].shape
    ld = lambda t: t.stride(0) if t is not None and t.dim() == 2 else 0  # noqa: E731
    new = lambda: torch.full((rows, hidden), 9.0, device="cuda", dtype=T[dtype])  # noqa: E731
    vec = lambda: torch.full((hidden,), 9.0, device="cuda")  # noqa: E731
    o = dict(dx=new(), dresidual=new() if dresidual else None, dweight=vec() if dy is not None else None,
             dpost_weight=vec() if i["post_weight"] is not None else None,
             dgate=None if i["gate"] is None else new() if gate_rows else vec())
    o.update(out or {})
    P.purlin_block_norm_backward(
        ctx, dy, i["x"], total, i["weight"] if dy is not None else None, o["dx"], o["dweight"], rows,
        hidden, EPS, dtype, dtotal=dtotal, post_weight=i["post_weight"], gate=i["gate"],
        gate_layout=P.PURLIN_GATE_ROWS if gate_rows else P.PURLIN_GATE_COLUMNS, residual_scale=a,
        block_scale=b, dresidual=o["dresidual"], dpost_weight=o["dpost_weight"], dgate=o["dgate"],
        lddy=ld(dy), lddt=ld(dtotal), ldx=ld(i["x"]), ldt=ld(total), ldg=ld(i["gate"]),
        lddx=ld(o["dx"]), lddr=ld(o["dresidual"]), lddg=ld(o["dgate"]))
    P.purlin_check(ctx)
    return o


def check_backward(P, ctx, i, dy, dtotal, total, dtype, a, b, gate_rows, **kw):
    o = run_backward(P, ctx, i, dy, dtotal, total, dtype, a, b, gate_rows, **kw)
    want = backward64(i, dy, dtotal, total, a, b)
    err = backward_errors(i, dy, dtotal, total, a, b, gate_rows)
    for name, key in (("dx", "x"), ("dresidual", "residual"), ("dweight", "weight"),
                      ("dpost_weight", "post_weight"), ("dgate", "gate")):
        if o[name] is not None and want[key] is not None:
            near(o[name], want[key], err[name])
    return o


BACKWARD = [(1, 1), (3, 7), (1, 64), (1500, 64), (5, 200), (130, 1000), (33, 1021), (1, 4096),
            (700, 1024), (19, 4099), (7, 7168), (650, 2048), (3, 16384), (2, 33000)]


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", BACKWARD)
@pytest.mark.parametrize("post", [False, True], ids=["", "post"])
@pytest.mark.parametrize("gate", [None, "columns", "rows"])
def test_backward(P, ctx, dtype, rows, hidden, post, gate):
    i = inputs(rows, hidden, dtype, post, gate, True, seed=80)
    dy = randn(rows, hidden, seed=90, dtype=T[dtype])
    dtotal = randn(rows, hidden, seed=91, dtype=T[dtype]) if rows != 5 else None
    total = randn(rows, hidden, seed=92, dtype=T[dtype], scale=2.0)
    o = check_backward(P, ctx, i, dy, dtotal, total, dtype, 0.9, 0.25, gate == "rows")
    again = run_backward(P, ctx, i, dy, dtotal, total, dtype, 0.9, 0.25, gate == "rows")
    for k, v in o.items():       # the same bits every time
        assert v is None or torch.equal(v, again[k])


@pytest.mark.parametrize("dtype,hidden", [(0, 2048), (0, 2041), (0, 4090), (1, 4096), (1, 4089), (1, 7168), (1, 8181)])
@pytest.mark.parametrize("gate", [None, "columns", "rows"])
def test_backward_of_many_rows(P, ctx, dtype, hidden, gate):
    """More than 32 rows an SM, of about four, seven and eight warps of four windows each."""
    rows = 5003
    i = inputs(rows, hidden, dtype, gate != "rows", gate, True, seed=85)
    dy, dtotal, total = (randn(rows, hidden, seed=s, dtype=T[dtype]) for s in (95, 96, 97))
    o = check_backward(P, ctx, i, dy, dtotal, total, dtype, 0.9, 0.25, gate == "rows")
    again = run_backward(P, ctx, i, dy, dtotal, total, dtype, 0.9, 0.25, gate == "rows")
    for k, v in o.items():
        assert v is None or torch.equal(v, again[k])
    if gate == "columns":
        i = inputs(rows, hidden, dtype, True, "rows", True, 86, 1, 1)    # rows out of step
        check_backward(P, ctx, i, dy, None, total, dtype, 1.0, 0.5, True)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("gate", [None, "columns", "rows"])
def test_backward_of_total_alone(P, ctx, dtype, gate):
    for rows, hidden in ((40, 500), (640, 1024)):
        i = inputs(rows, hidden, dtype, True, gate, True, seed=100)
        dtotal = randn(rows, hidden, seed=101, dtype=T[dtype])
        check_backward(P, ctx, i, None, dtotal, None, dtype, 1.0, 0.5, gate == "rows")
        i["post_weight"] = None
        check_backward(P, ctx, i, None, dtotal, None, dtype, 1.0, 0.5, gate == "rows", dresidual=False)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("pitch,offset", [(3, 0), (8, 8), (1, 1)])
def test_backward_views(P, ctx, dtype, pitch, offset):
    for rows, hidden in ((40, 1000), (700, 1024), (9, 4096)):
        i = inputs(rows, hidden, dtype, True, "rows", True, 110, pitch, offset)
        more = inputs(rows, hidden, dtype, False, "rows", True, 120, pitch, offset)
        check_backward(P, ctx, i, more["x"], more["gate"], more["residual"], dtype, 1.0, 0.5, True)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", [(9, 1021), (700, 1024), (300, 4096), (2, 40000)])
def test_backward_in_place(P, ctx, dtype, rows, hidden):
    i = inputs(rows, hidden, dtype, True, "rows", True, 130)
    dy, dtotal, total = (randn(rows, hidden, seed=s, dtype=T[dtype]) for s in (131, 132, 133))
    o = run_backward(P, ctx, i, dy, dtotal, total, dtype, 0.9, 0.5, True)
    for places in (("dy", "dtotal", "total"), ("x", "gate", "dy"), ("total", "x", "gate"),
                   ("dtotal", "dy", "x")):
        c = dict(dy=dy.clone(), dtotal=dtotal.clone(), total=total.clone(), x=i["x"].clone(),
                 gate=i["gate"].clone())
        j = dict(i, x=c["x"], gate=c["gate"])
        out = dict(zip(("dx", "dresidual", "dgate"), (c[p] for p in places)))
        got = run_backward(P, ctx, j, c["dy"], c["dtotal"], c["total"], dtype, 0.9, 0.5, True, out=out)
        for k, v in o.items():
            assert torch.equal(v, got[k]), (places, k)


def test_backward_by_differences(P, ctx):
    """Central differences of the forward pass at two steps: the smaller one's error is
    a third of their difference (the next order's share, 4 to 1), which is allowed three
    times over, and the forward pass's own error over the step."""
    rows, hidden, a, b = 3, 24, 0.9, 0.5
    for gate in ("columns", "rows"):
        i = inputs(rows, hidden, 0, True, gate, True, 140)
        c, ct = randn(rows, hidden, seed=141, dtype=torch.float32), randn(rows, hidden, seed=142, dtype=torch.float32)
        y, t, _ = run(P, ctx, i, 0, a, b, gate_rows=gate == "rows")
        o = run_backward(P, ctx, i, c, ct, t, 0, a, b, gate == "rows")

        def value(j):
            y, t, _ = run(P, ctx, j, 0, a, b, gate_rows=gate == "rows")
            return float((y.double() * c).sum() + (t.double() * ct).sum())

        noise = float((y.abs() * c.abs()).sum() + (t.abs() * ct.abs()).sum()) * 110 * U
        for key, grad in (("x", "dx"), ("residual", "dresidual"), ("weight", "dweight"),
                          ("post_weight", "dpost_weight"), ("gate", "dgate")):
            d = randn(*i[key].shape, seed=143, dtype=torch.float32)
            diffs = []
            for h in (2.0 ** -5, 2.0 ** -6):
                ends = [value(dict(i, **{key: i[key] + s * h * d})) for s in (1, -1)]
                diffs.append((ends[0] - ends[1]) / (2 * h))
            want = float((o[grad].double() * d.double()).sum())
            # (the inputs' own rounding is in the noise: a step moves by 2^-24 relative)
            assert abs(diffs[1] - want) <= abs(diffs[0] - diffs[1]) + 2 * noise / 2.0 ** -6, key


def test_backward_of_no_rows(P, ctx):
    e = torch.empty(0, 40, device="cuda")
    v = [torch.full((40,), 5.0, device="cuda") for _ in range(3)]
    w = torch.ones(40, device="cuda")
    P.purlin_block_norm_backward(ctx, None, None, None, w, None, v[0], 0, 40, EPS, 0, post_weight=w,
                                 gate=w, dpost_weight=v[1], dgate=v[2])
    P.purlin_block_norm(ctx, None, None, None, 0, 40, EPS, 0)
    P.purlin_check(ctx)
    assert not any(bool(t.any()) for t in v)
    assert e.numel() == 0
