"""The norms around a block for many wide rows on a GPU: teams of up to sixteen warps,
rings of one stage and of more, windows held and read again, vectors in shared and in
global memory, with and without ends; and rows of special values, and in place, among as
many rows as take that way.  References and tolerances are those of
test_block_norm_gpu.py.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_block_norm_gpu import (EPS, T, U, P, check_backward, ctx, forward64, inputs, near, randn,  # noqa: E402, F401
                                 run, run_backward)

ROWS = 700      # four or five a block of one team: every stage is filled again

WIDE = [(0, 4099), (0, 5120), (0, 7161), (0, 8192), (0, 8200), (0, 10001), (0, 12001), (0, 16384),
        (1, 4099), (1, 5120), (1, 7168), (1, 8200), (1, 10001), (1, 12001), (1, 16380), (1, 16384)]


@pytest.mark.parametrize("dtype,hidden", WIDE)
@pytest.mark.parametrize("gate", [None, "columns", "rows"])
def test_forward(P, ctx, dtype, hidden, gate):  # noqa: F811
    for post, residual, pitch, offset in ((True, True, 0, 0), (gate is None, gate != "rows", 1, 1)):
        i = inputs(ROWS, hidden, dtype, post, gate, residual, 200, pitch, offset)
        y, t, _ = run(P, ctx, i, dtype, 0.9, 0.25, gate_rows=gate == "rows")
        t64, et, v, ev = forward64(i["x"], i["residual"], i["post_weight"], i["gate"], i["weight"], 0.9, 0.25)
        near(t, t64, et)
        near(y, v, ev)
        y2, none, _ = run(P, ctx, i, dtype, 0.9, 0.25, total=False, gate_rows=gate == "rows")
        _, t2, _ = run(P, ctx, i, dtype, 0.9, 0.25, y=False, gate_rows=gate == "rows")
        assert torch.equal(y2, y) and torch.equal(t2, t) and none is None


@pytest.mark.parametrize("dtype,hidden", WIDE)
@pytest.mark.parametrize("gate", ["columns", "rows"])
def test_forward_e4m3(P, ctx, dtype, hidden, gate):  # noqa: F811
    for pitch in (0, 1):
        i = inputs(ROWS, hidden, dtype, True, gate, True, 210, pitch, pitch)
        # (their sum is to stay a view with that pitch)
        y, _, scales = run(P, ctx, i, dtype, 1.0, 0.5, out="e4m3", total=False, gate_rows=gate == "rows")
        t64, et, v, ev = forward64(i["x"], i["residual"], i["post_weight"], i["gate"], i["weight"], 1.0, 0.5)
        want = (v.abs().amax(1) / 448).clamp_min(2.0 ** -126)
        es = ev.amax(1) / 448 + want * 4 * U
        near(scales, want, es)
        q = v / want[:, None]
        eq = ev / want[:, None] + q.abs() * (es / want)[:, None] + q.abs() * 4 * U
        half = torch.maximum(q.abs() * 2.0 ** -4, torch.full_like(q, 2.0 ** -10))
        assert bool(((y.float().double() - q).abs() <= (half + eq) * 1.05).all())


@pytest.mark.parametrize("dtype,hidden", WIDE)
@pytest.mark.parametrize("gate", [None, "columns", "rows"])
def test_backward(P, ctx, dtype, hidden, gate):  # noqa: F811
    for post, dt, pitch, offset in ((True, True, 0, 0), (gate == "columns", gate is None, 1, 1)):
        i = inputs(ROWS, hidden, dtype, post, gate, True, 220, pitch, offset)
        more = inputs(ROWS, hidden, dtype, False, "rows", True, 230, pitch, offset)
        dy, total, dtotal = more["x"], more["residual"], more["gate"] if dt else None
        o = check_backward(P, ctx, i, dy, dtotal, total, dtype, 0.9, 0.25, gate == "rows")
        again = run_backward(P, ctx, i, dy, dtotal, total, dtype, 0.9, 0.25, gate == "rows")
        for k, v in o.items():
            assert v is None or torch.equal(v, again[k])


# whole windows and rows with ends, rings of one stage among them
IN_PLACE = [(0, 1021), (0, 5121), (0, 10001), (0, 8192), (1, 1021), (1, 4099), (1, 8200), (1, 12001)]


@pytest.mark.parametrize("dtype,hidden", IN_PLACE)
def test_in_place(P, ctx, dtype, hidden):  # noqa: F811
    i = inputs(ROWS, hidden, dtype, True, "rows", True, 240)
    y, t, _ = run(P, ctx, i, dtype, 0.9, 0.25, gate_rows=True)
    for swap in (False, True):
        x, res = i["x"].clone(), i["residual"].clone()
        to_y, to_t = (res, x) if swap else (x, res)
        P.purlin_block_norm(ctx, x, i["weight"], to_y, ROWS, hidden, EPS, dtype, residual=res, total=to_t,
                            post_weight=i["post_weight"], gate=i["gate"], gate_layout=P.PURLIN_GATE_ROWS,
                            residual_scale=0.9, block_scale=0.25)
        P.purlin_check(ctx)
        assert torch.equal(to_y, y) and torch.equal(to_t, t)
    dy, dtotal, total = (randn(ROWS, hidden, seed=s, dtype=T[dtype]) for s in (241, 242, 243))
    o = run_backward(P, ctx, i, dy, dtotal, total, dtype, 0.9, 0.5, True)
    for places in (("dy", "dtotal", "total"), ("x", "gate", "dy"), ("total", "x", "gate"), ("dtotal", "dy", "x")):
        c = dict(dy=dy.clone(), dtotal=dtotal.clone(), total=total.clone(), x=i["x"].clone(), gate=i["gate"].clone())
        j = dict(i, x=c["x"], gate=c["gate"])
        out = dict(zip(("dx", "dresidual", "dgate"), (c[p] for p in places)))
        got = run_backward(P, ctx, j, c["dy"], c["dtotal"], c["total"], dtype, 0.9, 0.5, True, out=out)
        for k, v in o.items():
            assert torch.equal(v, got[k]), (places, k)


@pytest.mark.parametrize("hidden", [256, 1021, 7168, 10001])
def test_special_rows_among_many(P, ctx, hidden):  # noqa: F811
    """A row of specials shows in itself alone; the others keep their bits."""
    def make():
        return inputs(ROWS, hidden, 0, True, "columns", True, 250)

    clean, i = make(), make()
    at = [0, 151, 152, 303, 460, 699]      # in a block's first, second, third and last row
    i["x"][at[0]] = 0.0
    i["x"][at[1]], i["residual"][at[1]] = 0.0, 0.0
    i["x"][at[2], 7] = math.inf
    i["residual"][at[3], 9] = math.nan
    i["x"][at[4]] *= 1e-25
    i["residual"][at[5], hidden - 1] = -math.inf
    others = torch.ones(ROWS, dtype=torch.bool, device="cuda")
    others[at] = False
    for out in (None, "e4m3"):
        y0, t0, s0 = run(P, ctx, clean, 0, 0.9, 0.25, out=out)
        y, t, s = run(P, ctx, i, 0, 0.9, 0.25, out=out)
        yf = y.float()
        assert torch.equal(yf[others], y0.float()[others]) and torch.equal(t[others], t0[others])
        assert torch.equal(t[at[0]], i["residual"][at[0]] * 0.9)
        assert not bool(yf[at[1]].any()) and not bool(t[at[1]].any())
        assert bool(torch.isnan(t[at[2], 7])) and bool(torch.isnan(yf[at[2]]).all())
        assert int(torch.isnan(t[at[3]]).sum()) == 1 and bool(torch.isnan(yf[at[3]]).all())
        assert bool(torch.isfinite(t[at[4]]).all()) and bool(torch.isfinite(yf[at[4]]).all())
        # an infinite mean: every finite value is 0, the infinite one NaN
        assert bool(torch.isnan(yf[at[5], hidden - 1])) and not bool(yf[at[5], :hidden - 1].any())
        if out:
            assert torch.equal(s[others], s0[others]) and float(s[at[1]]) == 2.0 ** -126


@pytest.mark.parametrize("hidden", [256, 1021, 7168, 10001])
@pytest.mark.parametrize("gate", ["columns", "rows"])
def test_special_rows_of_the_gradient(P, ctx, hidden, gate):  # noqa: F811
    i = inputs(ROWS, hidden, 0, True, gate, True, 260)
    given = {k: randn(ROWS, hidden, seed=s, dtype=torch.float32) for k, s in (("dy", 261), ("dtotal", 262), ("total", 263))}

    def gradients(i, given):
        return run_backward(P, ctx, i, given["dy"], given["dtotal"], given["total"], 0, 0.9, 0.25, gate == "rows")

    o = gradients(i, given)
    bad = dict(i, x=i["x"].clone()), {k: v.clone() for k, v in given.items()}
    at = [1, 153, 304, 699]
    bad[1]["dy"][at[0], 5] = math.nan
    bad[1]["dtotal"][at[1], hidden - 1] = math.nan
    bad[1]["total"][at[2], 0] = math.inf
    bad[0]["x"][at[3], 3] = math.nan
    got = gradients(*bad)
    others = torch.ones(ROWS, dtype=torch.bool, device="cuda")
    others[at] = False
    for k in ("dx", "dresidual") + (("dgate",) if gate == "rows" else ()):
        assert torch.equal(got[k][others], o[k][others])
        assert bool(torch.isfinite(got[k][others]).all())
    nan = torch.isnan(got["dresidual"])
    assert bool(nan[at[0]].all())                         # the projection on t takes it everywhere
    assert int(nan[at[1]].sum()) == 1 and bool(nan[at[1], hidden - 1])
    assert not bool(nan[at[3]].any())
    assert bool(torch.isnan(got["dx"][at]).all(1)[[0, 1, 3]].all())
    assert bool(torch.isnan(got["dweight"][5])) and bool(torch.isnan(got["dpost_weight"]).any())


@pytest.mark.parametrize("hidden", [264, 2048, 7161, 10001])
def test_tiny_and_infinite_scales(P, ctx, hidden):  # noqa: F811
    """Rows of 1 and no eps: v is the weight.  Quotients near the smallest normal scale
    are the same as far from it; an infinite scale leaves finite values zero."""
    one = torch.ones(ROWS, hidden, device="cuda")
    w = torch.rand(hidden, device="cuda", generator=torch.Generator(device="cuda").manual_seed(270)) + 0.5
    w[0] = 2.0

    def norm(x, w):
        y = torch.empty(ROWS, hidden, device="cuda", dtype=torch.float8_e4m3fn)
        scales = torch.empty(ROWS, device="cuda")
        P.purlin_block_norm(ctx, x, w, y, ROWS, hidden, 0.0, 0, P.PURLIN_E4M3, scales=scales)
        P.purlin_check(ctx)
        return y.float(), scales

    want = (w / (w[0] / 448)).to(torch.float8_e4m3fn).float()
    for power in (0, -70, -90, -115, 100):
        y, s = norm(one, w * 2.0 ** power)
        assert bool((s == w[0] / 448 * 2.0 ** power).all())
        assert torch.equal(y, want.expand(ROWS, hidden))
    x = one * 2
    x[:, 1::2] = 0.125                  # mean square just above 2: the root is below 1
    big = torch.ones(hidden, device="cuda")
    big[0] = 3.4e38
    y, s = norm(x, big)                 # 2 / root(2) times 3.4e38: past the largest value
    assert bool(s.isinf().all()) and bool(y[:, 0].isnan().all()) and not bool(y[:, 1:].any())
