"""The norm and its gradients where the operands start at different places of a
16-byte window, or have pitches that differ: rows then go element by element.

Each operand has an offset and a pitch of its own, in a buffer whose other bytes
must stay as they were.  The bounds are those of the aligned rows (the sums have
another order, which those bounds allow).
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_rms_norm_gpu import (EPS, T, U, P, assert_close, assert_rounds, backward64,  # noqa: E402,F401
                               ctx, forward64, randn, slack)

# one element a thread, up to eight of them, and rows past the registers (2048 columns
# backward, 8192 forward); short rows a warp each; few rows and many
SHAPES = [(1, 1), (3, 7), (70, 31), (2000, 64), (300, 200), (5, 1000), (1300, 1021), (7, 2048),
          (6, 2049), (400, 4099), (3, 8192), (2, 8193), (3, 33000)]
# offset in elements and extra pitch of each operand in turn
PLACES = [((0, 0), (1, 0), (0, 0), (0, 0)), ((1, 3), (2, 5), (3, 0), (0, 8)),
          ((0, 1), (0, 2), (0, 1), (0, 0)), ((5, 8), (5, 8), (4, 8), (5, 16))]


def view(rows, hidden, place, dtype, fill):
    off, pad = place
    buf = torch.full((off + rows * (hidden + pad) + 32,), fill, device="cuda").to(dtype)
    v = torch.as_strided(buf, (rows, hidden), (hidden + pad, 1), off)
    return buf, v


def untouched(buf, v, fill):
    """Everything of buf outside v still holds fill."""
    v.copy_(torch.full_like(v, fill, dtype=torch.float32).to(v.dtype))
    assert bool((buf.float() == fill).all())


@pytest.mark.parametrize("dtype,out", [(0, 0), (1, 1), (0, 2), (1, 2)],
                         ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("places", PLACES, ids=["residual", "all", "pitches", "y"])
def test_forward(P, ctx, dtype, out, rows, hidden, places):
    dt = T[dtype]
    odt = torch.float8_e4m3fn if out == 2 else dt
    _, x = view(rows, hidden, places[0], dt, math.nan)
    _, res = view(rows, hidden, places[1], dt, math.nan)
    ybuf, y = view(rows, hidden, places[2], odt, 5.0)
    tbuf, tot = view(rows, hidden, places[3], dt, 5.0)
    x.copy_(randn(rows, hidden, seed=1, dtype=dt))
    res.copy_(randn(rows, hidden, seed=2, dtype=dt, scale=2.0))
    w = randn(hidden + 3, seed=3, dtype=dt)[3:]
    scales = torch.full((rows + 1,), -1.0, device="cuda") if out == 2 else None
    P.purlin_rms_norm(ctx, x, w, y, rows, hidden, EPS, dtype, out, residual=res, total=tot,
                      scales=scales, ldx=hidden + places[0][1], ldr=hidden + places[1][1],
                      ldy=hidden + places[2][1], ldt=hidden + places[3][1])
    P.purlin_check(ctx)
    t64, v64 = forward64(x, res, w)
    assert_close(tot, t64, 2 * U)
    if out == 2:
        want = (v64.abs().amax(1) / 448).clamp_min(2.0 ** -126)
        assert_close(scales[:rows], want, (slack(hidden) + 4 * U) * 1.01)
        assert float(scales[rows]) == -1.0
        q64 = v64 / want[:, None]
        bound = torch.maximum(q64.abs() * 2.0 ** -4, torch.full_like(q64, 2.0 ** -10))
        bound = bound + q64.abs() * 2 * (slack(hidden) + 4 * U)
        assert bool(((y.float().double() - q64).abs() <= bound * 1.01).all())
    else:
        assert_close(y, v64, slack(hidden) * 1.01)
    untouched(ybuf, y, 5.0)
    untouched(tbuf, tot, 5.0)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("hidden", [64, 1021, 9000])
def test_no_residual_and_in_place(P, ctx, dtype, hidden):
    """y at another phase than x; then total over the residual, at x's other phase."""
    rows, dt = 37, T[dtype]
    _, x = view(rows, hidden, (1, 0), dt, math.nan)
    ybuf, y = view(rows, hidden, (0, 3), dt, 5.0)
    x.copy_(randn(rows, hidden, seed=4, dtype=dt))
    w = randn(hidden, seed=5, dtype=dt)
    P.purlin_rms_norm(ctx, x, w, y, rows, hidden, EPS, dtype, ldy=hidden + 3)
    P.purlin_check(ctx)
    assert_close(y, forward64(x, None, w)[1], slack(hidden) * 1.01)
    untouched(ybuf, y, 5.0)
    rbuf, res = view(rows, hidden, (2, 3), dt, 5.0)
    res.copy_(randn(rows, hidden, seed=6, dtype=dt))
    t64, v64 = forward64(x, res, w)
    P.purlin_rms_norm(ctx, x, w, x, rows, hidden, EPS, dtype, residual=res, total=res,
                      ldr=hidden + 3, ldt=hidden + 3)
    P.purlin_check(ctx)
    assert_close(x, v64, slack(hidden) * 1.01)
    assert_close(res, t64, 2 * U)
    untouched(rbuf, res, 5.0)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("places", PLACES, ids=["total", "all", "pitches", "dtotal"])
@pytest.mark.parametrize("stream_grad", [False, True], ids=["plain", "dtotal"])
def test_backward(P, ctx, dtype, rows, hidden, places, stream_grad):
    dt = T[dtype]
    _, dy = view(rows, hidden, places[0], dt, math.nan)
    _, t = view(rows, hidden, places[1], dt, math.nan)
    _, dtot = view(rows, hidden, places[2], dt, math.nan)
    xbuf, dx = view(rows, hidden, places[3], dt, 5.0)
    dy.copy_(randn(rows, hidden, seed=21, dtype=dt))
    t.copy_(randn(rows, hidden, seed=20, dtype=dt, scale=2.0))
    dtot.copy_(randn(rows, hidden, seed=23, dtype=dt))
    dtot = dtot if stream_grad else None
    w = randn(hidden + 1, seed=22, dtype=dt)[1:]
    dw = torch.full((hidden + 1,), 9.0, device="cuda")
    lds = dict(lddy=hidden + places[0][1], ldt=hidden + places[1][1],
               lddt=hidden + places[2][1], lddx=hidden + places[3][1])

    def call():
        P.purlin_rms_norm_backward(ctx, dy, t, w, dx, dw, rows, hidden, EPS, dtype, dtotal=dtot,
                                   **lds)
        P.purlin_check(ctx)

    call()
    dx64, dw64 = backward64(t, dy, w, dtot)
    r = 1 / torch.sqrt(t.double().square().mean(1, keepdim=True) + EPS)
    g, td = (dy.double() * w.double()).abs(), t.double().abs()
    scale = r * (g + td * r * r * (g * td).mean(1, keepdim=True))
    if dtot is not None:
        scale = scale + dtot.double().abs()
    assert_rounds(dx, dx64, 4 * slack(hidden) * scale + 1e-37)
    size = (dy.double() * t.double() * r).abs().sum(0)
    assert bool(((dw[:hidden].double() - dw64).abs() <=
                 (rows * U + 2 * slack(hidden)) * size + 1e-37).all())
    assert float(dw[hidden]) == 9.0
    first, first_w = dx.clone(), dw.clone()
    call()
    assert torch.equal(dx, first) and torch.equal(dw, first_w)     # the same bits every time
    untouched(xbuf, dx, 5.0)
