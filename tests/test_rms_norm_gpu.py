"""The RMS norm with the residual's addition, its e4m3 output and its backward
pass on a GPU, against the definitions in 64 bits.

Tolerances.  With u = 2^-24 (binary32): t carries one rounding (u, relative);
the sum of squares of `hidden` positive terms, split over threads that add at
most hidden / 32 terms each and joined by at most 64 more additions, is off by
(hidden / 32 + 64) u relative, half of that in its root; the root, the products
and the division add a few u.  So a value before its output rounding is off by
at most S u relative, S = hidden / 32 + 80.  An output in f32 or bf16 then has
to be what some value within that error rounds to: rounding is monotone, so it
lies between the roundings of the interval's two ends.  e4m3 adds 2^-4 relative
or 2^-10 absolute (half its smallest step).  Backward sums have signs, so their
bounds use the sums of absolute values.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5
T = {0: torch.float32, 1: torch.bfloat16}


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


def slack(hidden):
    return (hidden / 32 + 80) * U


def randn(*shape, seed, dtype, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def forward64(x, res, w, eps=EPS):
    t = x.double() if res is None else x.double() + res.double()
    v = t / torch.sqrt(t.square().mean(1, keepdim=True) + eps) * w.double()
    return t, v


def assert_rounds(got, want, err):
    """got is the rounding of some value within err of want (rounding is monotone)."""
    low, high = (want - err).to(got.dtype), (want + err).to(got.dtype)
    bad = ~((got >= low) & (got <= high))
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} off, e.g. {got[bad][0]} for {want[bad][0]}")


def assert_close(got, want, rel):
    assert_rounds(got, want, want.abs() * rel + 1e-37)


# one row and many; one warp a row, blocks, scalar columns, rows past the registers
SHAPES = [(1, 1), (3, 7), (1, 64), (257, 64), (5, 200), (130, 1000), (33, 1021), (1, 4096),
          (19, 4099), (7, 7168), (3, 16384), (2, 33000), (2, 66000)]


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("residual,total", [(False, False), (True, True), (True, False),
                                            (False, True)])
def test_forward(P, ctx, dtype, rows, hidden, residual, total):
    dt = T[dtype]
    x = randn(rows, hidden, seed=1, dtype=dt)
    res = randn(rows, hidden, seed=2, dtype=dt, scale=2.0) if residual else None
    w = randn(hidden, seed=3, dtype=dt)
    y = torch.full((rows, hidden), 9.0, device="cuda", dtype=dt)
    tot = torch.full_like(y, 9.0) if total else None
    P.purlin_rms_norm(ctx, x, w, y, rows, hidden, EPS, dtype, residual=res, total=tot)
    P.purlin_check(ctx)
    t64, v64 = forward64(x, res, w)
    assert_close(y, v64, slack(hidden) * 1.01)
    if total:
        assert_close(tot, t64, 2 * U)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", SHAPES)
def test_forward_e4m3(P, ctx, dtype, rows, hidden):
    dt = T[dtype]
    x = randn(rows, hidden, seed=4, dtype=dt)
    res = randn(rows, hidden, seed=5, dtype=dt)
    w = randn(hidden, seed=6, dtype=dt)
    y = torch.full((rows, hidden), 9.0, device="cuda").to(torch.float8_e4m3fn)
    tot = torch.empty_like(x)
    scales = torch.full((rows,), -1.0, device="cuda")
    P.purlin_rms_norm(ctx, x, w, y, rows, hidden, EPS, dtype, P.PURLIN_E4M3, residual=res,
                      total=tot, scales=scales)
    P.purlin_check(ctx)
    t64, v64 = forward64(x, res, w)
    want_scale = (v64.abs().amax(1) / 448).clamp_min(2.0 ** -126)
    assert_close(scales, want_scale, (slack(hidden) + 4 * U) * 1.01)
    q64 = v64 / want_scale[:, None]
    got = y.float().double()
    # an element's own error moves it by 2 S u of itself before it is rounded
    bound = torch.maximum(q64.abs() * 2.0 ** -4, torch.full_like(q64, 2.0 ** -10))
    bound = bound + q64.abs() * 2 * (slack(hidden) + 4 * U)
    assert bool(((got - q64).abs() <= bound * 1.01).all())
    assert float(got.abs().max()) == 448.0          # each row's largest value uses the range
    assert_close(tot, t64, 2 * U)


def test_e4m3_rounds_to_nearest_even(P, ctx):
    # rows whose norm is exact: t in {+-1}, weights chosen so that v / scale hits
    # ties, subnormals and the largest value
    w = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, -17.0, 1.0],
                     device="cuda")
    x = torch.ones(1, 8, device="cuda")
    y = torch.empty(1, 8, device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty(1, device="cuda")
    P.purlin_rms_norm(ctx, x, w, y, 1, 8, 0.0, 0, P.PURLIN_E4M3, scales=scales)
    P.purlin_check(ctx)
    assert float(scales) == 1.0
    want = [448.0, 16.0, 20.0, 0.0, 2.0 ** -8, 2.0 ** -9, -16.0, 1.0]
    assert y.float().reshape(-1).tolist() == want


@pytest.mark.parametrize("hidden", [8, 1000, 1021, 40000])
@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
def test_empty_rows_and_special_values(P, ctx, dtype, hidden):
    """A zero row, a NaN, an infinity and a row whose squares overflow, with
    ordinary rows between them that must not notice."""
    dt = T[dtype]
    x = randn(6, hidden, seed=7, dtype=dt)
    x[1] = 0
    x[2, hidden // 2] = math.nan
    x[3, 0] = math.inf
    x[4] = 1e30
    w = randn(hidden, seed=8, dtype=dt)
    w[w == 0] = 1
    y = torch.empty_like(x)
    P.purlin_rms_norm(ctx, x, w, y, 6, hidden, EPS, dtype)
    q = torch.empty(6, hidden, device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty(6, device="cuda")
    P.purlin_rms_norm(ctx, x, w, q, 6, hidden, EPS, dtype, P.PURLIN_E4M3, scales=scales)
    P.purlin_check(ctx)
    for row in (0, 5):
        _, v = forward64(x[row:row + 1], None, w)
        assert_close(y[row:row + 1], v, slack(hidden) * 1.01)
    assert bool((y[1] == 0).all()) and bool((q[1].float() == 0).all())
    assert float(scales[1]) == 2.0 ** -126
    assert bool(y[2].isnan().all()) and bool(q[2].float().isnan().all())
    assert bool(y[3, 0].isnan()) and bool((y[3, 1:] == 0).all())
    assert bool((y[4] == 0).all())            # the mean square overflows binary32
    assert bool(scales[[0, 5]].isfinite().all()) and bool(q[[0, 5]].float().isfinite().all())


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 3], ids=["aligned", "off1", "off3"])
@pytest.mark.parametrize("pad", [0, 1, 24])
def test_strides_alignment_and_guards(P, ctx, dtype, offset, pad):
    rows, hidden = 21, 264
    dt = T[dtype]

    def view(fill, odt=dt, seed=None):
        buf = torch.full((rows * (hidden + pad) + 64,), fill, device="cuda", dtype=odt)
        v = buf[offset:offset + rows * (hidden + pad)].view(rows, hidden + pad)[:, :hidden]
        if seed is not None:
            v.copy_(randn(rows, hidden, seed=seed, dtype=odt))
        return buf, v

    _, x = view(math.nan, seed=9)
    _, res = view(math.nan, seed=10)
    w = randn(hidden, seed=11, dtype=dt)
    ybuf, y = view(5.0)
    tbuf, tot = view(5.0)
    ld = hidden + pad
    P.purlin_rms_norm(ctx, x, w, y, rows, hidden, EPS, dtype, residual=res, total=tot, ldx=ld,
                      ldr=ld, ldy=ld, ldt=ld)
    P.purlin_check(ctx)
    t64, v64 = forward64(x, res, w)
    assert_close(y, v64, slack(hidden) * 1.01)
    assert_close(tot, t64, 2 * U)
    for buf, v in ((ybuf, y), (tbuf, tot)):
        v.fill_(5.0)
        assert bool((buf == 5.0).all())       # nothing outside the view was written


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("hidden", [512, 4099, 70000])
def test_in_place(P, ctx, dtype, hidden):
    rows, dt = 9, T[dtype]
    x = randn(rows, hidden, seed=12, dtype=dt)
    res = randn(rows, hidden, seed=13, dtype=dt)
    w = randn(hidden, seed=14, dtype=dt)
    y, tot = torch.empty_like(x), torch.empty_like(x)
    P.purlin_rms_norm(ctx, x, w, y, rows, hidden, EPS, dtype, residual=res, total=tot)
    a, b = x.clone(), res.clone()             # y over x, total over the residual
    P.purlin_rms_norm(ctx, a, w, a, rows, hidden, EPS, dtype, residual=b, total=b)
    P.purlin_check(ctx)
    assert torch.equal(a, y) and torch.equal(b, tot)


def backward64(t, dy, w, dtotal, eps=EPS):
    t, dy, w = t.double(), dy.double(), w.double()
    r = 1 / torch.sqrt(t.square().mean(1, keepdim=True) + eps)
    g = dy * w
    dx = r * (g - t * r * r * (g * t).mean(1, keepdim=True))
    if dtotal is not None:
        dx = dx + dtotal.double()
    return dx, (dy * t * r).sum(0)


BACKWARD_SHAPES = [(1, 1), (2, 9), (1, 64), (700, 64), (65, 1000), (400, 1021), (3, 4096),
                   (305, 4099), (37, 7168), (4, 16384), (3, 33000), (311, 8200), (2, 70000)]


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", BACKWARD_SHAPES)
@pytest.mark.parametrize("stream_grad", [False, True], ids=["plain", "dtotal"])
def test_backward(P, ctx, dtype, rows, hidden, stream_grad):
    dt = T[dtype]
    t = randn(rows, hidden, seed=20, dtype=dt, scale=2.0)
    dy = randn(rows, hidden, seed=21, dtype=dt)
    w = randn(hidden, seed=22, dtype=dt)
    dtot = randn(rows, hidden, seed=23, dtype=dt) if stream_grad else None
    dx = torch.full_like(t, 9.0)
    dw = torch.full((hidden,), 9.0, device="cuda")
    P.purlin_rms_norm_backward(ctx, dy, t, w, dx, dw, rows, hidden, EPS, dtype, dtotal=dtot)
    P.purlin_check(ctx)
    dx64, dw64 = backward64(t, dy, w, dtot)
    r = 1 / torch.sqrt(t.double().square().mean(1, keepdim=True) + EPS)
    g, td = (dy.double() * w.double()).abs(), t.double().abs()
    scale = r * (g + td * r * r * (g * td).mean(1, keepdim=True))
    if dtot is not None:
        scale = scale + dtot.double().abs()
    # r^3 carries three halves of the sum's error, mean(g t) a whole one
    assert_rounds(dx, dx64, 4 * slack(hidden) * scale + 1e-37)
    # rows additions in any order, each term off by S u
    size = (dy.double() * t.double() * r).abs().sum(0)
    assert bool(((dw.double() - dw64).abs() <= (rows * U + 2 * slack(hidden)) * size + 1e-37).all())
    again, aw = torch.empty_like(dx), torch.empty_like(dw)
    P.purlin_rms_norm_backward(ctx, dy, t, w, again, aw, rows, hidden, EPS, dtype, dtotal=dtot)
    P.purlin_check(ctx)
    assert torch.equal(again, dx) and torch.equal(aw, dw)     # the same bits every time


def test_backward_against_differences(P, ctx):
    rows, hidden = 3, 17
    x = randn(rows, hidden, seed=30, dtype=torch.float32)
    dy = randn(rows, hidden, seed=31, dtype=torch.float32)
    dtot = randn(rows, hidden, seed=32, dtype=torch.float32)
    w = randn(hidden, seed=33, dtype=torch.float32)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    P.purlin_rms_norm_backward(ctx, dy, x, w, dx, dw, rows, hidden, EPS, 0, dtotal=dtot)
    P.purlin_check(ctx)

    def loss(xx, ww):
        t, v = forward64(xx, None, ww)
        return float((v * dy.double()).sum() + (t * dtot.double()).sum())

    h = 1e-4   # central differences in 64 bits: error h^2 times a third derivative of order 10
    for i in range(rows):
        for j in range(hidden):
            e = torch.zeros_like(x, dtype=torch.float64)
            e[i, j] = h
            d = (loss(x.double() + e, w) - loss(x.double() - e, w)) / (2 * h)
            assert abs(d - float(dx[i, j])) < 2e-5
    for j in range(hidden):
        e = torch.zeros_like(w, dtype=torch.float64)
        e[j] = h
        d = (loss(x, w.double() + e) - loss(x, w.double() - e)) / (2 * h)
        assert abs(d - float(dw[j])) < 2e-5


@pytest.mark.parametrize("into", ["dy", "total", "dtotal"])
@pytest.mark.parametrize("hidden", [512, 1021, 70000])
def test_backward_in_place(P, ctx, into, hidden):
    rows = 11
    bufs = {k: randn(rows, hidden, seed=40 + i, dtype=torch.bfloat16)
            for i, k in enumerate(("dy", "total", "dtotal"))}
    w = randn(hidden, seed=44, dtype=torch.bfloat16)
    dx = torch.empty_like(bufs["dy"])
    dw, dw2 = torch.empty(hidden, device="cuda"), torch.empty(hidden, device="cuda")
    P.purlin_rms_norm_backward(ctx, bufs["dy"], bufs["total"], w, dx, dw, rows, hidden, EPS, 1,
                               dtotal=bufs["dtotal"])
    P.purlin_rms_norm_backward(ctx, bufs["dy"], bufs["total"], w, bufs[into], dw2, rows, hidden,
                               EPS, 1, dtotal=bufs["dtotal"])
    P.purlin_check(ctx)
    assert torch.equal(bufs[into], dx) and torch.equal(dw, dw2)


def test_no_rows(P, ctx):
    w = torch.ones(32, device="cuda")
    dw = torch.full((32,), 3.0, device="cuda")
    P.purlin_rms_norm(ctx, 0, w, 0, 0, 32, EPS, 0)
    P.purlin_rms_norm_backward(ctx, 0, 0, w, 0, dw, 0, 32, EPS, 0)
    P.purlin_check(ctx)
    assert bool((dw == 0).all())


def test_offsets_past_32_bits(P, ctx):
    """Rows 2^31 elements apart: row offsets pass 32 bits in elements and bytes."""
    ld, hidden = (1 << 31) + 8, 256
    if torch.cuda.mem_get_info()[0] < 3 * ld * 2:
        pytest.skip("needs 13 GB")
    buf = torch.empty(2 * ld + hidden, device="cuda", dtype=torch.bfloat16)
    x = torch.as_strided(buf, (3, hidden), (ld, 1))
    x.copy_(randn(3, hidden, seed=50, dtype=torch.bfloat16))
    w = randn(hidden, seed=51, dtype=torch.bfloat16)
    y = torch.empty(3, hidden, device="cuda", dtype=torch.bfloat16)
    P.purlin_rms_norm(ctx, x, w, y, 3, hidden, EPS, 1, ldx=ld)
    P.purlin_check(ctx)
    assert_close(y, forward64(x, None, w)[1], slack(hidden) * 1.01)


def test_side_stream_and_graph(P):
    s = torch.cuda.Stream()
    c = P.purlin_init(1, s)
    try:
        rows, hidden = 64, 1024
        w = randn(hidden, seed=60, dtype=torch.bfloat16)
        x, dy = (randn(rows, hidden, seed=k, dtype=torch.bfloat16) for k in (61, 62))
        y, dx = torch.empty_like(x), torch.empty_like(x)
        dw = torch.empty(hidden, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        # a graph cannot allocate: the workspace has to be there before it
        with torch.cuda.graph(g, stream=s):
            P.purlin_rms_norm(c, x, w, y, rows, hidden, EPS, 1)
            with pytest.raises(P.PurlinError) as e:
                P.purlin_rms_norm_backward(c, dy, y, w, dx, dw, rows, hidden, EPS, 1)
            assert e.value.status == P.PURLIN_ERR_UNSUPPORTED
        P.purlin_rms_norm_backward(c, dy, y, w, dx, dw, rows, hidden, EPS, 1)
        P.purlin_check(c)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            P.purlin_rms_norm(c, x, w, y, rows, hidden, EPS, 1)
            P.purlin_rms_norm_backward(c, dy, y, w, dx, dw, rows, hidden, EPS, 1)
        # a later call that outgrows the workspace must leave the graph's alone
        big = torch.ones(2000, 8192, device="cuda", dtype=torch.bfloat16)
        P.purlin_rms_norm_backward(c, big, big, big[0], torch.empty_like(big),
                                   torch.empty(8192, device="cuda"), 2000, 8192, EPS, 1)
        for k in range(3):
            with torch.cuda.stream(s):
                x.copy_(randn(rows, hidden, seed=70 + k, dtype=torch.bfloat16))
            s.synchronize()
            g.replay()
            s.synchronize()
            assert_close(y, forward64(x, None, w)[1], slack(hidden) * 1.01)
            dw64 = backward64(y, dy, w, None)[1]
            size = (dy.double() * y.double()).abs().sum(0) * 2
            assert bool(((dw.double() - dw64).abs() <= 200 * U * size).all())
    finally:
        c.close()


# rows enough for persistent blocks that bring rows through shared memory: one to
# five blocks an SM, two to four stages, every window edge, both operand counts
MANY = [(2600, 1032), (2500, 1027), (1900, 4096), (1700, 4099), (1000, 7168), (700, 8192),
        (640, 16384), (640, 16379), (3000, 2049)]


@pytest.mark.parametrize("dtype,out", [(0, 0), (1, 1), (0, 2), (1, 2)],
                         ids=["f32", "bf16", "f32-e4m3", "bf16-e4m3"])
@pytest.mark.parametrize("rows,hidden", MANY)
@pytest.mark.parametrize("residual", [False, True])
def test_forward_many_rows(P, ctx, dtype, out, rows, hidden, residual):
    dt = T[dtype]
    x = randn(rows, hidden, seed=80, dtype=dt)
    res = randn(rows, hidden, seed=81, dtype=dt) if residual else None
    w = randn(hidden, seed=82, dtype=dt)
    y = torch.empty(rows, hidden, device="cuda", dtype=torch.float8_e4m3fn if out == 2 else dt)
    tot = torch.empty_like(x)
    scales = torch.empty(rows, device="cuda") if out == 2 else None
    P.purlin_rms_norm(ctx, x, w, y, rows, hidden, EPS, dtype, out, residual=res, total=tot,
                      scales=scales)
    P.purlin_check(ctx)
    t64, v64 = forward64(x, res, w)
    assert_close(tot, t64, 2 * U)
    if out != 2:
        assert_close(y, v64, slack(hidden) * 1.01)
        return
    want = (v64.abs().amax(1) / 448).clamp_min(2.0 ** -126)
    assert_close(scales, want, (slack(hidden) + 4 * U) * 1.01)
    q64 = v64 / want[:, None]
    bound = torch.maximum(q64.abs() * 2.0 ** -4, torch.full_like(q64, 2.0 ** -10))
    bound = bound + q64.abs() * 2 * (slack(hidden) + 4 * U)
    assert bool(((y.float().double() - q64).abs() <= bound * 1.01).all())


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", MANY)
@pytest.mark.parametrize("stream_grad", [False, True], ids=["plain", "dtotal"])
def test_backward_many_rows(P, ctx, dtype, rows, hidden, stream_grad):
    test_backward(P, ctx, dtype, rows, hidden, stream_grad)


def test_many_rows_in_place_and_offset(P, ctx):
    """Views that start in the middle of a window, rows enough to be staged, and
    results over the inputs: a block fetches rows ahead of the ones it writes."""
    rows, hidden, off = 1500, 4099, 5
    bufs = [torch.empty(rows * hidden + 16, device="cuda", dtype=torch.bfloat16)
            for _ in range(3)]
    x, res, dy = (b[off:off + rows * hidden].view(rows, hidden) for b in bufs)
    for k, t in enumerate((x, res, dy)):
        t.copy_(randn(rows, hidden, seed=90 + k, dtype=torch.bfloat16))
    w = randn(hidden + 3, seed=93, dtype=torch.bfloat16)[3:]
    t64, v64 = forward64(x, res, w)
    P.purlin_rms_norm(ctx, x, w, x, rows, hidden, EPS, 1, residual=res, total=res)
    P.purlin_check(ctx)
    assert_close(x, v64, slack(hidden) * 1.01)
    assert_close(res, t64, 2 * U)
    dx64, dw64 = backward64(res, dy, w, x)
    g, td = (dy.double() * w.double()).abs(), res.double().abs()
    r = 1 / torch.sqrt(res.double().square().mean(1, keepdim=True) + EPS)
    scale = r * (g + td * r * r * (g * td).mean(1, keepdim=True)) + x.double().abs()
    size = (dy.double() * res.double() * r).abs().sum(0)
    dw = torch.empty(hidden, device="cuda")
    P.purlin_rms_norm_backward(ctx, dy, res, w, dy, dw, rows, hidden, EPS, 1, dtotal=x)
    P.purlin_check(ctx)
    assert_rounds(dy, dx64, 4 * slack(hidden) * scale + 1e-37)
    assert bool(((dw.double() - dw64).abs() <= (rows * U + 2 * slack(hidden)) * size + 1e-37).all())
