"""The norm's quotients on a GPU: e4m3 values are v / scale and means are
sum / hidden, as stated, not products with a reciprocal.

Rows of +-1 with eps 0 have a mean square of exactly 1, so v is the weight (or
minus it) and the quotient can be computed on the host bit for bit.  The weights
are picked so that v / scale lies on, or within an ulp of, a tie between two e4m3
values and v * (1 / scale) falls on its other side.  Rows of small whole numbers
have exact sums in any order: every kernel of the norm gives them the same bits.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

F = np.float32


def e4m3(v):
    return torch.from_numpy(np.asarray(v, F)).to(torch.float8_e4m3fn).float().numpy()


def telling_weights(dtype, most):
    """Weights w, and whether the quotient and the reciprocal's product with
    `most` as the largest |w| round to different e4m3 values."""
    scale = F(F(most) / F(448))
    ties = np.concatenate([np.arange(17, 32, 2) * 2.0 ** e for e in range(-6, 5)])
    ties = ties[ties < 440]
    if dtype == "f32":
        w = (ties.astype(F) * scale).astype(F)
        w = np.concatenate([w + k * np.spacing(w) for k in range(-4, 5)]).astype(F)
    else:   # every bf16 value below the largest
        bits = np.arange(0x3000, 0x4380, dtype=np.uint32) << 16
        w = bits.view(F)
        w = w[w < most]
    q, p = e4m3(w / scale), e4m3(w * F(F(1) / scale))
    return w[q != p]


def weights(dtype, hidden):
    """hidden weights, the largest first; all the others tell the two apart."""
    rng = np.random.default_rng(hidden)
    best, most = np.empty(0, F), 0.0
    for k in range(400):
        m = F(1 + rng.random()) if dtype == "f32" else F((128 + k % 128) * 2.0 ** (k // 128))
        w = telling_weights(dtype, m)
        if len(w) > len(best):
            best, most = w, m
    assert len(best) >= 2
    return np.concatenate([[most], np.resize(best, hidden - 1)]).astype(F)


def test_the_weights_tell_quotients_from_products():
    for dtype in ("f32", "bf16"):
        w = weights(dtype, 64)
        scale = F(w[0] / F(448))
        assert bool((e4m3(w / scale)[1:] != e4m3(w * F(F(1) / scale))[1:]).all())
        if dtype == "bf16":
            t = torch.from_numpy(w)
            assert torch.equal(t.bfloat16().float(), t)


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


# a warp a row, a block a row, rows through shared memory with and without edges,
# rows past the registers
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,hidden", [(3, 8), (900, 264), (5, 1021), (3, 4096), (900, 2048),
                                         (900, 2051), (400, 7168), (2, 40000)])
def test_e4m3_values_are_quotients(P, ctx, dtype, rows, hidden):
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    w = weights(dtype, hidden)
    g = torch.Generator().manual_seed(rows)
    x = torch.randint(0, 2, (rows, hidden), generator=g).float() * 2 - 1
    y = torch.empty(rows, hidden, device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty(rows, device="cuda")
    P.purlin_rms_norm(ctx, x.cuda().to(dt), torch.from_numpy(w).cuda().to(dt), y, rows, hidden,
                      0.0, 0 if dtype == "f32" else 1, P.PURLIN_E4M3, scales=scales)
    P.purlin_check(ctx)
    scale = F(w[0] / F(448))
    assert bool((scales == float(scale)).all())
    want = torch.from_numpy(e4m3(w / scale)) * x
    assert torch.equal(y.float().cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,hidden", [(3, 264), (900, 2048), (2, 40000)])
def test_tiny_and_infinite_scales(P, ctx, rows, hidden):
    """Quotients near the smallest normal scale, where a remainder would vanish;
    an infinite scale leaves finite values zero."""
    w = weights("f32", hidden)
    x = torch.ones(rows, hidden, device="cuda")
    y = torch.empty(rows, hidden, device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty(rows, device="cuda")

    def norm(weight):
        P.purlin_rms_norm(ctx, x, torch.from_numpy(weight).cuda(), y, rows, hidden, 0.0, 0,
                          P.PURLIN_E4M3, scales=scales)
        P.purlin_check(ctx)
        return y.float().cpu(), scales.cpu()

    scale = F(w[0] / F(448))
    for power in (-115, -90, -70, 100):
        p = F(2.0) ** F(power)
        got, s = norm((w * p).astype(F))
        assert bool((s == float(scale * p)).all())
        assert torch.equal(got, torch.from_numpy(e4m3(w / scale)).expand(rows, hidden))
    x *= 2
    x[:, 1::2] = 0.125          # mean square just above 2: the root is below 1
    big = np.ones(hidden, F)
    big[0] = 3.4e38
    got, s = norm(big)          # 2 / root(2) times 3.4e38: past the largest value
    assert bool(s.isinf().all())
    assert bool(got[:, 0].isnan().all()) and bool((got[:, 1:] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,hidden", [(3, 264), (3, 1021), (900, 2048), (2, 40000)])
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-5])
def test_zero_rows(P, ctx, rows, hidden, eps):
    """0 / root(0 + eps): zeros, or NaN without an eps, as the formula has it."""
    x, w = torch.zeros(rows, hidden, device="cuda"), torch.ones(hidden, device="cuda")
    y, scales = torch.empty_like(x), torch.empty(rows, device="cuda")
    q = torch.empty(rows, hidden, device="cuda", dtype=torch.float8_e4m3fn)
    P.purlin_rms_norm(ctx, x, w, y, rows, hidden, eps, 0)
    P.purlin_rms_norm(ctx, x, w, q, rows, hidden, eps, 0, P.PURLIN_E4M3, scales=scales)
    P.purlin_check(ctx)
    for t in (y, q.float()):
        assert bool((t.isnan() if eps == 0 else t == 0).all())
    assert bool((scales == 2.0 ** -126).all())


# hidden sizes whose binary32 reciprocal is not exact; few rows and many
@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [1100, 1101, 2052, 4099, 7168])
@pytest.mark.parametrize("out", [0, 2], ids=["f32", "e4m3"])
def test_rows_have_the_same_bits_among_few_and_many(P, ctx, hidden, out):
    rows = 1600
    g = torch.Generator(device="cuda").manual_seed(hidden)
    x = torch.randint(-3, 4, (rows, hidden), device="cuda", generator=g).float()
    w = torch.randint(1, 5, (hidden,), device="cuda", generator=g).float()
    kind = torch.float8_e4m3fn if out else torch.float32

    def norm(n):
        y = torch.empty(n, hidden, device="cuda", dtype=kind)
        scales = torch.empty(n, device="cuda") if out else None
        P.purlin_rms_norm(ctx, x, w, y, n, hidden, 0.0, 0, out, scales=scales)
        P.purlin_check(ctx)
        return y.float(), scales

    few, many = norm(5), norm(rows)
    assert torch.equal(few[0], many[0][:5])
    if out:
        assert torch.equal(few[1], many[1][:5])
    r = (x.square().sum(1, keepdim=True).cpu() / hidden).cuda().rsqrt()
    if not out:   # the same quotient and root on the host's side
        assert torch.equal(many[0], x * r * w)


@pytest.mark.gpu
@pytest.mark.parametrize("hidden", [1100, 1101, 2052, 4099])
def test_gradients_have_the_same_bits_among_few_and_many(P, ctx, hidden):
    rows = 1600
    g = torch.Generator(device="cuda").manual_seed(hidden)
    t, dy = (torch.randint(-3, 4, (rows, hidden), device="cuda", generator=g).float()
             for _ in range(2))
    w = torch.randint(1, 5, (hidden,), device="cuda", generator=g).float()

    def gradient(n):
        dx, dw = torch.empty(n, hidden, device="cuda"), torch.empty(hidden, device="cuda")
        P.purlin_rms_norm_backward(ctx, dy, t, w, dx, dw, n, hidden, 0.0, 0)
        P.purlin_check(ctx)
        return dx

    assert torch.equal(gradient(5), gradient(rows)[:5])
