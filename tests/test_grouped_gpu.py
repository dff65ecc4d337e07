"""The products grouped by expert on a GPU.

Most cases use small whole numbers, whose binary32 sums are exact in any
order: the result is the 64-bit sum rounded once, compared bit for bit.  Cases
with real values are held to K additions of binary32 (each off by at most 2^-23
of the sum of absolute products, truncation included); the bf16 output then lies
between the roundings of that interval's two ends.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


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


def pitch(cols, dtype):
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return (cols + per - 1) // per * per


def fill(shape, dtype, seed, whole, pad=0, junk=math.nan):
    """A matrix (or a stack) in a pitched buffer whose padding holds junk."""
    ld = pitch(shape[-1], dtype) + pad
    buf = torch.full((*shape[:-1], ld), junk, device="cuda").to(dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)
    if whole:
        v = torch.randint(-4, 5, shape, device="cuda", generator=g).float()
    else:
        v = torch.randn(shape, device="cuda", generator=g)
    buf[..., :shape[-1]] = v.to(dtype)
    return buf[..., :shape[-1]]


def assert_rounds(got, want, err):
    """got is the rounding of some value within err of want (rounding is monotone)."""
    assert bool(((got >= (want - err).to(BF16)) & (got <= (want + err).to(BF16))).all())


def i64(v):
    return torch.tensor(v, device="cuda", dtype=torch.int64)


def packed(counts):
    return [sum(counts[:g]) for g in range(len(counts))], sum(counts)


def padded(counts, cap):
    return [g * cap for g in range(len(counts))], cap * len(counts)


def product(P, ctx, x, w, begin, count, layout=0, xs=None, ws=None, ldy_pad=0, guard=7.0):
    groups = w.shape[0]
    n = w.shape[1] if layout == 0 else w.shape[2]
    k = x.shape[1]
    buf = torch.full((x.shape[0] + 1, n + ldy_pad), guard, device="cuda", dtype=BF16)
    P.purlin_grouped_matmul(ctx, x, w, buf, i64(begin), i64(count), groups, x.shape[0], n, k,
                            P.PURLIN_BF16 if x.dtype == BF16 else P.PURLIN_E4M3, layout,
                            x_scales=xs, w_scales=ws, ldx=x.stride(0), ldw=w.stride(1),
                            ldy=n + ldy_pad)
    P.purlin_check(ctx)
    return buf


def expected(x, w, begin, count, layout, xs=None, ws=None, n=None, ldy_pad=0, guard=7.0):
    n = w.shape[1] if layout == 0 else w.shape[2]
    out = torch.full((x.shape[0] + 1, n + ldy_pad), guard, device="cuda", dtype=BF16)
    for g, (b, c) in enumerate(zip(begin, count)):
        a = x[b:b + c].float().double()
        m = w[g].float().double()
        y = a @ (m.t() if layout == 0 else m)
        if xs is not None:
            y = y * xs[b:b + c].double()[:, None] * ws[g].double()[None, :]
        out[b:b + c, :n] = y.to(torch.float32).to(BF16)
    return out


# counts: single tokens, empty groups at either end and between, ragged tiles, one
# group alone, more than one tile of rows
COUNTS = [[1], [0, 1, 0], [5, 0, 3, 0], [16, 17, 15], [64, 63, 65, 1], [0, 0], [129, 257, 31],
          [300, 2, 0, 700], [1] * 37]
SIZES = [(8, 8), (1, 1), (7, 33), (64, 64), (128, 128), (130, 70), (257, 129), (64, 515),
         (512, 200), (1030, 264)]


@pytest.mark.parametrize("layout", [0, 1], ids=["nk", "kn"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "c" + "_".join(map(str, c[:4])))
@pytest.mark.parametrize("k,n", SIZES)
def test_whole_numbers_bf16(P, ctx, layout, counts, k, n):
    begin, rows = packed(counts)
    rows = max(rows, 1)
    x = fill((rows, k), BF16, 1, True)
    w = fill((len(counts), n, k) if layout == 0 else (len(counts), k, n), BF16, 2, True)
    got = product(P, ctx, x, w, begin, counts, layout, ldy_pad=3)
    assert torch.equal(got, expected(x, w, begin, counts, layout, ldy_pad=3))


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "c" + "_".join(map(str, c[:4])))
@pytest.mark.parametrize("k,n", SIZES)
def test_whole_numbers_e4m3(P, ctx, counts, k, n):
    begin, rows = packed(counts)
    rows = max(rows, 1)
    x = fill((rows, k), E4M3, 3, True)
    w = fill((len(counts), n, k), E4M3, 4, True)
    g = torch.Generator(device="cuda").manual_seed(5)
    xs = torch.exp2(torch.randint(-3, 4, (rows,), device="cuda", generator=g).float())
    ws = torch.exp2(torch.randint(-3, 4, (len(counts), n), device="cuda", generator=g).float())
    got = product(P, ctx, x, w, begin, counts, 0, xs, ws, ldy_pad=3)
    assert torch.equal(got, expected(x, w, begin, counts, 0, xs, ws, ldy_pad=3))


@pytest.mark.parametrize("dtype", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("counts", [[3, 0, 40, 17], [130, 1, 260]],
                         ids=["small", "tiles"])
def test_rows_of_no_group_do_not_matter(P, ctx, dtype, counts):
    """Capacity-padded groups in any order; rows between them hold NaN."""
    k, n, cap = 200, 150, 300
    begin, rows = padded(counts, cap)
    begin = begin[::-1]
    x = fill((rows, k), dtype, 6, True, pad=16)
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for b, c in zip(begin, counts):
        inside[b:b + c] = True
    x[~inside] = torch.full((1,), math.nan, device="cuda").to(dtype)
    w = fill((len(counts), n, k), dtype, 7, True, pad=32)
    xs = ws = None
    if dtype == E4M3:
        xs = torch.full((rows,), math.nan, device="cuda")
        xs[inside] = 0.5
        ws = torch.full((len(counts), n), 2.0, device="cuda")
    got = product(P, ctx, x, w, begin, counts, 0, xs, ws)
    assert torch.equal(got, expected(x, w, begin, counts, 0, xs, ws))


def test_special_values_stay_in_their_rows(P, ctx):
    counts, k, n = [20, 20], 96, 40
    begin, rows = packed(counts)
    x = fill((rows, k), BF16, 8, True)
    w = fill((2, n, k), BF16, 9, True)
    x[3, 5] = math.nan
    x[30, 90] = math.inf
    w[0, 7, 11] = math.inf
    x[:20, 11] = 1                       # no 0 * inf for the rows of group 0
    w[1, :, 90] = 1
    got = product(P, ctx, x, w, begin, counts)
    want = expected(x, w, begin, counts, 0)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(1.0), want.nan_to_num(1.0))
    assert bool(got[3, :n].isnan().all()) and bool((got[30, :n] == math.inf).all())
    assert int(got[:rows].isnan().sum()) == n


@pytest.mark.parametrize("dtype,layout", [(BF16, 0), (BF16, 1), (E4M3, 0)],
                         ids=["nk", "kn", "e4m3"])
@pytest.mark.parametrize("counts,k,n", [([8], 7168, 256), ([700, 0, 90], 2048, 515),
                                        ([1, 2, 3], 4000, 4096)])
def test_real_values(P, ctx, dtype, layout, counts, k, n):
    begin, rows = packed(counts)
    x = fill((rows, k), dtype, 10, False)
    w = fill((len(counts), n, k) if layout == 0 else (len(counts), k, n), dtype, 11, False)
    xs = ws = None
    if dtype == E4M3:
        xs = torch.rand(rows, device="cuda") + 0.5
        ws = torch.rand(len(counts), n, device="cuda") + 0.5
    got = product(P, ctx, x, w, begin, counts, layout, xs, ws)
    for g, (b, c) in enumerate(zip(begin, counts)):
        a, m = x[b:b + c].float().double(), w[g].float().double()
        m = m.t() if layout == 0 else m
        y, size = a @ m, a.abs() @ m.abs()
        if xs is not None:
            s = xs[b:b + c].double()[:, None] * ws[g].double()[None, :]
            y, size = y * s, size * s
        assert_rounds(got[b:b + c], y, (k + 4) * 2.0 ** -23 * size)
    again = product(P, ctx, x, w, begin, counts, layout, xs, ws)
    assert torch.equal(again, got)            # the same bits every time


def weight_grad(P, ctx, dy, x, begin, count, ld_pad=0, guard=7.0):
    n, k, groups = dy.shape[1], x.shape[1], len(count)
    buf = torch.full((groups * n + 1, k + ld_pad), guard, device="cuda", dtype=BF16)
    P.purlin_grouped_matmul_weight_grad(ctx, dy, x, buf, i64(begin), i64(count), groups,
                                        x.shape[0], n, k, P.PURLIN_BF16, lddy=dy.stride(0),
                                        ldx=x.stride(0), lddw=k + ld_pad)
    P.purlin_check(ctx)
    return buf


def expected_grad(dy, x, begin, count, ld_pad=0, guard=7.0):
    n, k = dy.shape[1], x.shape[1]
    out = torch.full((len(count) * n + 1, k + ld_pad), guard, device="cuda", dtype=BF16)
    for g, (b, c) in enumerate(zip(begin, count)):
        m = dy[b:b + c].double().t() @ x[b:b + c].double()
        out[g * n:(g + 1) * n, :k] = m.to(torch.float32).to(BF16)
    return out


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "c" + "_".join(map(str, c[:4])))
@pytest.mark.parametrize("k,n", SIZES)
def test_weight_grad_whole_numbers(P, ctx, counts, k, n):
    begin, rows = packed(counts)
    rows = max(rows, 1)
    dy = fill((rows, n), BF16, 12, True)
    x = fill((rows, k), BF16, 13, True)
    got = weight_grad(P, ctx, dy, x, begin, counts, ld_pad=5)
    assert torch.equal(got, expected_grad(dy, x, begin, counts, ld_pad=5))


@pytest.mark.parametrize("counts", [[3, 0, 40, 17], [130, 1, 260], [64, 128, 256], [15, 16, 33]])
def test_weight_grad_ignores_rows_of_no_group(P, ctx, counts):
    k, n, cap = 200, 150, 300
    begin, rows = padded(counts, cap)
    dy, x = fill((rows, n), BF16, 14, True, pad=8), fill((rows, k), BF16, 15, True, pad=24)
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for b, c in zip(begin, counts):
        inside[b:b + c] = True
    dy[~inside] = math.nan
    x[~inside] = math.inf
    got = weight_grad(P, ctx, dy, x, begin, counts)
    assert torch.equal(got, expected_grad(dy, x, begin, counts))


@pytest.mark.parametrize("counts,k,n", [([5000, 0, 133], 300, 264), ([2, 1, 70], 1000, 1040)])
def test_weight_grad_real_values(P, ctx, counts, k, n):
    begin, rows = packed(counts)
    dy, x = fill((rows, n), BF16, 16, False), fill((rows, k), BF16, 17, False)
    got = weight_grad(P, ctx, dy, x, begin, counts)
    for g, (b, c) in enumerate(zip(begin, counts)):
        a, m = dy[b:b + c].double().t(), x[b:b + c].double()
        y, size = a @ m, a.abs() @ m.abs()
        assert_rounds(got[g * n:(g + 1) * n], y, (c + 4) * 2.0 ** -23 * size)
    assert torch.equal(weight_grad(P, ctx, dy, x, begin, counts), got)


def test_gradients_against_differences(P, ctx):
    """The product is linear in x and in w: differences of the 64-bit loss
    sum(dy * y) by whole steps give the gradients exactly."""
    counts, k, n = [3, 0, 5], 24, 16
    begin, rows = packed(counts)
    x, dy = fill((rows, k), BF16, 18, True), fill((rows, n), BF16, 19, True)
    w = fill((3, n, k), BF16, 20, True)
    dx = product(P, ctx, dy, w, begin, counts, 1)[:rows]
    dw = weight_grad(P, ctx, dy, x, begin, counts)[:3 * n].view(3, n, k)

    def loss(xx, ww):
        return sum(float((dy[b:b + c].double() * (xx[b:b + c] @ ww[g].t())).sum())
                   for g, (b, c) in enumerate(zip(begin, counts)))

    x64, w64 = x.double(), w.double()
    base = loss(x64, w64)
    for i in range(rows):
        for j in range(0, k, 5):
            e = x64.clone()
            e[i, j] += 1
            assert loss(e, w64) - base == float(dx[i, j])
    for g in range(3):
        for i in range(0, n, 3):
            for j in range(0, k, 7):
                e = w64.clone()
                e[g, i, j] += 1
                assert loss(x64, e) - base == float(dw[g, i, j])


@pytest.mark.parametrize("begin,count", [([0, 4], [4, 7]), ([0, -1], [4, 2]), ([0, 4], [-1, 2]),
                                         ([0, 1 << 62], [1, 1 << 62]), ([0, 0], [9, 9]),
                                         ([0, 11], [1, 0])])
def test_bad_groups_write_nothing(P, ctx, begin, count):
    rows, k, n = 10, 64, 32
    x = torch.ones(rows, k, device="cuda", dtype=BF16)
    w = torch.ones(2, n, k, device="cuda", dtype=BF16)
    y = torch.full((rows, n), 7.0, device="cuda", dtype=BF16)
    P.purlin_grouped_matmul(ctx, x, w, y, i64(begin), i64(count), 2, rows, n, k, P.PURLIN_BF16)
    assert P.purlin_check_status(ctx) == P.PURLIN_ERR_INVALID_ARG
    dw = torch.full((2, n, k), 7.0, device="cuda", dtype=BF16)
    P.purlin_grouped_matmul_weight_grad(ctx, y, x, dw, i64(begin), i64(count), 2, rows, n, k,
                                        P.PURLIN_BF16)
    assert P.purlin_check_status(ctx) == P.PURLIN_ERR_INVALID_ARG
    assert bool((y == 7).all()) and bool((dw == 7).all())
    good = product(P, ctx, x, w, [0, 4], [4, 6])          # the context stays usable
    assert bool((good[:rows] == k).all())


def test_nothing_to_do(P, ctx):
    dw = torch.full((2, 16, 24), 7.0, device="cuda", dtype=BF16)
    P.purlin_grouped_matmul(ctx, 0, 0, 0, 0, 0, 2, 0, 16, 24, P.PURLIN_BF16)
    P.purlin_grouped_matmul(ctx, 0, 0, 0, 0, 0, 0, 5, 16, 24, P.PURLIN_BF16)
    P.purlin_grouped_matmul_weight_grad(ctx, 0, 0, dw, 0, 0, 2, 0, 16, 20, P.PURLIN_BF16,
                                        lddw=24)
    P.purlin_check(ctx)
    assert bool((dw[:, :, :20] == 0).all()) and bool((dw[:, :, 20:] == 7).all())


def test_many_groups(P, ctx):
    groups, k, n = 1024, 64, 24
    g = torch.Generator().manual_seed(3)
    counts = torch.randint(0, 4, (groups,), generator=g).tolist()
    begin, rows = packed(counts)
    x, w = fill((rows, k), BF16, 21, True), fill((groups, n, k), BF16, 22, True)
    assert torch.equal(product(P, ctx, x, w, begin, counts), expected(x, w, begin, counts, 0))
    dy = fill((rows, n), BF16, 23, True)
    assert torch.equal(weight_grad(P, ctx, dy, x, begin, counts),
                       expected_grad(dy, x, begin, counts))


def test_offsets_past_32_bits(P, ctx):
    """x rows 2^31 elements apart, and weights of more than 2^32 bytes."""
    ld, k, n = (1 << 31) + 8, 128, 72
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 30 GB")
    buf = torch.empty(2 * ld + k, device="cuda", dtype=BF16)
    x = torch.as_strided(buf, (3, k), (ld, 1))
    x.copy_(fill((3, k), BF16, 24, True))
    w = fill((2, n, k), BF16, 25, True)
    assert torch.equal(product(P, ctx, x, w, [0, 1], [1, 2]), expected(x, w, [0, 1], [1, 2], 0))
    del buf, x
    wide = torch.zeros(3, n, 1 << 24, device="cuda", dtype=BF16)
    wide[:, :, :k] = fill((3, n, k), BF16, 26, True)
    w = wide[:, :, :k]
    x = fill((9, k), BF16, 27, True)
    assert torch.equal(product(P, ctx, x, w, [0, 4, 5], [4, 1, 4]),
                       expected(x, w, [0, 4, 5], [4, 1, 4], 0))


def test_graph_replay_with_counts_from_the_device(P):
    """Counts written on the device between replays: no host round trip."""
    s = torch.cuda.Stream()
    c = P.purlin_init(1, s)
    try:
        groups, cap, k, n = 4, 80, 264, 136
        w = fill((groups, n, k), BF16, 28, True)
        x = fill((groups * cap, k), BF16, 29, True)
        begin = i64([g * cap for g in range(groups)])
        count = i64([1, 2, 3, 4])
        y = torch.zeros(groups * cap, n, device="cuda", dtype=BF16)
        dw = torch.zeros(groups, n, k, device="cuda", dtype=BF16)
        torch.cuda.synchronize()

        def call():
            P.purlin_grouped_matmul(c, x, w, y, begin, count, groups, groups * cap, n, k,
                                    P.PURLIN_BF16, ldx=x.stride(0), ldw=w.stride(1))
            P.purlin_grouped_matmul_weight_grad(c, y, x, dw, begin, count, groups, groups * cap,
                                                n, k, P.PURLIN_BF16, ldx=x.stride(0))

        call()
        P.purlin_check(c)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        for counts in ([0, 80, 1, 17], [80, 0, 0, 0], [5, 6, 7, 8]):
            with torch.cuda.stream(s):
                count.copy_(i64(counts))
                y.fill_(7.0)
            s.synchronize()
            graph.replay()
            P.purlin_check(c)
            want = expected(x, w, begin.tolist(), counts, 0)[:-1]
            assert torch.equal(y, want)
            y0 = y.clone()
            assert torch.equal(dw.view(-1, k), expected_grad(y0, x, begin.tolist(), counts)[:-1])
    finally:
        c.close()


# Work enough for CTA pairs: rows x k x n of 8e9 and more, channels that fill 256.
# Ragged and empty groups, tiles a row past a width, K blocks that end anywhere.
PAIRS = [([1500, 0, 257, 1300], 1501, 2003), ([3, 2040, 513, 64, 1], 2056, 1792),
         ([17] * 40 + [2500], 1024, 2560)]


@pytest.mark.parametrize("layout", [0, 1], ids=["nk", "kn"])
@pytest.mark.parametrize("counts,k,n", PAIRS, ids=["odd", "ragged", "small groups"])
def test_pairs_whole_numbers(P, ctx, layout, counts, k, n):
    begin, rows = packed(counts)
    x = fill((rows, k), BF16, 30, True)
    w = fill((len(counts), n, k) if layout == 0 else (len(counts), k, n), BF16, 31, True)
    got = product(P, ctx, x, w, begin, counts, layout, ldy_pad=5)
    assert torch.equal(got, expected(x, w, begin, counts, layout, ldy_pad=5))


@pytest.mark.parametrize("counts,k,n", PAIRS, ids=["odd", "ragged", "small groups"])
def test_pairs_whole_numbers_e4m3(P, ctx, counts, k, n):
    begin, rows = padded(counts, max(counts) + 3)
    x = fill((rows, k), E4M3, 32, True)
    w = fill((len(counts), n, k), E4M3, 33, True)
    xs = torch.full((rows,), math.nan, device="cuda")
    for b, c in zip(begin, counts):
        xs[b:b + c] = torch.exp2(torch.arange(c, device="cuda") % 5 - 2.0)
    ws = torch.exp2(torch.arange(len(counts) * n, device="cuda").view(-1, n) % 7 - 3.0)
    got = product(P, ctx, x, w, begin, counts, 0, xs, ws)
    assert torch.equal(got, expected(x, w, begin, counts, 0, xs, ws))


@pytest.mark.parametrize("counts,k,n", PAIRS, ids=["odd", "ragged", "small groups"])
def test_pairs_weight_grad(P, ctx, counts, k, n):
    """Rows outside the groups hold NaN and infinities: a pair cuts its last
    stages in both CTAs."""
    begin, rows = padded(counts, max(counts) + 9)
    dy, x = fill((rows, n), BF16, 34, True), fill((rows, k), BF16, 35, True)
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for b, c in zip(begin, counts):
        inside[b:b + c] = True
    dy[~inside] = math.nan
    x[~inside] = math.inf
    got = weight_grad(P, ctx, dy, x, begin, counts)
    assert torch.equal(got, expected_grad(dy, x, begin, counts))
    assert torch.equal(weight_grad(P, ctx, dy, x, begin, counts), got)


def test_calls_in_a_row_on_one_stream(P, ctx):
    """Launches overlap the end of the one before: each reads what it wrote."""
    counts, k = [100, 0, 30, 200], 512
    begin, rows = packed(counts)
    x = fill((rows, k), BF16, 36, True)
    w = torch.zeros(4, k, k, device="cuda", dtype=BF16)
    perm = torch.randperm(k, generator=torch.Generator().manual_seed(1)).cuda()
    w[:, torch.arange(k, device="cuda"), perm] = 1        # y[:, j] = x[:, perm[j]]
    a, b = x.clone(), torch.empty_like(x)
    for _ in range(20):
        for s, d in ((a, b), (b, a)):
            P.purlin_grouped_matmul(ctx, s, w, d, i64(begin), i64(counts), 4, rows, k, k,
                                    P.PURLIN_BF16)
    P.purlin_check(ctx)
    want = x
    for _ in range(40):
        want = want[:, perm]
    assert torch.equal(a, want)
