"""Products by CTA pairs whose tiles are too few for the pairs: K runs, partial
accumulators of both CTAs of a pair, and their join.

The plan that a launch makes on the device is computed here once more (for the 152
SMs of a GB300), so that the cases are known to be what they stand for: a CPU test
checks that each selects pairs, cuts its tiles into runs, and that the runs of a tile
cover its K blocks in order with a slot of their own.  On the GPU the sums are of small
whole numbers, exact in any order, and compared bit for bit.
"""
import math

import pytest

torch = pytest.importorskip("torch")

SMS, JOIN, MOST_COST = 152, 12, 48


def block_cost(nj):
    return 16 + (nj + 7) // 8


def plan(mode, counts, rows, k, n, bk):
    """(pairs?, K runs or None, [(blocks, nj, runs of the tile)])."""
    ni = k if mode == "grad" else n
    wide, narrow = (ni + 255) // 256 * 2, (ni + 127) // 128
    cg = 2 if float(rows) * n * k >= 8e9 and 8 * wide <= 9 * narrow else 1
    ctas, i_tiles = SMS // cg, -(-ni // (128 * cg))
    width, least = 32, None
    if mode == "grad" or max(counts) > 32:
        for w in range(256, 0, -32):   # the wider of two equal ones
            down = -(-n // w) * len(counts) if mode == "grad" else sum(-(-c // w) for c in counts)
            even = down * i_tiles / ctas
            blocks = max(1.0, sum(counts) / (bk * len(counts))) if mode == "grad" else -(-k // bk)
            cost = (math.ceil(even) * blocks if even >= 1 else min(blocks, even * blocks + JOIN)) * \
                max(2.0 * w, (16384 + w * 128 / cg) / 65) + 12 * w
            if least is None or cost < least * (1 - 1e-6):
                width, least = w, cost
    tiles = []
    for c in counts:
        tall = n if mode == "grad" else c
        blocks = max(1, -(-(c if mode == "grad" else k) // bk))
        for j in range(0, tall, width):
            tiles += [(blocks, min(width, tall - j))] * i_tiles
    units = [(b, block_cost(nj)) for b, nj in tiles]
    spent = sum(b * u for b, u in units)
    idle = ctas - len(tiles)
    if not tiles or idle <= 0 or idle * spent < JOIN * ctas * block_cost(width) * len(tiles):
        return cg == 2, None, [(b, nj, 1) for b, nj in tiles]
    runs = max(1, min(ctas, spent // (4 * MOST_COST)))
    begin = [spent * r // runs for r in range(runs + 1)]
    at, out, slots = 0, [], set()
    for (blocks, nj), (_, u) in zip(tiles, units):
        mine = [(r, max(0, -(-(begin[r] - at) // u)), min(blocks, -(-(begin[r + 1] - at) // u)))
                for r in range(runs) if begin[r] < at + blocks * u and begin[r + 1] > at]
        mine = [m for m in mine if m[1] < m[2]]
        assert [m[1] for m in mine[1:]] == [m[2] for m in mine[:-1]]
        assert mine[0][1] == 0 and mine[-1][2] == blocks
        assert [m[0] for m in mine] == list(range(mine[0][0], mine[0][0] + len(mine)))
        if len(mine) > 1:
            for r, _, _ in mine:
                slot = 2 * r + (1 if r == mine[0][0] and begin[r] < at else 0)
                assert slot not in slots and slot * cg + cg - 1 < 2 * SMS
                slots.add(slot)
        out.append((blocks, nj, len(mine)))
        at += blocks * u
    return cg == 2, runs, out


# mode, counts, rows of each group's place (0: packed), k, n.  Ragged and empty groups,
# capacity buffers with few real rows, K blocks that end anywhere, row counts of the
# weight gradient that are no multiple of 16 (cut stages inside a pair's runs)
CASES = {
    "nk one group": ("nk", [512], 0, 8192, 2048),
    "nk ragged": ("nk", [300, 0, 17, 195], 0, 8200, 2047),
    "nk capacity": ("nk", [3, 0, 0, 9, 1, 0, 7, 0], 600, 2560, 1024),
    "nk few tiles": ("nk", [250], 600, 16384, 1024),
    "kn one group": ("kn", [511], 0, 8192, 2048),
    "kn ragged": ("kn", [0, 130, 5, 260], 300, 7001, 1160),
    "e4m3 one group": ("e4m3", [500], 0, 8192, 2048),
    "e4m3 capacity": ("e4m3", [33, 0, 1, 64], 300, 8208, 1023),
    "grad one group": ("grad", [4101], 0, 2048, 1000),
    "grad ragged": ("grad", [9001, 0, 18000, 15], 18005, 1001, 240),
    "grad capacity": ("grad", [6007, 3], 35000, 1024, 128),
}


def laid_out(counts, cap):
    if cap:
        return [g * cap for g in range(len(counts))], cap * len(counts)
    return [sum(counts[:g]) for g in range(len(counts))], sum(counts)


@pytest.mark.parametrize("case", CASES.values(), ids=CASES.keys())
def test_the_cases_are_pairs_with_runs(case):
    mode, counts, cap, k, n = case
    rows = laid_out(counts, cap)[1]
    pairs, runs, tiles = plan(mode, counts, rows, k, n, 128 if mode == "e4m3" else 64)
    assert pairs and runs is not None and runs > 1
    assert any(shared > 1 for _, _, shared in tiles)


def test_some_tiles_have_many_runs_and_some_blocks_are_cut():
    most = max(t[2] for mode, counts, cap, k, n in CASES.values()
               for t in plan(mode, counts, laid_out(counts, cap)[1], k, n, 64)[2])
    assert most >= 8
    assert all(any(c % 16 for c in counts) for mode, counts, *_ in CASES.values() if mode == "grad")


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


def whole(shape, dtype, seed, inside=None):
    """Whole numbers in rows of a 16-byte pitch; padding, and rows outside the
    groups, hold NaN."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    ld = (shape[-1] + per - 1) // per * per
    buf = torch.full((*shape[:-1], ld), math.nan, device="cuda").to(dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf[..., :shape[-1]] = torch.randint(-3, 4, shape, device="cuda", generator=g).to(dtype)
    if inside is not None:
        buf[~inside] = torch.full((1,), math.nan, device="cuda").to(dtype)
    return buf[..., :shape[-1]]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES.values(), ids=CASES.keys())
def test_pairs_with_runs(P, ctx, case):
    mode, counts, cap, k, n = case
    begin, rows = laid_out(counts, cap)
    groups = len(counts)
    inside = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for b, c in zip(begin, counts):
        inside[b:b + c] = True
    b64, c64 = (torch.tensor(v, device="cuda", dtype=torch.int64) for v in (begin, counts))
    dt = torch.float8_e4m3fn if mode == "e4m3" else torch.bfloat16
    x = whole((rows, k), dt, 1, inside)
    if mode == "grad":
        dy = whole((rows, n), dt, 2, inside)
        out = torch.full((groups * n + 1, k + 3), 7.0, device="cuda", dtype=torch.bfloat16)
        want = out.clone()
        for g, (b, c) in enumerate(zip(begin, counts)):
            m = dy[b:b + c].double().t() @ x[b:b + c].double()
            want[g * n:(g + 1) * n, :k] = m.float().bfloat16()

        def call():
            P.purlin_grouped_matmul_weight_grad(ctx, dy, x, out, b64, c64, groups, rows, n, k,
                                                P.PURLIN_BF16, lddy=dy.stride(0),
                                                ldx=x.stride(0), lddw=k + 3)
    else:
        w = whole((groups, k, n) if mode == "kn" else (groups, n, k), dt, 2)
        xs = ws = None
        if mode == "e4m3":
            xs = torch.full((rows,), math.nan, device="cuda")
            xs[inside] = torch.exp2(torch.arange(int(inside.sum()), device="cuda") % 5 - 2.0)
            ws = torch.exp2(torch.arange(groups * n, device="cuda").view(groups, n) % 7 - 3.0)
        out = torch.full((rows + 1, n + 5), 7.0, device="cuda", dtype=torch.bfloat16)
        want = out.clone()
        for g, (b, c) in enumerate(zip(begin, counts)):
            m = w[g].float().double()
            y = x[b:b + c].float().double() @ (m if mode == "kn" else m.t())
            if xs is not None:
                y = y * xs[b:b + c].double()[:, None] * ws[g].double()[None, :]
            want[b:b + c, :n] = y.float().bfloat16()

        def call():
            P.purlin_grouped_matmul(ctx, x, w, out, b64, c64, groups, rows, n, k,
                                    P.PURLIN_E4M3 if mode == "e4m3" else P.PURLIN_BF16,
                                    P.PURLIN_WEIGHTS_KN if mode == "kn" else P.PURLIN_WEIGHTS_NK,
                                    x_scales=xs, w_scales=ws, ldx=x.stride(0), ldw=w.stride(1),
                                    ldy=n + 5)

    # twice in a row, and again behind a small product that shares the join's counters
    for turn in range(3):
        if turn == 2:
            one = torch.ones(4, 4096, device="cuda", dtype=torch.bfloat16)
            y1 = torch.empty(4, 128, device="cuda", dtype=torch.bfloat16)
            P.purlin_grouped_matmul(ctx, one, one[:1].expand(128, 4096).contiguous(), y1,
                                    torch.zeros(1, device="cuda").long(),
                                    torch.full((1,), 4, device="cuda"), 1, 4, 128, 4096,
                                    P.PURLIN_BF16)
            P.purlin_check(ctx)
            assert bool((y1 == 4096).all())
        out.fill_(7.0)
        call()
        P.purlin_check(ctx)
        assert torch.equal(out, want)
