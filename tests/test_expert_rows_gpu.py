"""The order of slots by expert, the rows' way to their places and back, and its
gradients on a GPU, against plain indexing.

Order and copies are exact.  The weighted sum of k rows and a shared one: each product
and sum is one fused rounding, so the error before the output's rounding is at most
k u times the sum of the absolute values of the terms, u = 2^-24.  A product's gradient
w dy has one rounding of its own.  dweights, a sum of `cols` products whose order is
not said: cols u times the sum of their absolute values bounds every order.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T = {0: torch.float32, 1: torch.bfloat16, 2: torch.float8_e4m3fn}
HALF = {0: 2.0 ** -24, 1: 2.0 ** -8}     # half a step, relative


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


def order_reference(chosen, groups, capacity):
    seen, rank, valid = [0] * groups, [], []
    for e in chosen:
        ok = 0 <= e < groups
        rank.append(seen[e] if ok else -1)
        if ok:
            seen[e] += 1
    if capacity:
        begin = [g * capacity for g in range(groups)]
        count = [min(c, capacity) for c in seen]
    else:
        begin, count = [sum(seen[:g]) for g in range(groups)], seen
    place = [begin[e] + r if 0 <= e < groups and (not capacity or r < capacity) else -1
             for e, r in zip(chosen, rank)]
    return place, begin, count


def run_order(P, ctx, chosen, groups, capacity):
    slots = chosen.numel()
    place = torch.full((slots + 2,), -9, device="cuda", dtype=torch.int32)
    begin = torch.full((groups + 2,), -9, device="cuda", dtype=torch.int64)
    count = torch.full((groups + 2,), -9, device="cuda", dtype=torch.int64)
    P.purlin_expert_order(ctx, chosen, place[1:], begin[1:], count[1:], slots, groups, capacity)
    P.purlin_check(ctx)
    for t, n in ((place, slots), (begin, groups), (count, groups)):
        t = t.tolist()
        assert t[0] == -9 and t[n + 1] == -9            # nothing before or behind
    return place[1:-1], begin[1:-1], count[1:-1]


@pytest.mark.parametrize("groups", [1, 2, 8, 60, 256, 257, 1000, 1024])
@pytest.mark.parametrize("slots", [1, 31, 32, 33, 255, 1024, 2048, 2049, 5000, 70001])
def test_order(P, ctx, slots, groups):
    g = torch.Generator().manual_seed(slots + groups)
    chosen = torch.randint(-1, groups + 1, (slots,), generator=g)      # some are nobody's
    skewed = (chosen.clamp(0, groups - 1) ** 2) // groups
    for c in (chosen, skewed, torch.full((slots,), groups - 1)):
        for capacity in (0, 1, max(1, slots // groups)):
            got = run_order(P, ctx, c.int().cuda(), groups, capacity)
            want = order_reference(c.tolist(), groups, capacity)
            for a, b in zip(got, want):
                assert a.tolist() == b


def test_order_of_more_slots_than_blocks_have_at_once(P, ctx):
    n = 2_000_003
    chosen = torch.randint(0, 64, (n,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    place, begin, count = run_order(P, ctx, chosen.int(), 64, 0)
    order = chosen.sort(stable=True).indices
    want = torch.empty_like(order)
    want[order] = torch.arange(n, device="cuda")
    assert torch.equal(place.long(), want)
    assert torch.equal(count, torch.bincount(chosen, minlength=64))
    assert torch.equal(begin, count.cumsum(0) - count)


def test_order_of_nothing(P, ctx):
    empty = torch.empty(0, device="cuda", dtype=torch.int32)
    begin, count = (torch.full((5,), 9, device="cuda", dtype=torch.int64) for _ in range(2))
    P.purlin_expert_order(ctx, empty, None, begin, count, 0, 5, 7)
    assert begin.tolist() == [0, 7, 14, 21, 28] and count.tolist() == [0] * 5
    place = torch.full((40,), 5, device="cuda", dtype=torch.int32)
    P.purlin_expert_order(ctx, torch.zeros_like(place), place, None, None, 40, 0, 0)
    assert place.tolist() == [-1] * 40
    P.purlin_expert_order(ctx, None, None, None, None, 0, 0, 0)


def test_order_is_captured_after_a_first_call(P):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = P.purlin_init(1, s)
        chosen = torch.randint(0, 100, (30000,), device="cuda").int()
        place = torch.empty_like(chosen)
        begin, count = (torch.empty(100, device="cuda", dtype=torch.int64) for _ in range(2))
        P.purlin_expert_order(c, chosen, place, begin, count, 30000, 100)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            P.purlin_expert_order(c, chosen, place, begin, count, 30000, 100)
        for seed in (1, 2):
            chosen.copy_(torch.randint(0, 100, (30000,), device="cuda",
                                       generator=torch.Generator(device="cuda").manual_seed(seed)))
            g.replay()
            s.synchronize()
            want = order_reference(chosen.tolist(), 100, 0)
            assert place.tolist() == want[0] and count.tolist() == want[2]
        c.close()


def places(tokens, k, rows, seed, share=0.8):
    """Distinct places, some slots without one, some numbers outside."""
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(max(rows, tokens * k), generator=g)[:tokens * k]
    perm = torch.where(perm < rows, perm, -1)
    drop = torch.rand(tokens * k, generator=g) > share
    outside = torch.where(torch.arange(tokens * k) % 2 == 0, -1, rows + 3)
    return torch.where(drop, outside, perm).view(tokens, k).int().cuda()


def matrix(rows, cols, dtype, seed, pitch=0, offset=0, fill=None):
    """A rows x cols view with guards around it: `pitch` more columns, from `offset` on."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.full((rows + 2, cols + pitch + offset), 7.0, device="cuda")
    if fill is None:
        t[1:rows + 1, offset:offset + cols] = torch.randn(rows, cols, device="cuda", generator=g)
    else:
        t[1:rows + 1, offset:offset + cols] = fill
    t = t.to(T[dtype])
    return t, t[1:rows + 1, offset:offset + cols]


def guards_stand(t, view, offset=0):
    g = t.float().clone()
    rows, cols = view.shape
    g[1:rows + 1, offset:offset + cols] = 7.0
    return bool((g == 7.0).all())


SHAPES = [(1, 1, 1, 3), (3, 2, 7, 5), (17, 8, 64, 136), (40, 3, 1021, 100), (9, 32, 130, 300),
          (5, 6, 4100, 33), (64, 4, 512, 256), (130, 1, 96, 131)]


@pytest.mark.parametrize("dtype", [0, 1, 2], ids=["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("tokens,k,cols,rows", SHAPES)
@pytest.mark.parametrize("pitch,offset", [(0, 0), (5, 0), (16, 16), (3, 1)])
def test_dispatch(P, ctx, tokens, k, cols, rows, dtype, pitch, offset):
    place = places(tokens, k, rows, tokens + cols)
    _, x = matrix(tokens, cols, dtype, 1, pitch, offset)
    t, out = matrix(rows, cols, dtype, 2, pitch, offset)
    want = out.float().clone()
    scales = torch.rand(tokens, device="cuda")
    out_scales = torch.full((rows + 1,), -5.0, device="cuda")
    want_scales = out_scales.clone()
    P.purlin_dispatch_rows(ctx, x, place, out, tokens, k, cols, rows, dtype, scales=scales,
                           out_scales=out_scales, ldx=x.stride(0), ldo=out.stride(0))
    P.purlin_check(ctx)
    for at in range(tokens):
        for p in place[at].tolist():
            if 0 <= p < rows:
                want[p] = x[at].float()
                want_scales[p] = scales[at]
    assert torch.equal(out.float(), want) and torch.equal(out_scales, want_scales)
    assert guards_stand(t, out, offset)


def combine64(rows, place, w, shared):
    n = rows.shape[0]
    real = (place >= 0) & (place < n)
    at = torch.where(real, place, 0).long()
    terms = rows.double()[at] * torch.where(real, w.double(), 0.0)[:, :, None]
    terms = torch.where(real[:, :, None], terms, 0.0)
    y, size = terms.sum(1), terms.abs().sum(1)
    if shared is not None:
        y, size = y + shared.double(), size + shared.double().abs()
    return y, size


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens,k,cols,rows", SHAPES)
@pytest.mark.parametrize("weighted,shared", [(True, False), (True, True), (False, False)])
@pytest.mark.parametrize("pitch,offset", [(0, 0), (8, 8), (3, 1)])
def test_combine(P, ctx, tokens, k, cols, rows, dtype, weighted, shared, pitch, offset):
    place = places(tokens, k, rows, tokens + cols)
    place[0] = -1                                    # a token that was dropped everywhere
    _, r = matrix(rows, cols, dtype, 3, pitch, offset)
    w = torch.randn(tokens, k, device="cuda") if weighted else None
    _, sh = matrix(tokens, cols, dtype, 4, pitch, offset) if shared else (None, None)
    t, y = matrix(tokens, cols, dtype, 5, pitch, offset)
    P.purlin_combine_rows(ctx, r, place, y, tokens, k, cols, rows, dtype, weights=w, shared=sh,
                          ldr=r.stride(0), lds=sh.stride(0) if shared else 0, ldy=y.stride(0))
    P.purlin_check(ctx)
    ones = torch.ones(tokens, k, device="cuda")
    want, size = combine64(r, place, w if weighted else ones, sh)
    err = size * (k + 1) * U
    assert bool(((y.double() - want).abs() <= err + (want.abs() + err) * HALF[dtype] + 1e-38).all())
    assert guards_stand(t, y, offset)
    if shared:      # in place of the shared rows
        P.purlin_combine_rows(ctx, r, place, sh, tokens, k, cols, rows, dtype, weights=w, shared=sh,
                              ldr=r.stride(0), lds=sh.stride(0), ldy=sh.stride(0))
        P.purlin_check(ctx)
        assert torch.equal(sh, y)
    else:
        assert not bool(y[0].any())


def test_combine_skips_rows_without_a_place(P, ctx):
    # weights of dropped slots and rows that nobody names may hold anything
    place = torch.tensor([[1, -1], [-1, -1], [5, 99]], device="cuda", dtype=torch.int32)
    r = torch.full((6, 40), float("nan"), device="cuda")
    r[1], r[5] = 2.0, 3.0
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 1.0], [1.0, float("nan")]], device="cuda")
    y = torch.empty(3, 40, device="cuda")
    P.purlin_combine_rows(ctx, r, place, y, 3, 2, 40, 6, 0, weights=w)
    P.purlin_check(ctx)
    assert y[:, 0].tolist() == [1.0, 0.0, 3.0] and torch.equal(y, y[:, :1].expand(3, 40))
    dy, d = torch.ones(3, 40, device="cuda"), torch.zeros_like(r)
    dw = torch.full((3, 2), 9.0, device="cuda")
    P.purlin_combine_rows_backward(ctx, dy, r, place, w, d, dw, 3, 2, 40, 6, 0)
    P.purlin_check(ctx)
    assert dw.tolist() == [[80.0, 0.0], [0.0, 0.0], [120.0, 0.0]]
    assert d[:, 0].tolist() == [0.0, 0.5, 0.0, 0.0, 0.0, 1.0]


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens,k,cols,rows", SHAPES + [(3, 5, 20000, 20)])
@pytest.mark.parametrize("pitch,offset", [(0, 0), (8, 8), (3, 1)])
def test_combine_backward(P, ctx, tokens, k, cols, rows, dtype, pitch, offset):
    place = places(tokens, k, rows, tokens + cols)
    _, dy = matrix(tokens, cols, dtype, 6, pitch, offset)
    _, r = matrix(rows, cols, dtype, 7, pitch, offset)
    w = torch.randn(tokens, k, device="cuda")
    t, d = matrix(rows, cols, dtype, 8, pitch, offset)
    before = d.clone()
    dw = torch.full((tokens, k), 9.0, device="cuda")
    P.purlin_combine_rows_backward(ctx, dy, r, place, w, d, dw, tokens, k, cols, rows, dtype,
                                   lddy=dy.stride(0), ldr=r.stride(0), lddr=d.stride(0))
    P.purlin_check(ctx)
    real = (place >= 0) & (place < rows)
    at = torch.where(real, place, 0).long()
    prod = r.double()[at] * dy.double()[:, None, :]
    want = torch.where(real, prod.sum(2), 0.0)
    assert bool(((dw.double() - want).abs() <= prod.abs().sum(2) * (cols + 1) * U * real).all())
    named = torch.zeros(rows, dtype=torch.bool, device="cuda")
    named[at[real]] = True
    assert torch.equal(d[~named], before[~named])
    full = (w.double()[:, :, None] * dy.double()[:, None, :])[real]
    got = d.double()[at[real]]
    assert bool(((got - full).abs() <= full.abs() * (U + HALF[dtype]) * 1.01 + 1e-38).all())
    assert guards_stand(t, d, offset)
    dw2 = torch.empty_like(dw)
    P.purlin_combine_rows_backward(ctx, dy, r, place, w, r, dw2, tokens, k, cols, rows, dtype,
                                   lddy=dy.stride(0), ldr=r.stride(0), lddr=r.stride(0))
    P.purlin_check(ctx)
    assert torch.equal(dw, dw2) and torch.equal(r[named], d[named])    # in place of the rows


def test_gradients_by_differences(P, ctx):
    """sum(c * y) is linear in rows and weights alike: a step's difference is the
    gradient, off by the sums' roundings alone."""
    place = torch.tensor([[2, 0], [1, -1]], device="cuda", dtype=torch.int32)
    g = torch.Generator(device="cuda").manual_seed(9)
    r, w, c = (torch.randint(-4, 5, s, device="cuda", generator=g).float() for s in ((3, 8), (2, 2), (2, 8)))

    def value(r, w):
        y = torch.empty(2, 8, device="cuda")
        P.purlin_combine_rows(ctx, r, place, y, 2, 2, 8, 3, 0, weights=w)
        P.purlin_check(ctx)
        return float((y * c).sum())           # small whole numbers: exact

    d, dw = torch.zeros_like(r), torch.empty_like(w)
    P.purlin_combine_rows_backward(ctx, c, r, place, w, d, dw, 2, 2, 8, 3, 0)
    P.purlin_check(ctx)
    base = value(r, w)
    for t, grad in ((r, d), (w, dw)):
        for i in range(t.numel()):
            step = t.clone()
            step.view(-1)[i] += 1
            moved = value(step, w) if t is r else value(r, step)
            assert moved - base == float(grad.view(-1)[i])


def test_dispatch_and_its_gradient_are_adjoint(P, ctx):
    place = places(50, 4, 180, 3)
    x, c = (torch.randint(-4, 5, s, device="cuda").float() for s in ((50, 33), (180, 33)))
    out, dx = torch.zeros(180, 33, device="cuda"), torch.empty(50, 33, device="cuda")
    P.purlin_dispatch_rows(ctx, x, place, out, 50, 4, 33, 180, 0)
    P.purlin_combine_rows(ctx, c, place, dx, 50, 4, 33, 180, 0)
    P.purlin_check(ctx)
    assert float((out * c).sum()) == float((x * dx).sum())


def test_nothing_to_do(P, ctx):
    place = torch.zeros(2, 2, device="cuda", dtype=torch.int32)
    w = torch.ones(2, 2, device="cuda")
    t = torch.ones(2, 8, device="cuda")
    P.purlin_dispatch_rows(ctx, t, place, None, 2, 2, 8, 0, 0)
    P.purlin_dispatch_rows(ctx, None, None, None, 0, 2, 8, 4, 0)
    P.purlin_combine_rows(ctx, None, None, None, 0, 2, 8, 4, 0)
    y = t.clone()
    P.purlin_combine_rows(ctx, None, place, y, 2, 2, 8, 0, 0, weights=w)     # no rows at all
    dw = torch.full((2, 2), 5.0, device="cuda")
    P.purlin_combine_rows_backward(ctx, t, None, place, w, None, dw, 2, 2, 8, 0, 0)
    P.purlin_check(ctx)
    assert not bool(y.any()) and not bool(dw.any())
    dw.fill_(5.0)
    P.purlin_combine_rows_backward(ctx, None, None, place, w, None, dw, 2, 2, 0, 4, 0)
    P.purlin_check(ctx)
    assert not bool(dw.any())


def test_scales_of_no_rows(P, ctx):
    """An empty tensor has no address: no tokens, or no rows for them, is not a
    scale that was left out."""
    from collective_datapath_atom_gb300 import torch_api

    def place(*shape):
        return torch.full(shape, -1, device="cuda", dtype=torch.int32)

    x, s = torch.ones(3, 16, device="cuda"), torch.ones(3, device="cuda")
    out, scales = torch_api.dispatch_rows(x[:0], place(0, 2), ctx, out_rows=4, scales=s[:0])
    assert out.shape == (4, 16) and not bool(out.any()) and not bool(scales.any())
    out, scales = torch_api.dispatch_rows(x, place(3, 2), ctx, out_rows=0, scales=s)
    assert out.shape == (0, 16) and scales.shape == (0,)
    P.purlin_check(ctx)


def test_offsets_past_32_bits(P, ctx):
    """Rows behind 2^31 elements (2^32 bytes) of a buffer."""
    rows, cols = 140_000, 16_384
    place = torch.tensor([[139_999, 131_072], [1, 139_000]], device="cuda", dtype=torch.int32)
    x = torch.randn(2, cols, device="cuda").bfloat16()
    out = torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16)
    P.purlin_dispatch_rows(ctx, x, place, out, 2, 2, cols, rows, 1)
    y = torch.empty_like(x)
    P.purlin_combine_rows(ctx, out, place, y, 2, 2, cols, rows, 1)
    w, dw = torch.full((2, 2), 2.0, device="cuda"), torch.empty(2, 2, device="cuda")
    P.purlin_combine_rows_backward(ctx, x, out, place, w, out, dw, 2, 2, cols, rows, 1)
    P.purlin_check(ctx)
    for t in range(2):
        for p in place[t].tolist():
            assert torch.equal(out[p].float(), 2 * x[t].float())
    assert torch.equal(y.float(), 2 * x.float())
    norm = x.double().square().sum(1, keepdim=True).expand(2, 2)
    assert bool(((dw.double() - norm).abs() <= norm * (cols + 1) * U).all())
    assert int(out.any(1).sum()) == 4
