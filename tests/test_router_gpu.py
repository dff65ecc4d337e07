"""The router and its gradient on a GPU, against the definitions in 64 bits.

The choice has to be equal.  Tolerances of the weights, with u = 2^-24: an exponential
is off by 2 ulp (4 u) and by its argument's rounding, |argument| u; a sum of n positive
terms held HELD a lane and joined over 32 lanes by at most HELD + 5 u, HELD <= 64; sums,
quotients and products by a u each.  So a weight is off by at most (69 + 4 + 10 + range)
u relative, range the largest difference of two logits that enter it, and as much for
its denominator: 2 (90 + range) u holds for both, and for the gradients times the sum
of the absolute values of their terms.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T = {0: torch.float32, 1: torch.bfloat16}
INF, NAN = math.inf, math.nan


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


def scores64(l, sigmoid):
    l = l.clamp(max=torch.finfo(torch.float32).max)
    if sigmoid:
        return torch.sigmoid(l)
    top = l.amax(1, keepdim=True)
    e = torch.exp(l - torch.where(top == -INF, 0.0, top))
    s = e.sum(1, keepdim=True)
    return torch.where(s > 0, e / s, 0.0)


def order_of(v):
    """Indices by falling value, ties to the lowest."""
    return v.sort(dim=-1, descending=True, stable=True).indices


def reference(l, bias, r):
    """(chosen, chosen logits, scores) of double logits on the CPU, expert by expert."""
    sigmoid = r["scores"] == 1
    s = scores64(l, sigmoid)
    # without a bias the scores' order is the logits', exactly
    c = l.clone() if bias is None else s + bias[None, :]
    out = (l == -INF) | torch.isnan(l) | torch.isnan(c) | (c == -INF)
    c[out] = -INF
    tokens, experts = l.shape
    groups = max(1, r.get("groups", 1))
    if groups > 1:
        by = (s if bias is None and r.get("group_top", 1) == 2 else c).clone()
        by[out] = -INF
        best = by.view(tokens, groups, -1).sort(2, descending=True).values[:, :, :max(1, r.get("group_top", 1))]
        v = torch.where(best == -INF, 0.0, best).sum(2)
        v[best[:, :, 0] == -INF] = -INF
        kept = order_of(v)[:, :r["top_groups"]]
        keep = torch.zeros(tokens, groups, dtype=torch.bool).scatter_(1, kept, True)
        c = torch.where(keep.repeat_interleave(experts // groups, 1), c, -INF)
    idx = order_of(c)[:, :r["top_k"]]
    chosen = torch.where(c.gather(1, idx) == -INF, -1, idx)
    return chosen, s


def weights64(l, chosen, s, r):
    real, at = chosen >= 0, chosen.clamp_min(0)
    scale = r.get("scale", 0.0) or 1.0
    if r.get("renormalise"):
        ll = torch.where(real, l.clamp(max=torch.finfo(torch.float32).max).gather(1, at), -INF)
        logs = torch.nn.functional.logsigmoid(ll) if r["scores"] == 1 else ll
        top = logs.amax(1, keepdim=True)
        n = torch.where(real, torch.exp(logs - torch.where(top == -INF, 0.0, top)), 0.0)
        d = n.sum(1, keepdim=True)
        return torch.where(d > 0, n / d, 0.0) * scale
    return torch.where(real, s.gather(1, at), 0.0) * scale


def run_once(P, ctx, l, bias, r, dtype):
    tokens = l.shape[0]
    w = torch.full((tokens, r["top_k"]), -7.0, device="cuda")
    chosen = torch.full((tokens, r["top_k"]), -7, device="cuda", dtype=torch.int32)
    P.purlin_route(ctx, l, w, chosen, tokens, P.purlin_router(**r), dtype, bias=bias, ld=l.stride(0))
    P.purlin_check(ctx)
    return w.cpu(), chosen.cpu().long()


def run(P, ctx, l, bias, r, dtype):
    """The router's answer; the same rows among many, where a warp has several tokens,
    have to get the same one (sums in another order: 2 * 37 u of positive terms)."""
    w, chosen = run_once(P, ctx, l, bias, r, dtype)
    tokens, times = l.shape[0], -(-6001 // l.shape[0])
    many = torch.cat([l] * times)[:6001] if l.is_contiguous() else l.repeat(times, 1)[:6001]
    wide = torch.full((6001, l.stride(0)), 60.0, device="cuda", dtype=l.dtype)[:, :l.shape[1]]
    wide.copy_(many)
    mw, mc = run_once(P, ctx, wide, bias, r, dtype)
    at = torch.arange(6001) % tokens
    assert torch.equal(mc, chosen[at])
    assert torch.equal(torch.isnan(mw), torch.isnan(w[at]))
    near = (mw - w[at]).abs() <= w[at].abs() * 80 * U
    assert bool((near | torch.isnan(mw)).all())
    return w, chosen


def spread(l):
    f = torch.where(torch.isfinite(l), l, 0.0)
    return float((f.amax() - f.amin()).clamp(max=200)) if l.numel() else 0.0


def check(P, ctx, l, bias, r, dtype):
    w, chosen = run(P, ctx, l, bias, r, dtype)
    l64 = l.cpu().double()
    want, s = reference(l64, None if bias is None else bias.cpu().double(), r)
    assert torch.equal(chosen, want)
    w64 = weights64(l64, want, s, r)
    # (1e-37: scores below it round in absolute steps)
    assert bool(((w.double() - w64).abs() <= w64 * 2 * (90 + spread(l64)) * U + 1e-37).all())


def logits(tokens, experts, seed, dtype, scale=1.5, pitch=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.full((tokens, pitch or experts), 50.0, device="cuda", dtype=T[dtype])
    t[:, :experts] = (torch.randn(tokens, experts, device="cuda", generator=g) * scale).to(T[dtype])
    return t[:, :experts]


def bias_of(experts, seed, scale=0.05):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(experts, device="cuda", generator=g) * scale


ROUTERS = [
    dict(experts=1, top_k=1, scores=0), dict(experts=8, top_k=2, scores=0, renormalise=1),
    dict(experts=7, top_k=7, scores=1, renormalise=1, scale=2.5),
    dict(experts=64, top_k=6, scores=0), dict(experts=60, top_k=4, scores=0, groups=3, top_groups=2),
    dict(experts=129, top_k=5, scores=1), dict(experts=256, top_k=8, scores=1, groups=8, top_groups=4,
                                               group_top=2, renormalise=1, scale=2.5),
    dict(experts=256, top_k=8, scores=0, groups=8, top_groups=8, group_top=2),
    dict(experts=160, top_k=6, scores=0, groups=8, top_groups=3, scale=16.0),
    dict(experts=1024, top_k=32, scores=0, renormalise=1), dict(experts=1024, top_k=8, scores=1),
    dict(experts=1020, top_k=9, scores=1, groups=17, top_groups=5, group_top=2),
    dict(experts=32, top_k=2, scores=0, groups=32, top_groups=2, group_top=2),
    dict(experts=96, top_k=32, scores=1, groups=2, top_groups=1, renormalise=1),
]


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("biased", [False, True], ids=["", "bias"])
@pytest.mark.parametrize("r", ROUTERS, ids=lambda r: f"{r['experts']}top{r['top_k']}")
def test_route(P, ctx, r, biased, dtype):
    for tokens in (1, 37, 1000):
        l = logits(tokens, r["experts"], 10 + tokens, dtype)
        check(P, ctx, l, bias_of(r["experts"], 3) if biased else None, r, dtype)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
def test_pitch_and_offset(P, ctx, dtype):
    r = dict(experts=100, top_k=4, scores=1, renormalise=1)
    check(P, ctx, logits(33, 100, 5, dtype, pitch=131), bias_of(100, 6), r, dtype)
    check(P, ctx, logits(33, 103, 5, dtype)[:, 3:], None, r, dtype)


@pytest.mark.parametrize("scores", [0, 1], ids=["softmax", "sigmoid"])
def test_large_logits(P, ctx, scores):
    # scores that leave binary32: the order is the logits', the weights theirs
    for scale, shift in ((30.0, 0.0), (5.0, -300.0), (5.0, 300.0), (3e37, 0.0)):
        l = logits(50, 64, 8, 0, scale) + shift
        check(P, ctx, l, None, dict(experts=64, top_k=6, scores=scores, renormalise=1), 0)


def near_ties(tokens, experts, seed):
    """Logits and a bias whose sigmoid choices differ by less than binary32 shows."""
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(tokens, experts, generator=g)
    bias = (0.8 - torch.sigmoid(l[0].double())).float()
    l = l[:1].repeat(tokens, 1) + torch.randint(-2, 3, (tokens, experts), generator=g) * 2.0 ** -24
    return l, bias


@pytest.mark.parametrize("experts,top_k", [(4, 2), (20, 4), (33, 6), (256, 8), (256, 32)])
@pytest.mark.parametrize("grouped", [False, True])
def test_near_ties(P, ctx, experts, top_k, grouped):
    """Every expert's choice value is 0.8 and some 1e-8: more than 32 of them near the
    border take the longest way."""
    r = dict(experts=experts, top_k=top_k, scores=1)
    if grouped and experts % 4 == 0 and top_k <= experts // 2:
        r.update(groups=4, top_groups=2, group_top=2)
    l, bias = near_ties(64, experts, 4)
    w, chosen = run(P, ctx, l.cuda(), bias.cuda(), r, 0)
    c = torch.sigmoid(l.double()) + bias.double()
    gaps = c.sort(1).values.diff(dim=1)
    assert float(gaps.max()) < 2.0 ** -20          # near indeed, for binary32
    assert bool(((gaps > 1e-15) | (gaps == 0)).all())   # and apart, for binary64
    assert torch.equal(chosen, reference(l.double(), bias.double(), r)[0])


@pytest.mark.parametrize("biased", [False, True])
def test_equal_logits_go_to_the_lowest(P, ctx, biased):
    r = dict(experts=256, top_k=8, scores=1, groups=8, top_groups=4, group_top=2, renormalise=1)
    bias = torch.zeros(256, device="cuda") if biased else None
    w, chosen = run(P, ctx, torch.zeros(40, 256, device="cuda"), bias, r, 0)
    assert torch.equal(chosen, torch.arange(8).expand(40, 8))
    assert torch.equal(w, torch.full((40, 8), 0.125))
    # many equal pairs: rounded logits, few different biases
    g = torch.Generator(device="cuda").manual_seed(2)
    l = torch.randint(-3, 4, (500, 256), device="cuda", generator=g).float() / 2
    b = torch.randint(0, 2, (256,), device="cuda", generator=g).float() / 64 if biased else None
    check(P, ctx, l, b, r, 0)
    check(P, ctx, l, b, dict(r, scores=0, renormalise=0), 0)
    check(P, ctx, -l.abs() * 0.0, b, r, 0)          # -0 is 0


@pytest.mark.parametrize("scores", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
def test_masks(P, ctx, scores, renormalise, biased):
    r = dict(experts=48, top_k=5, scores=scores, renormalise=renormalise, groups=4, top_groups=2,
             group_top=2)
    l = logits(60, 48, 12, 0)
    l[:, 5] = -INF
    l[0] = -INF                                     # nobody
    l[1, 1:] = -INF                                 # one
    l[2, :44] = -INF                                # one group, four of twelve
    l[3, ::2] = -INF
    l[4, 7] = INF                                   # counts as the largest value
    l[5, 3], l[5, 40] = INF, INF
    l[6] = torch.finfo(torch.float32).min           # finite, all the same
    b = bias_of(48, 2) if biased else None
    if biased:
        b[9], b[10] = -INF, NAN
    check(P, ctx, l, b, r, 0)
    w, chosen = run(P, ctx, l, b, r, 0)
    assert torch.equal(chosen[0], torch.full((5,), -1)) and not bool(w[0].any())
    assert chosen[1].tolist() == [0, -1, -1, -1, -1]


def test_nan_logits_show_in_the_weights(P, ctx):
    r = dict(experts=40, top_k=4, scores=1, renormalise=1)
    l = logits(20, 40, 13, 0)
    clean = l.clone()
    l[3, 17] = NAN
    clean[3, 17] = -INF
    w, chosen = run(P, ctx, l, bias_of(40, 1), r, 0)
    w0, chosen0 = run(P, ctx, clean, bias_of(40, 1), r, 0)
    assert torch.equal(chosen, chosen0)
    assert bool(torch.isnan(w[3]).all())
    w[3] = w0[3]
    assert torch.equal(w, w0)


def test_infinite_bias(P, ctx):
    r = dict(experts=16, top_k=3, scores=1)
    b = torch.zeros(16, device="cuda")
    b[4] = b[9] = INF
    b[2] = 1e30
    check(P, ctx, logits(9, 16, 1, 0), b, r, 0)


# ---------------------------------------------------------------- backward ---

def grads64(dw, l, chosen, r):
    """Gradient of the weights' definition by autograd in 64 bits."""
    l = l.clone().requires_grad_(True)
    real, at = chosen >= 0, chosen.clamp_min(0)
    scale = r.get("scale", 0.0) or 1.0
    if r.get("renormalise"):
        ll = torch.where(real, l.gather(1, at), -1e30)
        logs = torch.nn.functional.logsigmoid(ll) if r["scores"] == 1 else ll
        w = torch.softmax(logs, 1)
    else:
        s = torch.sigmoid(l) if r["scores"] == 1 else torch.softmax(l, 1)
        w = s.gather(1, at)
    w = torch.where(real, w, 0.0) * scale
    (w * torch.where(real, dw, 0.0)).sum().backward()
    return torch.nan_to_num(l.grad)


def check_backward(P, ctx, l, dw, chosen, r, dtype, in_place=False):
    tokens, experts = l.shape
    want = grads64(dw.double().cpu(), l.double().cpu(), chosen.cpu().long(), r)
    d = l if in_place else torch.full((tokens, experts), 9.0, device="cuda", dtype=l.dtype)
    P.purlin_route_backward(ctx, dw, l, chosen, d, tokens, P.purlin_router(**r), dtype,
                            ld=l.stride(0), ldd=d.stride(0))
    P.purlin_check(ctx)
    got = d.cpu().double()
    scale = r.get("scale", 0.0) or 1.0
    terms = scale * dw.double().cpu().abs().sum(1, keepdim=True)     # |g| (1 + sum of p)
    bound = 4 * terms * (90 + spread(l.double().cpu() if not in_place else want)) * U
    bound = bound + want.abs() * (2.0 ** -8 if dtype else U) + 1e-37
    assert bool(((got - want).abs() <= bound).all())
    assert bool((got[want == 0].abs() <= (terms.expand_as(got)[want == 0] * 1e-6)).all())


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("scores", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [0, 1])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 64, 6), (300, 129, 4), (33, 1024, 32),
                                              (1000, 8, 8)])
def test_backward(P, ctx, tokens, experts, k, scores, renormalise, dtype):
    r = dict(experts=experts, top_k=k, scores=scores, renormalise=renormalise, scale=2.5)
    l = logits(tokens, experts, 21, dtype)
    _, chosen = run(P, ctx, l, bias_of(experts, 4), r, dtype)
    chosen = chosen.int().cuda()
    if k > 2:
        chosen[::3, k - 1] = -1                     # fewer than top_k
        chosen[tokens // 2, 1:] = experts + 5       # outside: none
    g = torch.Generator(device="cuda").manual_seed(22)
    dw = torch.randn(tokens, k, device="cuda", generator=g)
    valid = torch.where(chosen < experts, chosen, -1)
    d = torch.full((tokens, experts), 9.0, device="cuda", dtype=l.dtype)
    P.purlin_route_backward(ctx, dw, l, chosen, d, tokens, P.purlin_router(**r), dtype)
    d2 = torch.full_like(d, 8.0)
    P.purlin_route_backward(ctx, dw, l, valid, d2, tokens, P.purlin_router(**r), dtype)
    P.purlin_check(ctx)
    assert torch.equal(d, d2)
    check_backward(P, ctx, l, dw, valid, r, dtype)


@pytest.mark.parametrize("scores,renormalise", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_backward_by_differences(P, ctx, scores, renormalise):
    """Central differences of the forward pass: with h = 2^-6 the third-order term is
    below h^2 (all derivatives of these weights are below 1), and the weights' own
    error, 2^-17 of values below 1, is divided by h."""
    r = dict(experts=12, top_k=4, scores=scores, renormalise=renormalise)
    base = torch.linspace(-1.5, 1.5, 12)[torch.randperm(12, generator=torch.Generator().manual_seed(1))]
    h, dw = 2.0 ** -6, torch.tensor([0.5, -1.0, 0.25, 2.0])
    steps = torch.cat([base + h * torch.eye(12), base - h * torch.eye(12)]).cuda()
    w, chosen = run(P, ctx, steps.contiguous(), None, r, 0)
    w0, chosen0 = run(P, ctx, base[None].cuda(), None, r, 0)
    assert torch.equal(chosen, chosen0.expand(24, 4))   # no step reaches another choice
    f = (w.double() * dw.double()).sum(1)
    want = (f[:12] - f[12:]) / (2 * h)
    d = torch.empty(1, 12, device="cuda")
    P.purlin_route_backward(ctx, dw[None].cuda(), base[None].cuda(), chosen0.int().cuda(), d, 1,
                            P.purlin_router(**r), 0)
    P.purlin_check(ctx)
    assert float((d.cpu().double()[0] - want).abs().max()) <= 3.75 * (h * h + 2.0 ** -17 / h)


@pytest.mark.parametrize("scores,renormalise", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_backward_in_place_pitch_and_masks(P, ctx, scores, renormalise):
    r = dict(experts=70, top_k=3, scores=scores, renormalise=renormalise)
    l = logits(40, 70, 31, 0, pitch=75)
    l[:, 4] = -INF
    l[7] = -INF
    _, chosen = run(P, ctx, l, None, r, 0)
    assert bool((chosen[7] == -1).all())
    dw = torch.randn(40, 3, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    chosen = chosen.int().cuda()
    d = torch.full((40, 77), 9.0, device="cuda")
    P.purlin_route_backward(ctx, dw, l, chosen, d, 40, P.purlin_router(**r), 0, ld=75, ldd=77)
    assert bool((d[:, 70:] == 9).all())             # behind the rows: as it was
    soft = l.clone()
    soft[7] = 0.0                                   # (an empty row has no softmax; its gradient is 0)
    want = grads64(dw.double().cpu(), soft.double().cpu(), chosen.cpu().long(), r)
    want[7] = 0
    assert float((d[:, :70].cpu().double() - want).abs().max()) < 1e-5
    full = l._base if l._base is not None else l
    P.purlin_route_backward(ctx, dw, l, chosen, l, 40, P.purlin_router(**r), 0, ld=75, ldd=75)
    P.purlin_check(ctx)
    assert torch.equal(l, d[:, :70])
    assert bool((full[:, 70:] == 50).all())


@pytest.mark.parametrize("scores,renormalise", [(0, 0), (1, 0)])
def test_backward_of_an_expert_twice(P, ctx, scores, renormalise):
    r = dict(experts=20, top_k=4, scores=scores, renormalise=renormalise)
    l = logits(6, 20, 41, 0)
    twice = torch.tensor([[3, 5, 3, 3]] * 6, device="cuda", dtype=torch.int32)
    once = torch.tensor([[3, 5, -1, -1]] * 6, device="cuda", dtype=torch.int32)
    dw = torch.tensor([[1.0, 2.0, 0.5, 0.25]] * 6, device="cuda")
    summed = torch.tensor([[1.75, 2.0, 0, 0]] * 6, device="cuda")
    a, b = torch.empty(6, 20, device="cuda"), torch.empty(6, 20, device="cuda")
    P.purlin_route_backward(ctx, dw, l, twice, a, 6, P.purlin_router(**r), 0)
    P.purlin_route_backward(ctx, summed, l, once, b, 6, P.purlin_router(**r), 0)
    P.purlin_check(ctx)
    assert float((a - b).abs().max()) <= 1e-6


def test_no_tokens(P, ctx):
    e = torch.empty(0, 8, device="cuda")
    r = P.purlin_router(experts=8, top_k=2)
    P.purlin_route(ctx, e, None, None, 0, r, 0)
    P.purlin_route_backward(ctx, None, e, None, None, 0, r, 0)
    P.purlin_check(ctx)
