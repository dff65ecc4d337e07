"""The router, the dispatch, the way back and the norms around a block, together: the
example with the collectives, a training step through the tensor calls, the tensor
calls' checks, and captured graphs.

Roundings to bf16 are followed in the 64-bit forms, so that the two differ where a
value lies next to a border, by at most a step, 2^-7 of it, for each of the roundings
on the way; sums average that out, and the comparisons below are of whole tensors'
norms, with 2^-7 for each rounding that can reach the tensor.
"""
import pytest

torch = pytest.importorskip("torch")

STEP = 2.0 ** -7
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def T():
    import __graft_entry__

    __graft_entry__.build()
    from collective_datapath_atom_gb300 import torch_api

    return torch_api


class FakeHandle:
    R = 2


def test_argument_checks_without_a_gpu(T):
    h = FakeHandle()
    x, w = torch.zeros(4, 8), torch.zeros(8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    config = T.router(8, 2)
    for call in (lambda: T.block_norm(x, w, h), lambda: T.block_norm_backward(x, x, x, w, h),
                 lambda: T.route(x, config, h), lambda: T.route_backward(x[:, :2], x, i, config, h),
                 lambda: T.expert_order(i, 8, h), lambda: T.dispatch_rows(x, i, h),
                 lambda: T.combine_rows(x, i, h), lambda: T.combine_rows_backward(x, x, i, w, h),
                 lambda: T.router(8, 2, scores="tanh"), lambda: T.router(8, 2, scale=0.0)):
        with pytest.raises(ValueError):       # host tensors, and a router that is none
            call()


@pytest.fixture
def handle(T):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = T.initialize(8, stream=torch.cuda.current_stream())
    yield h
    T.finalize(h)


@pytest.mark.gpu
def test_shapes_and_types_are_checked(T, handle):
    h = handle
    x = torch.zeros(4, 64, device="cuda", dtype=BF16)
    w = torch.zeros(64, device="cuda", dtype=BF16)
    i = torch.zeros(4, 2, device="cuda", dtype=torch.int32)
    f = torch.zeros(4, 2, device="cuda")
    config = T.router(64, 2)
    for bad in (lambda: T.block_norm(x.t(), w, h), lambda: T.block_norm(x, w[:63], h),
                lambda: T.block_norm(x, w, h, residual=x[:3]), lambda: T.block_norm(x, w, h, gate=w[:8]),
                lambda: T.block_norm(x, w, h, gate=x[:, :8]), lambda: T.block_norm(x, None, h, quantize=True),
                lambda: T.block_norm(x, w, h, post_weight=w[:5]),
                lambda: T.block_norm(w.expand(4, 64), w, h),
                lambda: T.block_norm_backward(x[:3], x, x, w, h),
                lambda: T.route(x[:, :32], config, h), lambda: T.route(x, config, h, bias=f[0]),
                lambda: T.route_backward(f[:3], x, i, config, h), lambda: T.expert_order(i.t(), 8, h),
                lambda: T.dispatch_rows(x, i[:3], h), lambda: T.dispatch_rows(x, i, h, out=x[:, :32]),
                lambda: T.dispatch_rows(x, i, h, scales=f[:3, 0]),
                lambda: T.dispatch_rows(x, i, h, out_scales=f[:, 0]),
                lambda: T.combine_rows(x, i, h, weights=f[:3]), lambda: T.combine_rows(x, i, h, shared=x[:3]),
                lambda: T.combine_rows_backward(x[:, :8], x, i, f, h)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: T.block_norm(x, w.float(), h), lambda: T.route(x.half(), config, h),
                lambda: T.expert_order(i.long(), 8, h), lambda: T.dispatch_rows(x, i.long(), h),
                lambda: T.combine_rows(x, i, h, weights=f.bfloat16()),
                lambda: T.block_norm(x, w, h, residual=x.float())):
        with pytest.raises(TypeError):
            bad()


def rms(t, eps=1e-5):
    return t / torch.sqrt(t.square().mean(1, keepdim=True) + eps)


def close(got, want, roundings):
    got, want = got.double(), want.detach().double()
    off = float((got - want).norm() / want.norm())
    assert off <= roundings * STEP, off


@pytest.mark.gpu
@pytest.mark.parametrize("skew", [0.0, 4.0], ids=["even", "skewed"])
def test_example(T, handle, skew):
    import collective_datapath_atom_gb300 as P
    from collective_datapath_atom_gb300.examples import moe_block as example

    R, tokens, H, N, k = 8, 8 * 40, 128, 96, 2
    g = torch.Generator(device="cuda").manual_seed(11)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).bfloat16()

    partials = [torch.randint(-8, 9, (tokens, H), device="cuda", generator=g).bfloat16() for _ in range(R)]
    residual = torch.randint(-8, 9, (tokens, H), device="cuda", generator=g).bfloat16()
    norms = [{n: (1 + 0.1 * randn(H).float()).bfloat16() for n in ("post", "gate", "weight")} for _ in range(2)]
    wr, up, down = randn(R, H, scale=H ** -0.5), randn(R, N, H, scale=H ** -0.5), randn(R, H, N, scale=N ** -0.5)
    bias = torch.linspace(skew, 0, R, device="cuda")
    got = example.moe_block(handle, partials, residual, norms, wr, bias, up, down, k, 0.9, 0.5)
    P.purlin_check(handle)

    def norm(x, before, n):
        t = 0.9 * before + 0.5 * n["gate"].double() * n["post"].double() * rms(x)
        return rms(t) * n["weight"].double(), t

    x = sum(p.double() for p in partials)
    hidden, total = norm(x, residual.double(), norms[0])
    close(got["hidden"], hidden, 1)
    # from the block's own input on: its choice is the router's of these rows
    h = got["hidden"].double()
    s = torch.sigmoid((h @ wr.double().t()).bfloat16().double())
    experts = got["experts"].long()
    picked = s.gather(1, experts)
    c = s + bias.double()
    worst = c.gather(1, experts).amin(1)
    rest = c.scatter(1, experts, -1.0).amax(1)
    assert bool((worst >= rest - STEP).all())        # (logits are rounded: a step of a score)
    close(got["weights"], picked / picked.sum(1, keepdim=True), 1)
    assert torch.equal(got["load"], torch.bincount(experts.view(-1), minlength=R))
    if skew:
        assert int(got["load"][0]) == tokens         # the bias sends every token there
    y = torch.zeros_like(h)
    for e in range(R):
        inner = (h @ up[e].double().t()).bfloat16().double().relu()
        outer = (inner @ down[e].double().t()).bfloat16().double()
        share = torch.where(experts == e, got["weights"].double(), 0.0).sum(1, keepdim=True)
        y += share * outer
    y, total = norm(y.bfloat16().double(), total.bfloat16().double(), norms[1])
    close(got["y"], y, 4)
    close(got["total"], total, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("capacity", [0, 30])
def test_training_step(T, handle, capacity):
    """Forward and backward of norm, router, dispatch, experts, way back, norm; the
    64-bit form by autograd, for the same choice."""
    h, tokens, H, E, k = handle, 100, 64, 10, 3
    g = torch.Generator(device="cuda").manual_seed(12)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).bfloat16()

    x, res = randn(tokens, H), randn(tokens, H)
    post, gate, w1, w2 = ((1 + 0.1 * randn(H).float()).bfloat16() for _ in range(4))
    wr, we = randn(E, H, scale=H ** -0.5), randn(E, H, H, scale=H ** -0.5)
    dy, dtotal = randn(tokens, H), randn(tokens, H)
    config = T.router(E, k, "softmax", groups=2, top_groups=2, renormalise=True, scale=2.0)

    hid, t1 = T.block_norm(x, w1, h, residual=res, post_weight=post, gate=gate, block_scale=0.5)
    logits = hid.float() @ wr.float().t()
    wts, experts = T.route(logits, config, h)
    place, begin, count = T.expert_order(experts, E, h, capacity=capacity)
    n = E * capacity if capacity else tokens * k
    sent = T.dispatch_rows(hid, place, h, out_rows=n)
    out = T.grouped_matmul(sent, we, begin, count, h)
    blk = T.combine_rows(out, place, h, weights=wts)
    y, t2 = T.block_norm(blk, w2, h, residual=t1)

    b2 = T.block_norm_backward(dy, blk, t2, w2, h, dtotal=dtotal)
    dout, dwts = T.combine_rows_backward(b2["dx"], out, place, wts, h)
    dsent = T.grouped_matmul(dout, we, begin, count, h, transposed=True)
    dwe = T.grouped_matmul_weight_grad(dout, sent, begin, count, h)
    dlogits = T.route_backward(dwts, logits, experts, config, h)
    dhid = T.combine_rows(dsent, place, h)
    dhid = (dhid.float() + dlogits @ wr.float()).bfloat16()
    b1 = T.block_norm_backward(dhid, x, t1, w1, h, dtotal=b2["dresidual"], post_weight=post, gate=gate,
                               block_scale=0.5)
    T.check(h)

    leaf = {n: t.double().requires_grad_(True) for n, t in
            dict(x=x, res=res, post=post, gate=gate, w1=w1, w2=w2, wr=wr, we=we).items()}
    one = leaf["res"] + 0.5 * leaf["gate"] * leaf["post"] * rms(leaf["x"])
    hid64 = rms(one) * leaf["w1"]
    l64 = hid64 @ leaf["wr"].t()
    at = experts.long()
    sm = torch.softmax(l64.gather(1, at), 1) * 2.0
    kept = place >= 0
    rows = torch.einsum("th,tkoh->tko", hid64, leaf["we"][at])
    blk64 = (torch.where(kept, sm, 0.0)[:, :, None] * rows).sum(1)
    t64 = one + blk64
    y64 = rms(t64) * leaf["w2"]
    ((y64 * dy.double()).sum() + (t64 * dtotal.double()).sum()).backward()
    if capacity:
        assert 0 < int((~kept).sum()) < tokens * k and int(count.max()) == capacity
    else:
        assert bool(kept.all())
    # the choice: no other expert has a larger logit than the least of the chosen
    assert bool((logits.gather(1, at).amin(1) >= logits.scatter(1, at, -1e9).amax(1)).all())
    close(y, y64, 5)                                   # hid, t1, out, blk, y
    close(t2, t64, 5)
    close(wts, sm, 2)
    for got, want, roundings in ((b1["dx"], "x", 12), (b1["dresidual"], "res", 12), (b1["dpost_weight"], "post", 12),
                                 (b1["dgate"], "gate", 12), (b1["dweight"], "w1", 12), (b2["dweight"], "w2", 8),
                                 (dlogits.t() @ hid.float(), "wr", 12), (dwe, "we", 8)):
        close(got, leaf[want].grad, roundings)


@pytest.mark.gpu
def test_two_captured_graphs_share_a_workspace(T):
    """Two graphs of one context, replayed one after the other with inputs that change:
    the gradients' partial sums and the order's counts lie in the same memory."""
    import collective_datapath_atom_gb300 as P

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ctx = P.purlin_init(1, s)
        H, n, E = 256, 700, 20
        ins = {k: torch.zeros(n, H, device="cuda", dtype=BF16) for k in ("dy", "x", "total", "dx")}
        w = torch.ones(H, device="cuda", dtype=BF16)
        dw, dp = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
        chosen = torch.zeros(9000, device="cuda", dtype=torch.int32)
        place = torch.empty_like(chosen)
        begin, count = (torch.empty(E, device="cuda", dtype=torch.int64) for _ in range(2))

        def one():
            P.purlin_block_norm_backward(ctx, ins["dy"], ins["x"], ins["total"], w, ins["dx"], dw, n, H, 1e-5, 1,
                                         post_weight=w, dpost_weight=dp)

        def two():
            P.purlin_expert_order(ctx, chosen, place, begin, count, 9000, E)

        graphs = []
        for f in (one, two):
            f()                                         # the workspace grows before a capture
            s.synchronize()
        for f in (one, two):
            f()
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                f()
            graphs.append(graph)
        for seed in range(3):
            g = torch.Generator(device="cuda").manual_seed(seed)
            for k in ("dy", "x", "total"):
                ins[k].copy_(torch.randn(n, H, device="cuda", generator=g))
            chosen.copy_(torch.randint(0, E, (9000,), device="cuda", generator=g))
            for graph in graphs + graphs[::-1]:
                graph.replay()
            s.synchronize()
            got = [t.clone() for t in (ins["dx"], dw, dp, place, begin, count)]
            one(), two()
            s.synchronize()
            for a, b in zip(got, (ins["dx"], dw, dp, place, begin, count)):
                assert torch.equal(a, b)
            assert torch.equal(count, torch.bincount(chosen, minlength=E))
            unit = rms(ins["total"].double())
            assert float((dw.double() - (ins["dy"].double() * unit).sum(0)).abs().max()) < 1e-3
        ctx.close()


@pytest.mark.gpu
def test_workspace_does_not_grow_during_capture():
    import collective_datapath_atom_gb300 as P

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ctx = P.purlin_init(1, s)
        chosen = torch.zeros(100000, device="cuda", dtype=torch.int32)
        place, begin = torch.empty_like(chosen), torch.empty(1024, device="cuda", dtype=torch.int64)
        count = torch.empty_like(begin)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(P.PurlinError) as e:
                P.purlin_expert_order(ctx, chosen, place, begin, count, 100000, 1024)
        assert e.value.status == P.PURLIN_ERR_UNSUPPORTED
        ctx.close()


@pytest.mark.gpu
def test_tensor_calls_on_another_stream(T):
    """Results of calls on a stream of their own, behind work that still fills the inputs."""
    side = torch.cuda.Stream()
    h = T.initialize(1, stream=side)
    g = torch.Generator(device="cuda").manual_seed(3)
    want = torch.randn(300, 96, device="cuda", generator=g).bfloat16()
    w = torch.ones(96, device="cuda", dtype=BF16)
    try:
        for _ in range(5):
            x = torch.zeros(300, 96, device="cuda", dtype=BF16)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.cuda._sleep(2_000_000)
                x.copy_(want)
            experts = torch.arange(600, device="cuda", dtype=torch.int32).view(300, 2) % 7
            side.wait_stream(torch.cuda.current_stream())
            place, begin, count = T.expert_order(experts, 7, h, capacity=100)
            sent = T.dispatch_rows(x, place, h, out_rows=700)
            y, total = T.block_norm(x, w, h)
            back = T.combine_rows(sent, place, h)
            torch.cuda.current_stream().wait_stream(side)
            assert torch.equal(back, (2 * want.float()).bfloat16())
            assert torch.equal(total, want)
            assert count.tolist() == torch.bincount(experts.view(-1), minlength=7).tolist()
            assert int((sent != 0).any(1).sum()) == 600     # the rest of the buffer: zeros
    finally:
        T.finalize(h)
