"""The layer operators through the tensor-level calls, and the example that runs
them with the collectives: argument checks on the CPU, results on a GPU."""
import pytest

torch = pytest.importorskip("torch")


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
    i = torch.zeros(2, dtype=torch.int64)
    for call in (lambda: T.rms_norm(x, w, h), lambda: T.rms_norm_backward(x, x, w, h),
                 lambda: T.grouped_matmul(x, torch.zeros(2, 8, 8), i, i, h),
                 lambda: T.grouped_matmul_weight_grad(x, x, i, i, h)):
        with pytest.raises(ValueError):       # host tensors
            call()


@pytest.mark.gpu
def test_shapes_and_types_are_checked(T):
    h = T.initialize(2, stream=torch.cuda.current_stream())
    try:
        x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
        w = torch.zeros(64, device="cuda", dtype=torch.bfloat16)
        e = torch.zeros(2, 32, 64, device="cuda", dtype=torch.bfloat16)
        i = torch.zeros(2, device="cuda", dtype=torch.int64)
        f = torch.zeros(4, device="cuda")
        for bad in (lambda: T.rms_norm(x.t(), w, h), lambda: T.rms_norm(x, w[:63], h),
                    lambda: T.rms_norm(x, w, h, residual=x[:3]),
                    lambda: T.rms_norm(x, w, h, scales=f),
                    lambda: T.rms_norm_backward(x, x, w, h, dx=x[:, :8]),
                    lambda: T.grouped_matmul(x[:, :32], e, i, i, h),
                    lambda: T.grouped_matmul(x, e, i[:1], i, h),
                    lambda: T.grouped_matmul(x, e, i, i, h, x_scales=f),
                    lambda: T.grouped_matmul(x, e[:, :16], i, i, h),
                    lambda: T.grouped_matmul_weight_grad(x, x[:3], i, i, h)):
            with pytest.raises(ValueError):
                bad()
        for bad in (lambda: T.rms_norm(x, w.float(), h), lambda: T.rms_norm(x.half(), w.half(), h),
                    lambda: T.grouped_matmul(x, e, i.int(), i, h),
                    lambda: T.grouped_matmul(x.float(), e.float(), i, i, h)):
            with pytest.raises(TypeError):
                bad()
    finally:
        T.finalize(h)


@pytest.mark.gpu
def test_tensor_calls(T):
    """Views with a row stride through the tensor-level calls."""
    g = torch.Generator(device="cuda").manual_seed(1)
    h = T.initialize(2, stream=torch.cuda.current_stream())
    try:
        wide = torch.randn(10, 128, device="cuda", generator=g).bfloat16()
        x, w = wide[:, :96], torch.randn(96, device="cuda", generator=g).bfloat16()
        t64 = x.double()
        unit = t64 / torch.sqrt(t64.square().mean(1, keepdim=True) + 1e-5)
        y = T.rms_norm(x, w, h)
        assert float((y.double() - unit * w.double()).abs().max()) < 0.05
        q, s = T.rms_norm(x, w, h, quantize=True)
        assert q.dtype == torch.float8_e4m3fn
        assert float((q.float() * s[:, None] - y.float()).abs().max()) < 0.5
        dx, dw = T.rms_norm_backward(y, x, w, h)
        assert float((dw.double() - (y.double() * unit).sum(0)).abs().max()) < 1e-3
        # whole numbers: exact
        x = torch.randint(-3, 4, (10, 128), device="cuda", generator=g).bfloat16()[:, :96]
        e = torch.randint(-3, 4, (2, 40, 96), device="cuda", generator=g).bfloat16()
        begin, count = (torch.tensor(v, device="cuda") for v in ([6, 0], [4, 5]))
        out = T.grouped_matmul(x, e, begin, count, h)
        want = torch.zeros(10, 40, device="cuda", dtype=torch.float64)
        want[6:10], want[0:5] = x[6:10].double() @ e[0].double().t(), x[:5].double() @ e[1].double().t()
        assert torch.equal(out, want.bfloat16())
        back = T.grouped_matmul(out, e, begin, count, h, transposed=True)
        want = torch.zeros(10, 96, device="cuda", dtype=torch.float64)
        want[6:10], want[0:5] = out[6:10].double() @ e[0].double(), out[:5].double() @ e[1].double()
        assert torch.equal(back, want.float().bfloat16())
        dw = T.grouped_matmul_weight_grad(out, x, begin, count, h)
        assert torch.equal(dw[0], (out[6:10].double().t() @ x[6:10].double()).float().bfloat16())
        T.check(h)
    finally:
        T.finalize(h)


@pytest.mark.gpu
@pytest.mark.parametrize("skew", ["even", "all to one", "some empty"])
def test_moe_layer_example(T, skew):
    import collective_datapath_atom_gb300 as P
    from collective_datapath_atom_gb300.examples import moe_layer as example

    R, tokens, H, N = 8, 64 * 8, 256, 96
    g = torch.Generator(device="cuda").manual_seed(2)
    # partial sums of whole numbers: the reduced rows are exact
    partials = [torch.randint(-8, 9, (tokens, H), device="cuda", generator=g).bfloat16()
                for _ in range(R)]
    residual = torch.randint(-8, 9, (tokens, H), device="cuda", generator=g).bfloat16()
    weight = torch.ones(H, device="cuda", dtype=torch.bfloat16)
    experts = torch.randn(R, N, H, device="cuda", generator=g).to(torch.float8_e4m3fn)
    expert_scales = torch.rand(R, N, device="cuda", generator=g) + 0.5
    dest = {"even": torch.arange(tokens, device="cuda") % R,
            "all to one": torch.full((tokens,), 5, device="cuda"),
            "some empty": torch.randint(0, 3, (tokens,), device="cuda", generator=g) * 3}[skew]
    ctx = P.purlin_init(R, torch.cuda.current_stream())
    try:
        got = example.moe_layer(ctx, partials, residual, weight, experts, expert_scales, dest)
        P.purlin_check(ctx)
    finally:
        ctx.close()
    total = sum(p.double() for p in partials) + residual.double()
    assert torch.equal(got["total"], total.bfloat16())
    v = total / torch.sqrt(total.square().mean(1, keepdim=True) + 1e-5)
    rows = got["q"].float().double() * got["scales"].double()[:, None]
    # e4m3 rounds to 2^-4 of a value, or half of its smallest step
    bound = torch.maximum(v.abs() * 2.0 ** -4, got["scales"].double()[:, None] * 2.0 ** -10)
    assert bool(((rows - v).abs() <= bound * 1.001).all())
    # the rows that were sent, through their own expert, back in their places
    for d in range(R):
        at = dest == d
        w = experts[d].float().double() * expert_scales[d].double()[:, None]
        y, size = rows[at] @ w.t(), rows[at].abs() @ w.abs().t()
        err = (H + 4) * 2.0 ** -23 * size
        part = got["y"][at]
        assert bool(((part >= (y - err).bfloat16()) & (part <= (y + err).bfloat16())).all())
