"""Means of the norms around a block are quotients by the hidden size on a GPU, not
products with its reciprocal, and elements take the same steps in every kernel.

Rows of small whole numbers, with whole weights, gates and residuals and no eps, have
exact sums in any order.  So a row has the same bits among few rows and many, whichever
kernel has it, and those of the same quotient, root and products made with torch.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_block_norm_gpu import P, ctx  # noqa: E402, F401

# hidden sizes whose binary32 reciprocal is not exact; a warp's rows, rows of one team
# and several, of the teams' four and eight windows a thread, of a block, read again
SIZES = [200, 1100, 1101, 2052, 4099, 7168, 9000, 33000]
FEW, MANY = 5, 640


def whole(*shape, seed, lo=-3, hi=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, device="cuda", generator=g).float()


def root(v):
    """1 / sqrt(mean of squares), the mean a correctly rounded quotient."""
    return (v.square().sum(1, keepdim=True).cpu() / v.shape[1]).cuda().rsqrt()


def head(t, n):
    return t if t is None or t.dim() < 2 else t[:n]


@pytest.mark.parametrize("hidden", SIZES)
@pytest.mark.parametrize("gate", [None, "columns", "rows"])
@pytest.mark.parametrize("quantize", [False, True], ids=["f32", "e4m3"])
def test_the_second_norm(P, ctx, hidden, gate, quantize):  # noqa: F811
    from collective_datapath_atom_gb300 import torch_api

    x, res, w = whole(MANY, hidden, seed=1), whole(MANY, hidden, seed=2), whole(hidden, seed=3, lo=1, hi=4)
    g = None if gate is None else whole(hidden, seed=4) if gate == "columns" else whole(MANY, hidden, seed=4)

    def norm(n):
        got = torch_api.block_norm(x[:n], w, ctx, residual=res[:n], gate=head(g, n), residual_scale=2.0,
                                   block_scale=3.0, eps=0.0, quantize=quantize)
        P.purlin_check(ctx)
        return [v.float() for v in got]

    few, many = norm(FEW), norm(MANY)
    for a, b in zip(few, many):
        assert torch.equal(a, b[:FEW])
    t = 2 * res + 3 * x * (1 if g is None else g)
    assert torch.equal(many[1], t)
    if not quantize:
        assert torch.equal(many[0], t * root(t) * w)


@pytest.mark.parametrize("hidden", SIZES)
@pytest.mark.parametrize("gate", [None, "columns", "rows"])
def test_the_first_norm(P, ctx, hidden, gate):  # noqa: F811
    from collective_datapath_atom_gb300 import torch_api

    x, post = whole(MANY, hidden, seed=5), whole(hidden, seed=6, lo=1, hi=4)
    g = None if gate is None else whole(hidden, seed=7) if gate == "columns" else whole(MANY, hidden, seed=7)

    def total(n):
        got = torch_api.block_norm(x[:n], None, ctx, post_weight=post, gate=head(g, n), block_scale=3.0, eps=0.0)
        P.purlin_check(ctx)
        return got[1]

    few, many = total(FEW), total(MANY)
    assert torch.equal(few, many[:FEW])
    assert torch.equal(many, x * root(x) * (3 * post * (1 if g is None else g)))


@pytest.mark.parametrize("hidden", SIZES)
@pytest.mark.parametrize("gate", [None, "columns", "rows"])
def test_gradients(P, ctx, hidden, gate):  # noqa: F811
    from collective_datapath_atom_gb300 import torch_api

    x, total, dy, dtotal = (whole(MANY, hidden, seed=s) for s in (8, 9, 10, 11))
    w, post = whole(hidden, seed=12, lo=1, hi=4), whole(hidden, seed=13, lo=1, hi=4)
    g = None if gate is None else whole(hidden, seed=14) if gate == "columns" else whole(MANY, hidden, seed=14)

    def gradients(n, dy, post):
        got = torch_api.block_norm_backward(dy[:n], x[:n], total[:n], w, ctx, dtotal=dtotal[:n], post_weight=post,
                                            gate=head(g, n), block_scale=3.0, eps=0.0)
        P.purlin_check(ctx)
        return [got[k] for k in ("dx", "dresidual")] + ([got["dgate"]] if gate == "rows" else [])

    # the second norm's gradient, and (its own being 0: dt is dtotal, whole) the first one's
    for d, p in ((dy, None), (torch.zeros_like(dy), post)):
        for a, b in zip(gradients(FEW, d, p), gradients(MANY, d, p)):
            assert torch.equal(a, b[:FEW])
