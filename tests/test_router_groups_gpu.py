"""Groups of experts whose value is the sum of two choices of opposite signs, on a GPU,
against the definition in 64 bits.

A bias of B on one expert of a group and of -B on the other leave the sum of their scores
as the group's value, while each choice carries binary32's rounding of B: which groups are
kept has to be told by how large the choices are, not their sum.  The rows are such that
64 bits tell every border apart.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_router_gpu import P, ctx, reference, run  # noqa: E402, F401


@pytest.mark.parametrize("scores", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [10.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("each", [2, 4])
def test_opposite_biases_in_a_group(P, ctx, scores, size, each):  # noqa: F811
    r = dict(experts=8 * each, top_k=4, scores=scores, groups=8, top_groups=4, group_top=2)
    g = torch.Generator().manual_seed(each)
    l = torch.randn(20000, 8 * each, generator=g)
    bias = torch.tensor([size, -size] + [-2 * size] * (each - 2)).repeat(8)
    chosen = run(P, ctx, l.cuda(), bias.cuda(), r, 0)[1]
    want, s = reference(l.double(), bias.double(), r)
    # the four chosen are the kept groups' first experts; 64 bits have size * 2^-53 a sum
    value = (s + bias.double()).view(-1, 8, each)[:, :, :2].sum(2).sort(1, descending=True).values
    order = s.gather(1, want).diff(dim=1).abs().amin(1)
    clear = (value[:, 3] - value[:, 4] > size * 2.0 ** -50) & (order > size * 2.0 ** -50)
    assert float(clear.double().mean()) > 0.99
    assert bool((want % each == 0).all())
    assert torch.equal(chosen[clear], want[clear])
