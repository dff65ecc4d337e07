"""Gradients of the norms around a block for rows far from 1, on a GPU, against
autograd in 64 bits.

r = 1 / rms(t) of such a row is an ordinary number, its cube, or its square times a
small gradient, is not: the result has to be right wherever it is an ordinary number
itself, in every kernel that the number of rows and their length lead to.  The gradient
dy has a share along t, whose projection is what the cube took away.  Tolerances are
those of test_block_norm_gpu.py: relative, and derived there for rows of any size.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_block_norm_gpu import T, P, backward_errors, ctx, mean, near, randn  # noqa: E402, F401

# largest values of total, x and dy, and eps
SCALES = [(1e13, 1.0, 1.0, 1e-5), (1e15, 1.0, 1.0, 1e-5), (1e15, 1e15, 1e-9, 1e-5), (1e16, 1.0, 1e-6, 1e-5),
          (1e-13, 1.0, 1.0, 0.0), (1e-14, 1e-14, 1.0, 0.0), (1e-18, 1.0, 1e-6, 0.0), (1.0, 1e-18, 1e-9, 0.0)]

# a warp and a block a row; teams with two windows a thread, four, eight, and four with
# fewer warps; rows past them; rows past the registers
SHAPES = [(0, 100, 200), (0, 100, 1024), (0, 300, 1024), (0, 300, 1021), (0, 300, 5120), (0, 300, 9000),
          (0, 5003, 2048), (0, 160, 16390), (0, 2, 33000), (1, 100, 1024), (1, 300, 1024), (1, 300, 1021),
          (1, 300, 9000), (1, 5003, 4096), (1, 2, 33000)]


def backward64(i, dy, total, a, b, eps):
    """Gradients by autograd in 64 bits, the second norm's at `total` and then the first
    one's (a constant that moved t there would round it to the other's steps)."""
    leaf = {k: v.double().requires_grad_(True) for k, v in i.items()}
    t = total.double().requires_grad_(True)
    (t / torch.sqrt(mean(t.square()) + eps) * leaf["weight"] * dy.double()).sum().backward()
    u = leaf["x"] / torch.sqrt(mean(leaf["x"].square()) + eps) * leaf["post_weight"] * leaf["gate"]
    (b * u * t.grad).sum().backward()
    return {**{k: v.grad for k, v in leaf.items()}, "residual": a * t.grad}


@pytest.mark.parametrize("dtype,rows,hidden", SHAPES)
@pytest.mark.parametrize("total_scale,x_scale,dy_scale,eps", SCALES)
def test_backward_of_large_and_small_rows(P, ctx, dtype, rows, hidden, total_scale, x_scale, dy_scale, eps):  # noqa: F811
    from collective_datapath_atom_gb300 import torch_api

    dt = T[dtype]
    t1 = randn(rows, hidden, seed=1, dtype=torch.float32)
    total, x = (t1 * total_scale).to(dt), randn(rows, hidden, seed=2, dtype=dt, scale=x_scale)
    dy = ((randn(rows, hidden, seed=3, dtype=torch.float32) + t1) * dy_scale).to(dt)
    for gate in (["columns", "rows"] if rows < 5000 else ["columns"]):
        i = dict(x=x, weight=randn(hidden, seed=4, dtype=dt), post_weight=randn(hidden, seed=5, dtype=dt),
                 gate=randn(hidden, seed=6, dtype=dt) if gate == "columns" else randn(rows, hidden, seed=6, dtype=dt))
        got = torch_api.block_norm_backward(dy, x, total, i["weight"], ctx, post_weight=i["post_weight"],
                                            gate=i["gate"], residual_scale=0.9, block_scale=0.25, eps=eps)
        P.purlin_check(ctx)
        want = backward64(i, dy, total, 0.9, 0.25, eps)
        err = backward_errors(i, dy, None, total, 0.9, 0.25, gate == "rows", eps)
        for name, key in (("dx", "x"), ("dresidual", "residual"), ("dweight", "weight"),
                          ("dpost_weight", "post_weight"), ("dgate", "gate")):
            near(got[name], want[key], err[name])
