"""Which overlaps between a norm's buffers are refused, on the CPU: the checks
run before the context is looked at, so a call without one returns INVALID_ARG
where every other argument is right, and nothing behind an address is read."""
import pytest

INVALID, ALIAS = 1, 4
A, B, C, D, E, F = (0x10000000 * i for i in range(1, 7))
F32, BF16, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def P():
    import __graft_entry__

    __graft_entry__.build()
    import collective_datapath_atom_gb300 as P

    return P


def norm(P, **kw):
    a = dict(x=A, ldx=0, residual=B, ldr=0, weight=C, y=D, ldy=0, total=E, ldt=0, scales=F,
             rows=64, hidden=64, eps=1e-5, dtype=F32, out_dtype=E4M3)
    a.update(kw)
    return P.lib.purlin_rms_norm(None, *a.values())


# a vector of scales as long as a row of x: the same extent as x's first row, but the
# blocks of other rows write it
@pytest.mark.parametrize("dtype,rows,hidden", [(F32, 64, 64), (BF16, 64, 128), (F32, 63, 64),
                                               (F32, 1, 1), (F32, 1, 64)])
@pytest.mark.parametrize("into", [A, B, C, A + 16, A - 4])
def test_scales_over_an_input_are_refused(P, dtype, rows, hidden, into):
    if into == A + 16 and rows * hidden == 1 or into == A - 4 and rows == 1:
        return   # past the only element, or before it
    assert norm(P, dtype=dtype, rows=rows, hidden=hidden) == INVALID
    assert norm(P, dtype=dtype, rows=rows, hidden=hidden, scales=into) == ALIAS


def test_results_over_their_inputs_pass(P):
    kw = dict(out_dtype=F32, scales=0)
    for extra in (dict(y=A), dict(y=B), dict(total=A), dict(total=B), dict(y=A, total=B)):
        assert norm(P, **kw, **extra) == INVALID
    assert norm(P, **kw, y=A, ldy=128) == ALIAS
