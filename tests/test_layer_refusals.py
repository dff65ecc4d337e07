"""Argument checks of the layer operators (RMS norm, grouped products): the
checks that need no context run before it is looked at, so they are tested
here without a GPU, through addresses that are never read."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def P():
    import __graft_entry__

    __graft_entry__.build()
    import collective_datapath_atom_gb300 as P

    return P


INVALID, ALIGNMENT, UNSUPPORTED, ALIAS = 1, 2, 3, 4
A, B, C, D, E, F = (0x10000000 * i for i in range(1, 7))   # buffers far apart


def norm(P, **kw):
    a = dict(x=A, ldx=0, residual=B, ldr=0, weight=C, y=D, ldy=0, total=E, ldt=0, scales=0,
             rows=4, hidden=64, eps=1e-5, dtype=1, out_dtype=1)
    a.update(kw)
    return P.lib.purlin_rms_norm(None, *a.values())


def backward(P, **kw):
    a = dict(dy=A, lddy=0, total=B, ldt=0, weight=C, dtotal=D, lddt=0, dx=E, lddx=0, dweight=F,
             rows=4, hidden=64, eps=1e-5, dtype=1)
    a.update(kw)
    return P.lib.purlin_rms_norm_backward(None, *a.values())


def product(P, **kw):
    a = dict(x=A, ldx=0, w=B, ldw=0, y=C, ldy=0, x_scales=0, w_scales=0, begin=D, count=E,
             groups=2, rows=4, n=32, k=64, dtype=1, layout=0)
    a.update(kw)
    return P.lib.purlin_grouped_matmul(None, *a.values())


def grad(P, **kw):
    a = dict(dy=A, lddy=0, x=B, ldx=0, dw=C, lddw=0, begin=D, count=E, groups=2, rows=4, n=32,
             k=64, dtype=1)
    a.update(kw)
    return P.lib.purlin_grouped_matmul_weight_grad(None, *a.values())


@pytest.mark.parametrize("call", [norm, backward, product, grad])
def test_no_context(P, call):
    # every other argument is right: only the missing context is left to refuse
    assert call(P) == INVALID
    assert call(P, rows=0) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), INVALID), (dict(dtype=7), INVALID),
    (dict(out_dtype=0), UNSUPPORTED), (dict(out_dtype=3), UNSUPPORTED),
    (dict(x=A + 1), ALIGNMENT), (dict(weight=C + 1), ALIGNMENT),
    (dict(dtype=0, out_dtype=0, total=E + 2), ALIGNMENT),
    (dict(out_dtype=2, scales=F + 2), ALIGNMENT),
    (dict(y=E), ALIAS), (dict(y=E + 2), ALIAS), (dict(y=C - 2), ALIAS),
    (dict(y=A + 2), ALIAS), (dict(y=A, ldy=128), ALIAS),
    (dict(total=B, ldt=80), ALIAS), (dict(out_dtype=2, scales=F, y=A), ALIAS),
    (dict(out_dtype=2, scales=A), ALIAS),
])
def test_norm_refusals(P, kw, want):
    assert norm(P, **kw) == want


def test_norm_in_place_and_interleaved_pass_the_alias_check(P):
    # only the missing context refuses these (INVALID, not ALIAS)
    assert norm(P, total=A) == INVALID
    assert norm(P, total=B) == INVALID
    assert norm(P, y=A) == INVALID
    # two column ranges of one buffer: extents interleave, no byte is shared
    assert norm(P, ldx=128, y=A + 128, ldy=128) == INVALID
    assert norm(P, ldx=128, y=A + 126, ldy=128) == ALIAS


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), INVALID), (dict(dy=A + 1), ALIGNMENT), (dict(dweight=F + 2), ALIGNMENT),
    (dict(dx=A + 2), ALIAS), (dict(dx=B, lddx=100), ALIAS), (dict(dx=C), ALIAS),
    (dict(dweight=D), ALIAS), (dict(dweight=E), ALIAS), (dict(dweight=C), ALIAS),
])
def test_backward_refusals(P, kw, want):
    assert backward(P, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=0), UNSUPPORTED), (dict(dtype=5), INVALID), (dict(layout=2), INVALID),
    (dict(dtype=2, layout=1, x_scales=F, w_scales=F + 4096), UNSUPPORTED),
    (dict(x=A + 8), ALIGNMENT), (dict(w=B + 2), ALIGNMENT), (dict(y=C + 1), ALIGNMENT),
    (dict(ldx=68), ALIGNMENT), (dict(ldw=65), ALIGNMENT), (dict(k=63), ALIGNMENT),
    (dict(layout=1, n=33), ALIGNMENT),
    (dict(dtype=2, ldx=72, x_scales=F, w_scales=F + 4096), ALIGNMENT),
    (dict(dtype=2, x_scales=F + 2, w_scales=F + 4096), ALIGNMENT),
    (dict(y=A), ALIAS), (dict(y=B + 64), ALIAS), (dict(y=A - 2), ALIAS),
    (dict(dtype=2, x_scales=C, w_scales=F), ALIAS),
    (dict(begin=C + 8), ALIAS), (dict(count=C + 248), ALIAS),
])
def test_product_refusals(P, kw, want):
    assert product(P, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=0), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype=9), INVALID),
    (dict(dy=A + 4), ALIGNMENT), (dict(x=B + 4), ALIGNMENT), (dict(dw=C + 1), ALIGNMENT),
    (dict(lddy=33), ALIGNMENT), (dict(k=65), ALIGNMENT),
    (dict(dw=A), ALIAS), (dict(dw=B + 2), ALIAS), (dict(begin=C + 8), ALIAS),
    (dict(count=C), ALIAS),
])
def test_grad_refusals(P, kw, want):
    assert grad(P, **kw) == want


# Refusals that share INVALID_ARG with a missing context need one: a GPU.

@pytest.fixture(scope="module")
def ctx(P):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = P.purlin_init(1, torch.cuda.current_stream())
    yield c
    c.close()


@pytest.mark.gpu
def test_invalid_arguments_with_a_context(P, ctx):
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    o = torch.full((4, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(2, 64, 64, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros(64, device="cuda", dtype=torch.bfloat16)
    i = torch.zeros(2, device="cuda", dtype=torch.int64)
    f = torch.zeros(128, device="cuda")
    p = lambda x: x.data_ptr()   # noqa: E731

    def refused(status):
        assert status == INVALID

    def n(**kw):
        a = dict(x=p(t), ldx=0, residual=0, ldr=0, weight=p(v), y=p(o), ldy=0, total=0, ldt=0,
                 scales=0, rows=4, hidden=64, eps=1e-5, dtype=1, out_dtype=1)
        a.update(kw)
        return P.lib.purlin_rms_norm(ctx.handle, *a.values())

    for kw in (dict(x=0), dict(weight=0), dict(y=0), dict(hidden=0), dict(ldx=63), dict(ldy=1),
               dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(scales=p(f)),
               dict(out_dtype=2), dict(rows=1 << 31), dict(hidden=1 << 31)):
        refused(n(**kw))

    def m(**kw):
        a = dict(x=p(t), ldx=0, w=p(w), ldw=0, y=p(o), ldy=0, x_scales=0, w_scales=0, begin=p(i),
                 count=p(i), groups=2, rows=4, n=64, k=64, dtype=1, layout=0)
        a.update(kw)
        return P.lib.purlin_grouped_matmul(ctx.handle, *a.values())

    for kw in (dict(x=0), dict(w=0), dict(y=0), dict(begin=0), dict(count=0), dict(k=0),
               dict(groups=-1), dict(groups=1025), dict(ldx=56), dict(ldw=32), dict(ldy=63),
               dict(begin=p(i) + 4), dict(x_scales=p(f)), dict(dtype=2), dict(rows=1 << 31)):
        refused(m(**kw))

    def g(**kw):
        a = dict(dy=p(t), lddy=0, x=p(t), ldx=0, dw=p(w), lddw=0, begin=p(i), count=p(i),
                 groups=2, rows=4, n=64, k=64, dtype=1)
        a.update(kw)
        return P.lib.purlin_grouped_matmul_weight_grad(ctx.handle, *a.values())

    for kw in (dict(dy=0), dict(x=0), dict(dw=0), dict(begin=0), dict(count=0), dict(groups=1025),
               dict(lddy=56), dict(lddw=8)):
        refused(g(**kw))

    def b(**kw):
        a = dict(dy=p(t), lddy=0, total=p(t), ldt=0, weight=p(v), dtotal=0, lddt=0, dx=p(o),
                 lddx=0, dweight=p(f), rows=4, hidden=64, eps=1e-5, dtype=1)
        a.update(kw)
        return P.lib.purlin_rms_norm_backward(ctx.handle, *a.values())

    for kw in (dict(dy=0), dict(total=0), dict(weight=0), dict(dx=0), dict(dweight=0),
               dict(hidden=0), dict(eps=-1e-9), dict(lddx=63)):
        refused(b(**kw))
    P.purlin_check(ctx)
    assert bool((o == 7.0).all())   # nothing was written


@pytest.mark.gpu
def test_errors_raise_in_python(P, ctx):
    torch = pytest.importorskip("torch")
    t = torch.zeros(2, 64, device="cuda")
    with pytest.raises(P.PurlinError) as e:
        P.purlin_rms_norm(ctx, t, t[0], t[1:], 1, 0, 1e-5, P.PURLIN_F32)
    assert e.value.status == INVALID
    assert isinstance(P.lib, ctypes.CDLL)
