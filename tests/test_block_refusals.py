"""Argument checks of the norms around a block, the router, the order by expert and
the rows' way there and back: checks that need no context run before it is looked
at, so they are tested here without a GPU, through addresses that are never read."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def P():
    import __graft_entry__

    __graft_entry__.build()
    import collective_datapath_atom_gb300 as P

    return P


INVALID, ALIGNMENT, UNSUPPORTED, ALIAS = 1, 2, 3, 4
A, B, C, D, E, F, G, H, I, J, K, L = (0x10000000 * i for i in range(1, 13))   # far apart
INF, NAN = float("inf"), float("nan")


def norm(P, **kw):
    a = dict(x=A, ldx=0, post=B, gate=C, ldg=0, layout=0, block_scale=0.5, residual=D, ldr=0,
             residual_scale=1.0, weight=E, y=F, ldy=0, total=G, ldt=0, scales=0, rows=4, hidden=64,
             eps=1e-5, dtype=1, out_dtype=1)
    a.update(kw)
    return P.lib.purlin_block_norm(None, *a.values())


def backward(P, **kw):
    a = dict(dy=A, lddy=0, dtotal=B, lddt=0, x=C, ldx=0, total=D, ldt=0, post=E, gate=F, ldg=0,
             layout=0, block_scale=0.5, residual_scale=1.0, weight=G, dx=H, lddx=0, dresidual=I,
             lddr=0, dpost=J, dgate=K, lddg=0, dweight=L, rows=4, hidden=64, eps=1e-5, dtype=1)
    a.update(kw)
    return P.lib.purlin_block_norm_backward(None, *a.values())


ROUTER = dict(experts=64, top_k=6, scores=1, groups=8, top_groups=4, group_top=2, renormalise=1,
              scale=2.5)


def route(P, router=None, **kw):
    a = dict(logits=A, ld=0, bias=B, weights=C, chosen=D, tokens=4,
             router=ctypes.byref(P.purlin_router(**{**ROUTER, **(router or {})})), dtype=0)
    a.update(kw)
    return P.lib.purlin_route(None, *a.values())


def route_backward(P, router=None, **kw):
    a = dict(dweights=A, logits=B, ld=0, chosen=C, dlogits=D, ldd=0, tokens=4,
             router=ctypes.byref(P.purlin_router(**{**ROUTER, **(router or {})})), dtype=0)
    a.update(kw)
    return P.lib.purlin_route_backward(None, *a.values())


def order(P, **kw):
    a = dict(chosen=A, place=B, begin=C, count=D, slots=24, groups=8, capacity=0)
    a.update(kw)
    return P.lib.purlin_expert_order(None, *a.values())


def dispatch(P, **kw):
    a = dict(x=A, ldx=0, scales=B, place=C, out=D, ldo=0, out_scales=E, tokens=4, top_k=6, cols=64,
             out_rows=24, dtype=2)
    a.update(kw)
    return P.lib.purlin_dispatch_rows(None, *a.values())


def combine(P, **kw):
    a = dict(rows=A, ldr=0, weights=B, place=C, shared=D, lds=0, y=E, ldy=0, tokens=4, top_k=6,
             cols=64, n_rows=24, dtype=1)
    a.update(kw)
    return P.lib.purlin_combine_rows(None, *a.values())


def combine_backward(P, **kw):
    a = dict(dy=A, lddy=0, rows=B, ldr=0, weights=C, place=D, drows=E, lddr=0, dweights=F, tokens=4,
             top_k=6, cols=64, n_rows=24, dtype=1)
    a.update(kw)
    return P.lib.purlin_combine_rows_backward(None, *a.values())


CALLS = [norm, backward, route, route_backward, order, dispatch, combine, combine_backward]


@pytest.mark.parametrize("call", CALLS)
def test_no_context(P, call):
    # every other argument is right: only the missing context is left to refuse
    assert call(P) == INVALID
    size = {norm: "rows", backward: "rows", order: "slots"}.get(call, "tokens")
    assert call(P, **{size: 0}) == INVALID


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), INVALID), (dict(dtype=9), INVALID), (dict(out_dtype=0), UNSUPPORTED),
    (dict(hidden=0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(block_scale=INF), INVALID), (dict(residual_scale=NAN), INVALID),
    (dict(layout=2), INVALID), (dict(ldx=63), INVALID), (dict(layout=1, ldg=63), INVALID),
    (dict(x=0), INVALID), (dict(y=0), INVALID), (dict(weight=0), INVALID),
    (dict(weight=0, y=0, total=0), INVALID), (dict(out_dtype=2), INVALID), (dict(scales=H), INVALID),
    (dict(weight=0, y=0, out_dtype=2, scales=H), INVALID),
    (dict(x=A + 1), ALIGNMENT), (dict(gate=C + 1), ALIGNMENT), (dict(post=B + 1), ALIGNMENT),
    (dict(dtype=0, out_dtype=0, total=G + 2), ALIGNMENT), (dict(out_dtype=2, scales=H + 2), ALIGNMENT),
    (dict(y=G), ALIAS), (dict(y=G + 2), ALIAS), (dict(y=A + 2), ALIAS), (dict(y=A, ldy=128), ALIAS),
    (dict(total=D, ldt=80), ALIAS), (dict(total=C), ALIAS), (dict(y=B - 2), ALIAS),
    (dict(y=E), ALIAS), (dict(layout=1, total=C), ALIAS), (dict(out_dtype=2, scales=H, y=A), ALIAS),
    (dict(out_dtype=2, scales=D), ALIAS),
])
def test_norm_refusals(P, kw, want):
    assert norm(P, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(total=A), dict(total=D), dict(y=A), dict(y=D, total=A), dict(residual=0), dict(post=0),
    dict(gate=0, ldg=1), dict(weight=0, y=0), dict(ldg=1), dict(layout=1),
    dict(ldx=128, y=A + 128, ldy=128),      # two column ranges of one buffer
])
def test_norm_what_passes_the_checks(P, kw):
    # the missing context is all that is left to refuse
    assert norm(P, **kw) == INVALID
    assert norm(P, **{**kw, "total": kw.get("total", G) + 1}) == ALIGNMENT


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), INVALID), (dict(layout=-1), INVALID), (dict(block_scale=NAN), INVALID),
    (dict(dweight=0), INVALID), (dict(weight=0), INVALID), (dict(dpost=0), INVALID),
    (dict(post=0), INVALID), (dict(dgate=0), INVALID), (dict(gate=0), INVALID),
    (dict(weight=0, dweight=0), INVALID), (dict(weight=0, dweight=0, dy=0, total=0, dtotal=0), INVALID),
    (dict(dx=0), INVALID), (dict(x=0), INVALID), (dict(dy=0), INVALID), (dict(lddr=10), INVALID),
    (dict(dy=A + 1), ALIGNMENT), (dict(dweight=L + 2), ALIGNMENT), (dict(dgate=K + 2), ALIGNMENT),
    (dict(layout=1, dgate=K + 1), ALIGNMENT), (dict(dpost=J + 1), ALIGNMENT),
    (dict(dx=I), ALIAS), (dict(dx=A + 2), ALIAS), (dict(dx=C, lddx=100), ALIAS), (dict(dx=G), ALIAS),
    (dict(dresidual=E), ALIAS), (dict(dweight=J), ALIAS), (dict(dpost=K), ALIAS),
    (dict(dgate=A), ALIAS), (dict(dweight=C), ALIAS), (dict(layout=1, dgate=H), ALIAS),
    (dict(layout=1, dgate=F + 2), ALIAS), (dict(dx=F), ALIAS), (dict(dresidual=L), ALIAS),
])
def test_backward_refusals(P, kw, want):
    assert backward(P, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(dx=A, dresidual=B), dict(dx=C, dresidual=D), dict(layout=1, dgate=F), dict(dresidual=0),
    dict(weight=0, dweight=0, dy=0, total=0), dict(post=0, dpost=0), dict(gate=0, dgate=0),
    dict(dtotal=0), dict(layout=1, lddg=128),
])
def test_backward_what_passes_the_checks(P, kw):
    assert backward(P, **kw) == INVALID
    assert backward(P, **{**kw, "x": C + 1}) == ALIGNMENT


@pytest.mark.parametrize("call", [route, route_backward])
@pytest.mark.parametrize("router,want", [
    (dict(experts=0), INVALID), (dict(experts=1025, groups=1), INVALID), (dict(top_k=0), INVALID),
    (dict(top_k=33), INVALID), (dict(scores=2), INVALID), (dict(groups=-1), INVALID),
    (dict(groups=7), INVALID), (dict(top_groups=0), INVALID), (dict(top_groups=9), INVALID),
    (dict(top_groups=1, top_k=9), INVALID), (dict(group_top=-1), INVALID),
    (dict(renormalise=2), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(group_top=3), UNSUPPORTED), (dict(groups=1, top_k=33), UNSUPPORTED),
    (dict(groups=64, top_groups=64), UNSUPPORTED),
])
def test_router_refusals(P, call, router, want):
    assert call(P, router=router, **({"logits": 0} if want == UNSUPPORTED else {})) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=5), INVALID), (dict(router=None), INVALID),
    (dict(ld=63), INVALID), (dict(logits=0), INVALID), (dict(weights=0), INVALID),
    (dict(chosen=0), INVALID), (dict(tokens=1 << 31), INVALID), (dict(logits=A + 2), ALIGNMENT),
    (dict(dtype=1, logits=A + 1), ALIGNMENT), (dict(bias=B + 2), ALIGNMENT),
    (dict(weights=C + 1), ALIGNMENT), (dict(chosen=D + 2), ALIGNMENT), (dict(weights=A), ALIAS),
    (dict(weights=D + 4), ALIAS), (dict(chosen=B), ALIAS), (dict(chosen=A + 1020), ALIAS),
])
def test_route_refusals(P, kw, want):
    if "router" in kw:
        assert P.lib.purlin_route(None, A, 0, B, C, D, 4, None, 0) == want
    else:
        assert route(P, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), UNSUPPORTED), (dict(ldd=63), INVALID), (dict(dweights=0), INVALID),
    (dict(dlogits=0), INVALID), (dict(dlogits=D + 2), ALIGNMENT), (dict(dlogits=B + 4), ALIAS),
    (dict(dlogits=B, ldd=80), ALIAS), (dict(dlogits=A), ALIAS), (dict(dlogits=C - 4), ALIAS),
    (dict(dlogits=B), INVALID),       # in place: the context alone is missing
])
def test_route_backward_refusals(P, kw, want):
    assert route_backward(P, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(groups=1025), INVALID), (dict(groups=-1), INVALID), (dict(slots=1 << 31), INVALID),
    (dict(capacity=1 << 29), INVALID), (dict(capacity=1 << 62), INVALID), (dict(chosen=0), INVALID),
    (dict(place=0), INVALID), (dict(begin=0), INVALID), (dict(count=0), INVALID),
    (dict(chosen=A + 2), ALIGNMENT), (dict(begin=C + 4), ALIGNMENT), (dict(count=D + 4), ALIGNMENT),
    (dict(place=A), ALIAS), (dict(begin=A + 88), ALIAS), (dict(count=C + 56), ALIAS),
    (dict(count=B), ALIAS),
])
def test_order_refusals(P, kw, want):
    assert order(P, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=3), INVALID), (dict(top_k=0), INVALID), (dict(top_k=33), INVALID),
    (dict(tokens=1 << 31), INVALID), (dict(cols=1 << 31), INVALID), (dict(out_rows=1 << 31), INVALID),
    (dict(ldx=63), INVALID), (dict(ldo=63), INVALID), (dict(scales=0), INVALID),
    (dict(out_scales=0), INVALID), (dict(x=0), INVALID), (dict(place=0), INVALID),
    (dict(out=0), INVALID), (dict(dtype=1, x=A + 1), ALIGNMENT), (dict(dtype=0, out=D + 2), ALIGNMENT),
    (dict(scales=B + 1), ALIGNMENT), (dict(place=C + 2), ALIGNMENT), (dict(out=A), ALIAS),
    (dict(out=A + 255), ALIAS), (dict(out_scales=A), ALIAS), (dict(out_scales=B), ALIAS),
    (dict(out_scales=D), ALIAS), (dict(out=C), ALIAS),
])
def test_dispatch_refusals(P, kw, want):
    assert dispatch(P, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), INVALID), (dict(top_k=33), INVALID),
    (dict(ldr=63), INVALID), (dict(lds=63), INVALID), (dict(ldy=63), INVALID), (dict(place=0), INVALID),
    (dict(y=0), INVALID), (dict(rows=0), INVALID), (dict(rows=A + 1), ALIGNMENT),
    (dict(weights=B + 2), ALIGNMENT), (dict(y=A), ALIAS), (dict(y=D + 2), ALIAS),
    (dict(y=D, ldy=80), ALIAS), (dict(y=B), ALIAS), (dict(y=C), ALIAS),
    (dict(y=D), INVALID),             # in place of shared: the context alone is missing
])
def test_combine_refusals(P, kw, want):
    assert combine(P, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), UNSUPPORTED), (dict(top_k=0), INVALID), (dict(lddy=63), INVALID),
    (dict(weights=0), INVALID), (dict(dweights=0), INVALID), (dict(dy=0), INVALID),
    (dict(drows=0), INVALID), (dict(drows=E + 1), ALIGNMENT), (dict(dweights=F + 2), ALIGNMENT),
    (dict(drows=A), ALIAS), (dict(drows=B + 2), ALIAS), (dict(drows=B, lddr=80), ALIAS),
    (dict(dweights=C), ALIAS), (dict(dweights=B), ALIAS), (dict(drows=F), ALIAS),
    (dict(drows=B), INVALID),         # in place of rows: the context alone is missing
])
def test_combine_backward_refusals(P, kw, want):
    assert combine_backward(P, **kw) == want
