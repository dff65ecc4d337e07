"""The rows' way to their experts and back for batches that take the kernels' forms for
many tokens on a GPU: a block with all of a token's places in the way back's gradient,
four windows a thread in the copies.  Against plain indexing, with the tolerances of
test_expert_rows_gpu.py."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_expert_rows_gpu import HALF, T, U, P, ctx, guards_stand, matrix, places  # noqa: E402, F401


@pytest.mark.parametrize("dtype", [0, 1, 2], ids=["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("tokens,cols", [(1300, 4100), (1300, 4099), (5003, 4099), (2500, 4096), (6000, 7168)])
@pytest.mark.parametrize("pitch,offset", [(0, 0), (16, 16), (3, 1)])
def test_dispatch(P, ctx, tokens, cols, dtype, pitch, offset):  # noqa: F811
    k, rows = 2, 2 * tokens + 100
    place = places(tokens, k, rows, tokens + cols)
    _, x = matrix(tokens, cols, dtype, 1, pitch, offset)
    t, out = matrix(rows, cols, dtype, 2, pitch, offset)
    want = out.float().clone()
    scales, out_scales = torch.rand(tokens, device="cuda"), torch.full((rows + 1,), -5.0, device="cuda")
    want_scales = out_scales.clone()
    P.purlin_dispatch_rows(ctx, x, place, out, tokens, k, cols, rows, dtype, scales=scales, out_scales=out_scales,
                           ldx=x.stride(0), ldo=out.stride(0))
    P.purlin_check(ctx)
    real = (place >= 0) & (place < rows)
    token = torch.arange(tokens, device="cuda")[:, None].expand(tokens, k)[real]
    want[place[real].long()] = x.float()[token]
    want_scales[place[real].long()] = scales[token]
    assert torch.equal(out.float(), want) and torch.equal(out_scales, want_scales)
    assert guards_stand(t, out, offset)


@pytest.mark.parametrize("dtype", [0, 1], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens,k,cols", [(1000, 3, 130), (1003, 8, 1021), (700, 8, 1024), (650, 5, 4100), (2000, 1, 64)])
@pytest.mark.parametrize("pitch,offset", [(0, 0), (8, 8), (3, 1)])
def test_combine_and_its_gradient(P, ctx, tokens, k, cols, dtype, pitch, offset):  # noqa: F811
    rows = tokens * k + 50
    place = places(tokens, k, rows, tokens + cols)
    place[7] = -1                                     # a token that was dropped everywhere
    _, r = matrix(rows, cols, dtype, 3, pitch, offset)
    _, dy = matrix(tokens, cols, dtype, 4, pitch, offset)
    w = torch.randn(tokens, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    real = (place >= 0) & (place < rows)
    at = torch.where(real, place, 0).long()
    picked = torch.where(real[:, :, None], r.double()[at], 0.0)

    t, y = matrix(tokens, cols, dtype, 6, pitch, offset)
    P.purlin_combine_rows(ctx, r, place, y, tokens, k, cols, rows, dtype, weights=w, ldr=r.stride(0), ldy=y.stride(0))
    P.purlin_check(ctx)
    terms = picked * w.double()[:, :, None]
    err = terms.abs().sum(1) * (k + 1) * U
    want = terms.sum(1)
    assert bool(((y.double() - want).abs() <= err + (want.abs() + err) * HALF[dtype] + 1e-38).all())
    assert guards_stand(t, y, offset)

    t, d = matrix(rows, cols, dtype, 7, pitch, offset)
    before, dw = d.clone(), torch.full((tokens, k), 9.0, device="cuda")
    P.purlin_combine_rows_backward(ctx, dy, r, place, w, d, dw, tokens, k, cols, rows, dtype,
                                   lddy=dy.stride(0), ldr=r.stride(0), lddr=d.stride(0))
    P.purlin_check(ctx)
    prod = picked * dy.double()[:, None, :]
    assert bool(((dw.double() - prod.sum(2)).abs() <= prod.abs().sum(2) * (cols + 1) * U).all())
    named = torch.zeros(rows, dtype=torch.bool, device="cuda")
    named[at[real]] = True
    assert torch.equal(d[~named], before[~named])
    full = (w.double()[:, :, None] * dy.double()[:, None, :])[real]
    assert bool(((d.double()[at[real]] - full).abs() <= full.abs() * (U + HALF[dtype]) * 1.01 + 1e-38).all())
    assert guards_stand(t, d, offset)
    dw2 = torch.empty_like(dw)
    P.purlin_combine_rows_backward(ctx, dy, r, place, w, r, dw2, tokens, k, cols, rows, dtype,
                                   lddy=dy.stride(0), ldr=r.stride(0), lddr=r.stride(0))
    P.purlin_check(ctx)
    assert torch.equal(dw, dw2) and torch.equal(r[named], d[named])    # in place of the rows
