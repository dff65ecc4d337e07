// block_api.cpp -- host side of the norms around a block (include/purlin.h,
// "layer operators"; kernels in block_norm.cu): argument checks, the workspace
// and the launches.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>

#include "checks.h"
#include "host.h"
#include "layers.h"

using namespace purlin;
using namespace purlin::host;

namespace {

bool bad_extents(size_t rows, size_t hidden, float eps, float block_scale, float residual_scale,
                 purlin_gate_layout layout) {
    return hidden == 0 || hidden > kMaxExtent / 2 || rows > kMaxExtent || !(eps >= 0) ||
           !std::isfinite(eps) || !std::isfinite(block_scale) || !std::isfinite(residual_scale) ||
           (layout != PURLIN_GATE_COLUMNS && layout != PURLIN_GATE_ROWS);
}

// `out` may be any of `inputs`, element for element, and shares nothing else with them.
bool clashes(const Matrix &out, std::initializer_list<Matrix> inputs) {
    for (const Matrix &m : inputs)
        if (overlap(out, m) && !same(out, m)) return true;
    return false;
}

}  // namespace

extern "C" {

purlin_status purlin_block_norm(purlin_ctx *ctx, const void *x, size_t ldx,
                                const void *post_weight, const void *gate, size_t ldg,
                                purlin_gate_layout gate_layout, float block_scale,
                                const void *residual, size_t ldr, float residual_scale,
                                const void *weight, void *y, size_t ldy, void *total, size_t ldt,
                                float *scales, size_t rows, size_t hidden, float eps,
                                purlin_dtype dtype, purlin_dtype out_dtype) {
    if (dtype != PURLIN_F32 && dtype != PURLIN_BF16) return PURLIN_ERR_INVALID_ARG;
    if (out_dtype != dtype && out_dtype != PURLIN_E4M3) return PURLIN_ERR_UNSUPPORTED;
    if (bad_extents(rows, hidden, eps, block_scale, residual_scale, gate_layout))
        return PURLIN_ERR_INVALID_ARG;
    const bool gate_rows = gate != nullptr && gate_layout == PURLIN_GATE_ROWS;
    ldx = ldx ? ldx : hidden;
    ldg = gate_rows && ldg ? ldg : hidden;
    ldr = ldr ? ldr : hidden;
    ldy = ldy ? ldy : hidden;
    ldt = ldt ? ldt : hidden;
    for (size_t ld : {ldx, ldg, ldr, ldy, ldt})
        if (bad_ld(ld, hidden)) return PURLIN_ERR_INVALID_ARG;
    if (rows == 0) return ctx ? PURLIN_OK : PURLIN_ERR_INVALID_ARG;
    if (x == nullptr || (weight != nullptr) != (y != nullptr) ||
        (y == nullptr && (total == nullptr || out_dtype != dtype)) ||
        (scales != nullptr) != (out_dtype == PURLIN_E4M3))
        return PURLIN_ERR_INVALID_ARG;
    const size_t es = (size_t)size_of(dtype);
    for (const void *p : {x, post_weight, gate, residual, weight, (const void *)total})
        if (misaligned(p, es)) return PURLIN_ERR_ALIGNMENT;
    if (misaligned(y, (size_t)size_of(out_dtype)) || misaligned(scales, 4))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix mx = matrix(x, rows, hidden, ldx, dtype);
    const Matrix mr = matrix(residual, rows, hidden, ldr, dtype);
    const Matrix mp = matrix(post_weight, 1, hidden, hidden, dtype);
    const Matrix mg = matrix(gate, gate_rows ? rows : 1, hidden, ldg, dtype);
    const Matrix mw = matrix(weight, 1, hidden, hidden, dtype);
    const Matrix my = matrix(y, rows, hidden, ldy, out_dtype);
    const Matrix mt = matrix(total, rows, hidden, ldt, dtype);
    const Matrix ms = matrix(scales, 1, rows, rows, PURLIN_F32);
    for (const Matrix &o : {my, mt})
        if (any_overlap(o, {mp, mg, mw}) || clashes(o, {mx, mr})) return PURLIN_ERR_ALIAS;
    if (any_overlap(ms, {mx, mr, mp, mg, mw, my, mt}) || overlap(my, mt)) return PURLIN_ERR_ALIAS;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;

    BlockNormArgs a;
    a.x = x;
    a.post_weight = post_weight;
    a.gate = gate;
    a.residual = residual;
    a.weight = weight;
    a.y = y;
    a.total = total;
    a.scales = scales;
    a.ldx = ldx;
    a.ldg = ldg;
    a.ldr = ldr;
    a.ldy = ldy;
    a.ldt = ldt;
    a.gate_rows = gate_rows;
    a.block_scale = block_scale;
    a.residual_scale = residual_scale;
    a.rows = rows;
    a.hidden = hidden;
    a.eps = eps;
    a.dtype = dtype;
    a.out_dtype = out_dtype;
    a.sms = ctx->sms;
    a.err = ctx->err;
    a.stream = ctx->stream;
    return done(launch_block_norm(a));
}

purlin_status purlin_block_norm_backward(purlin_ctx *ctx, const void *dy, size_t lddy,
                                         const void *dtotal, size_t lddt, const void *x,
                                         size_t ldx, const void *total, size_t ldt,
                                         const void *post_weight, const void *gate, size_t ldg,
                                         purlin_gate_layout gate_layout, float block_scale,
                                         float residual_scale, const void *weight, void *dx,
                                         size_t lddx, void *dresidual, size_t lddr,
                                         float *dpost_weight, void *dgate, size_t lddg,
                                         float *dweight, size_t rows, size_t hidden, float eps,
                                         purlin_dtype dtype) {
    if (dtype != PURLIN_F32 && dtype != PURLIN_BF16) return PURLIN_ERR_INVALID_ARG;
    if (bad_extents(rows, hidden, eps, block_scale, residual_scale, gate_layout))
        return PURLIN_ERR_INVALID_ARG;
    const bool gate_rows = gate != nullptr && gate_layout == PURLIN_GATE_ROWS;
    lddy = lddy ? lddy : hidden;
    lddt = lddt ? lddt : hidden;
    ldx = ldx ? ldx : hidden;
    ldt = ldt ? ldt : hidden;
    ldg = gate_rows && ldg ? ldg : hidden;
    lddx = lddx ? lddx : hidden;
    lddr = lddr ? lddr : hidden;
    lddg = gate_rows && lddg ? lddg : hidden;
    for (size_t ld : {lddy, lddt, ldx, ldt, ldg, lddx, lddr, lddg})
        if (bad_ld(ld, hidden)) return PURLIN_ERR_INVALID_ARG;
    // without rows the matrices may be missing, and which there are goes by the vectors
    const bool normed = weight != nullptr, any = rows > 0;
    if ((dweight != nullptr) != normed || (dpost_weight != nullptr) != (post_weight != nullptr) ||
        (dgate != nullptr) != (gate != nullptr) ||
        (!normed && (dy != nullptr || total != nullptr)) ||
        (any && (x == nullptr || dx == nullptr ||
                 (normed ? dy == nullptr || total == nullptr : dtotal == nullptr))))
        return PURLIN_ERR_INVALID_ARG;
    const size_t es = (size_t)size_of(dtype);
    for (const void *p : {dy, dtotal, x, total, post_weight, gate, weight, (const void *)dx,
                          (const void *)dresidual})
        if (misaligned(p, es)) return PURLIN_ERR_ALIGNMENT;
    if (misaligned(dgate, gate_rows ? es : 4) || misaligned(dpost_weight, 4) ||
        misaligned(dweight, 4))
        return PURLIN_ERR_ALIGNMENT;
    const auto full = [&](const void *p, size_t ld) { return matrix(p, rows, hidden, ld, dtype); };
    const auto row = [&](const void *p, int type) { return matrix(p, 1, hidden, hidden, type); };
    const Matrix none;
    const Matrix mdy = full(dy, lddy), mdt = full(dtotal, lddt), mx = full(x, ldx);
    const Matrix mt = full(total, ldt), mgr = gate_rows ? full(gate, ldg) : none;
    const Matrix mgc = gate_rows ? none : row(gate, dtype), mp = row(post_weight, dtype);
    const Matrix mw = row(weight, dtype);
    const Matrix odx = full(dx, lddx), odr = full(dresidual, lddr);
    const Matrix odg = gate_rows ? full(dgate, lddg) : none;
    const Matrix vdg = gate_rows ? none : row(dgate, PURLIN_F32);
    const Matrix vdp = row(dpost_weight, PURLIN_F32), vdw = row(dweight, PURLIN_F32);
    for (const Matrix &o : {odx, odr, odg})
        if (any_overlap(o, {mgc, mp, mw, vdg, vdp, vdw}) || clashes(o, {mdy, mdt, mx, mt, mgr}))
            return PURLIN_ERR_ALIAS;
    for (const Matrix &o : {vdg, vdp, vdw})
        if (any_overlap(o, {mdy, mdt, mx, mt, mgr, mgc, mp, mw})) return PURLIN_ERR_ALIAS;
    if (overlap(odx, odr) || overlap(odx, odg) || overlap(odr, odg) || overlap(vdg, vdp) ||
        overlap(vdg, vdw) || overlap(vdp, vdw))
        return PURLIN_ERR_ALIAS;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;
    if (!any) {
        for (void *v : {(void *)dweight, (void *)dpost_weight, gate_rows ? nullptr : dgate})
            if (v != nullptr &&
                cudaMemsetAsync(v, 0, hidden * sizeof(float), ctx->stream) != cudaSuccess)
                return PURLIN_ERR_CUDA;
        return PURLIN_OK;
    }

    BlockNormBackwardArgs a;
    a.dy = dy;
    a.dtotal = dtotal;
    a.x = x;
    a.total = total;
    a.post_weight = post_weight;
    a.gate = gate;
    a.weight = weight;
    a.dx = dx;
    a.dresidual = dresidual;
    a.dpost_weight = dpost_weight;
    a.dgate = dgate;
    a.dweight = dweight;
    a.lddy = lddy;
    a.lddt = lddt;
    a.ldx = ldx;
    a.ldt = ldt;
    a.ldg = ldg;
    a.lddx = lddx;
    a.lddr = lddr;
    a.lddg = lddg;
    a.gate_rows = gate_rows;
    a.block_scale = block_scale;
    a.residual_scale = residual_scale;
    a.rows = rows;
    a.hidden = hidden;
    a.eps = eps;
    a.dtype = dtype;
    a.sms = ctx->sms;
    a.err = ctx->err;
    a.stream = ctx->stream;
    if (const size_t bytes = block_norm_backward_workspace(a)) {
        void *work = nullptr;
        const purlin_status st = workspace(ctx, bytes, &work);
        if (st != PURLIN_OK) return st;
        a.partial = static_cast<float *>(work);
    }
    return done(launch_block_norm_backward(a));
}

}  // extern "C"
