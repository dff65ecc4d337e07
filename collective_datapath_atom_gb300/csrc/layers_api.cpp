// layers_api.cpp -- host side of the layer operators (include/purlin.h,
// "layer operators"; kernels in rms_norm.cu and grouped.cu): argument checks,
// the context's workspace and one launch a call.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "checks.h"
#include "host.h"
#include "layers.h"

using namespace purlin;
using namespace purlin::host;

namespace {

// A device array of one int64 a group.
Matrix group_array(const int64_t *p, int groups) {
    return matrix(p, 1, 2 * (size_t)groups, 2 * (size_t)groups, PURLIN_F32);
}

// Whether a grouped product's tiles (tall: rows, or n for the weight gradient)
// can be counted in 32 bits, and a weight matrix's pitch in the 40 that a
// tensor map has.
bool too_many_tiles(size_t channels, size_t tall, size_t each_group, int groups) {
    const size_t across = channels / kGroupedChannelTile + 1;
    const size_t down = tall / kGroupedRowTile + each_group * (size_t)groups;
    return across * down > kMaxExtent / 2;
}
bool too_long(size_t rows, size_t ld, size_t es) {
    return rows != 0 && ld * es >= ((size_t)1 << 40) / rows;
}

purlin_status run_grouped(purlin_ctx *ctx, GroupedArgs &a) {
    void *work = nullptr;
    const purlin_status st = workspace(ctx, grouped_workspace(ctx->sms), &work);
    if (st != PURLIN_OK) return st;
    a.sms = ctx->sms;
    a.partial = static_cast<float *>(work);
    a.arrived = ctx->arrived;
    a.err = ctx->err;
    a.stream = ctx->stream;
    return launch_grouped(a) == cudaSuccess ? PURLIN_OK : PURLIN_ERR_CUDA;
}

}  // namespace

namespace purlin {
namespace host {

// At least `bytes` of device memory for one call on the context's stream.
// Memory that a graph was captured with is kept until purlin_finalize.
purlin_status workspace(purlin_ctx *ctx, size_t bytes, void **out) {
    const bool cap = capturing(ctx->stream);
    if (bytes > ctx->work.bytes) {
        if (cap) return PURLIN_ERR_UNSUPPORTED;   // no allocation during capture
        bytes = std::max(bytes, 2 * ctx->work.bytes);
        void *p = nullptr;
        if (cudaMalloc(&p, bytes) != cudaSuccess) {
            cudaGetLastError();
            return PURLIN_ERR_OOM;
        }
        purlin_status st = PURLIN_OK;
        if (ctx->work.p && !ctx->work.pinned) {
            if (cudaStreamSynchronize(ctx->stream) != cudaSuccess) st = PURLIN_ERR_CUDA;
            cudaFree(ctx->work.p);
        } else if (ctx->work.p) {
            WorkMem *old = new (std::nothrow) WorkMem(ctx->work);
            if (!old) {
                cudaFree(p);
                return PURLIN_ERR_OOM;
            }
            old->next = ctx->old_work;
            ctx->old_work = old;
        }
        ctx->work = WorkMem{};
        ctx->work.p = p;
        ctx->work.bytes = bytes;
        if (st != PURLIN_OK) return st;
    }
    ctx->work.pinned |= cap;
    *out = ctx->work.p;
    return PURLIN_OK;
}

void free_workspace(purlin_ctx *ctx) {
    if (ctx->work.p) cudaFree(ctx->work.p);
    for (WorkMem *m = ctx->old_work; m != nullptr;) {
        WorkMem *next = m->next;
        cudaFree(m->p);
        delete m;
        m = next;
    }
    ctx->work = WorkMem{};
    ctx->old_work = nullptr;
}

}  // namespace host
}  // namespace purlin

extern "C" {

purlin_status purlin_rms_norm(purlin_ctx *ctx, const void *x, size_t ldx, const void *residual,
                              size_t ldr, const void *weight, void *y, size_t ldy, void *total,
                              size_t ldt, float *scales, size_t rows, size_t hidden, float eps,
                              purlin_dtype dtype, purlin_dtype out_dtype) {
    if (dtype != PURLIN_F32 && dtype != PURLIN_BF16) return PURLIN_ERR_INVALID_ARG;
    if (out_dtype != dtype && out_dtype != PURLIN_E4M3) return PURLIN_ERR_UNSUPPORTED;
    if (hidden == 0 || hidden > kMaxExtent / 2 || rows > kMaxExtent || !(eps >= 0) ||
        !std::isfinite(eps))
        return PURLIN_ERR_INVALID_ARG;
    ldx = ldx ? ldx : hidden;
    ldr = ldr ? ldr : hidden;
    ldy = ldy ? ldy : hidden;
    ldt = ldt ? ldt : hidden;
    if (bad_ld(ldx, hidden) || bad_ld(ldr, hidden) || bad_ld(ldy, hidden) || bad_ld(ldt, hidden))
        return PURLIN_ERR_INVALID_ARG;
    if (rows == 0) return ctx ? PURLIN_OK : PURLIN_ERR_INVALID_ARG;
    if (x == nullptr || weight == nullptr || y == nullptr ||
        (scales != nullptr) != (out_dtype == PURLIN_E4M3))
        return PURLIN_ERR_INVALID_ARG;
    const size_t es = (size_t)size_of(dtype);
    if (misaligned(x, es) || misaligned(residual, es) || misaligned(weight, es) ||
        misaligned(total, es) || misaligned(y, (size_t)size_of(out_dtype)) ||
        misaligned(scales, 4))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix mx = matrix(x, rows, hidden, ldx, dtype);
    const Matrix mr = matrix(residual, rows, hidden, ldr, dtype);
    const Matrix mw = matrix(weight, 1, hidden, hidden, dtype);
    const Matrix my = matrix(y, rows, hidden, ldy, out_dtype);
    const Matrix mt = matrix(total, rows, hidden, ldt, dtype);
    const Matrix ms = matrix(scales, 1, rows, rows, PURLIN_F32);
    for (const Matrix *o : {&my, &mt})
        if (overlap(*o, mw) || (overlap(*o, mx) && !same(*o, mx)) ||
            (overlap(*o, mr) && !same(*o, mr)))
            return PURLIN_ERR_ALIAS;
    // (scales are another row's elements, wherever in x they lie)
    if (overlap(ms, mx) || overlap(ms, mr) || overlap(ms, mw)) return PURLIN_ERR_ALIAS;
    if (overlap(my, mt) || overlap(my, ms) || overlap(mt, ms)) return PURLIN_ERR_ALIAS;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;

    NormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.y = y;
    a.total = total;
    a.scales = scales;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldy = ldy;
    a.ldt = ldt;
    a.rows = rows;
    a.hidden = hidden;
    a.eps = eps;
    a.dtype = dtype;
    a.out_dtype = out_dtype;
    a.sms = ctx->sms;
    a.err = ctx->err;
    a.stream = ctx->stream;
    return launch_norm(a) == cudaSuccess ? PURLIN_OK : PURLIN_ERR_CUDA;
}

purlin_status purlin_rms_norm_backward(purlin_ctx *ctx, const void *dy, size_t lddy,
                                       const void *total, size_t ldt, const void *weight,
                                       const void *dtotal, size_t lddt, void *dx, size_t lddx,
                                       float *dweight, size_t rows, size_t hidden, float eps,
                                       purlin_dtype dtype) {
    if (dtype != PURLIN_F32 && dtype != PURLIN_BF16) return PURLIN_ERR_INVALID_ARG;
    if (hidden == 0 || hidden > kMaxExtent / 2 || rows > kMaxExtent || !(eps >= 0) ||
        !std::isfinite(eps))
        return PURLIN_ERR_INVALID_ARG;
    lddy = lddy ? lddy : hidden;
    ldt = ldt ? ldt : hidden;
    lddt = lddt ? lddt : hidden;
    lddx = lddx ? lddx : hidden;
    if (bad_ld(lddy, hidden) || bad_ld(ldt, hidden) || bad_ld(lddt, hidden) ||
        bad_ld(lddx, hidden))
        return PURLIN_ERR_INVALID_ARG;
    if (dweight == nullptr || weight == nullptr ||
        (rows > 0 && (dy == nullptr || total == nullptr || dx == nullptr)))
        return PURLIN_ERR_INVALID_ARG;
    const size_t es = (size_t)size_of(dtype);
    if (misaligned(dy, es) || misaligned(total, es) || misaligned(weight, es) ||
        misaligned(dtotal, es) || misaligned(dx, es) || misaligned(dweight, 4))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix mdy = matrix(dy, rows, hidden, lddy, dtype);
    const Matrix mt = matrix(total, rows, hidden, ldt, dtype);
    const Matrix mw = matrix(weight, 1, hidden, hidden, dtype);
    const Matrix md = matrix(dtotal, rows, hidden, lddt, dtype);
    const Matrix mx = matrix(dx, rows, hidden, lddx, dtype);
    const Matrix mg = matrix(dweight, 1, hidden, hidden, PURLIN_F32);
    for (const Matrix *i : {&mdy, &mt, &md})
        if (overlap(mg, *i) || (overlap(mx, *i) && !same(mx, *i))) return PURLIN_ERR_ALIAS;
    if (overlap(mx, mw) || overlap(mg, mw) || overlap(mx, mg)) return PURLIN_ERR_ALIAS;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;
    if (rows == 0)
        return cudaMemsetAsync(dweight, 0, hidden * sizeof(float), ctx->stream) == cudaSuccess
                   ? PURLIN_OK
                   : PURLIN_ERR_CUDA;

    NormBackwardArgs a;
    a.dy = dy;
    a.total = total;
    a.weight = weight;
    a.dtotal = dtotal;
    a.dx = dx;
    a.dweight = dweight;
    a.lddy = lddy;
    a.ldt = ldt;
    a.lddt = lddt;
    a.lddx = lddx;
    a.rows = rows;
    a.hidden = hidden;
    a.eps = eps;
    a.dtype = dtype;
    a.sms = ctx->sms;
    a.err = ctx->err;
    a.stream = ctx->stream;
    void *work = nullptr;
    const purlin_status st =
        workspace(ctx, norm_backward_workspace(a), &work);
    if (st != PURLIN_OK) return st;
    a.partial = static_cast<float *>(work);
    return launch_norm_backward(a) == cudaSuccess ? PURLIN_OK : PURLIN_ERR_CUDA;
}

purlin_status purlin_grouped_matmul(purlin_ctx *ctx, const void *x, size_t ldx, const void *w,
                                    size_t ldw, void *y, size_t ldy, const float *x_scales,
                                    const float *w_scales, const int64_t begin[],
                                    const int64_t count[], int groups, size_t rows, size_t n,
                                    size_t k, purlin_dtype dtype, purlin_weights_layout layout) {
    if (layout != PURLIN_WEIGHTS_NK && layout != PURLIN_WEIGHTS_KN) return PURLIN_ERR_INVALID_ARG;
    if (dtype != PURLIN_BF16 && dtype != PURLIN_E4M3)
        return dtype == PURLIN_F32 ? PURLIN_ERR_UNSUPPORTED : PURLIN_ERR_INVALID_ARG;
    if (dtype == PURLIN_E4M3 && layout != PURLIN_WEIGHTS_NK) return PURLIN_ERR_UNSUPPORTED;
    if (groups < 0 || groups > kMaxGroups || rows > kMaxExtent || n > kMaxExtent ||
        k > kMaxExtent || k == 0)
        return PURLIN_ERR_INVALID_ARG;
    const size_t w_rows = layout == PURLIN_WEIGHTS_NK ? n : k;
    const size_t w_cols = layout == PURLIN_WEIGHTS_NK ? k : n;
    const size_t es = (size_t)size_of(dtype);
    ldx = ldx ? ldx : k;
    ldw = ldw ? ldw : w_cols;
    ldy = ldy ? ldy : n;
    if (bad_ld(ldx, k) || bad_ld(ldw, w_cols) || bad_ld(ldy, n)) return PURLIN_ERR_INVALID_ARG;
    if (rows == 0 || n == 0 || groups == 0) return ctx ? PURLIN_OK : PURLIN_ERR_INVALID_ARG;
    if (x == nullptr || w == nullptr || y == nullptr || begin == nullptr || count == nullptr ||
        misaligned(begin, 8) || misaligned(count, 8) ||
        (x_scales != nullptr) != (dtype == PURLIN_E4M3) ||
        (w_scales != nullptr) != (dtype == PURLIN_E4M3))
        return PURLIN_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(w, 16) || (ldx * es) % 16 != 0 || (ldw * es) % 16 != 0 ||
        misaligned(y, 2) || misaligned(x_scales, 4) || misaligned(w_scales, 4))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix my = matrix(y, rows, n, ldy, PURLIN_BF16);
    if (overlap(my, matrix(x, rows, k, ldx, dtype)) ||
        overlap(my, matrix(w, (size_t)groups * w_rows, w_cols, ldw, dtype)) ||
        overlap(my, matrix(x_scales, 1, rows, rows, PURLIN_F32)) ||
        overlap(my, matrix(w_scales, 1, (size_t)groups * n, (size_t)groups * n, PURLIN_F32)) ||
        overlap(my, group_array(begin, groups)) || overlap(my, group_array(count, groups)))
        return PURLIN_ERR_ALIAS;
    if (too_many_tiles(n, rows, 1, groups) || too_long(w_rows, ldw, es))
        return PURLIN_ERR_UNSUPPORTED;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;

    GroupedArgs a;
    a.mode = layout == PURLIN_WEIGHTS_NK ? kGroupedNK : kGroupedKN;
    a.x = x;
    a.w = w;
    a.y = y;
    a.x_scales = x_scales;
    a.w_scales = w_scales;
    a.begin = begin;
    a.count = count;
    a.ldx = ldx;
    a.ldw = ldw;
    a.ldy = ldy;
    a.groups = groups;
    a.rows = rows;
    a.n = n;
    a.k = k;
    a.dtype = dtype;
    return run_grouped(ctx, a);
}

purlin_status purlin_grouped_matmul_weight_grad(purlin_ctx *ctx, const void *dy, size_t lddy,
                                                const void *x, size_t ldx, void *dw, size_t lddw,
                                                const int64_t begin[], const int64_t count[],
                                                int groups, size_t rows, size_t n, size_t k,
                                                purlin_dtype dtype) {
    if (dtype != PURLIN_BF16)
        return dtype == PURLIN_F32 || dtype == PURLIN_E4M3 ? PURLIN_ERR_UNSUPPORTED
                                                           : PURLIN_ERR_INVALID_ARG;
    if (groups < 0 || groups > kMaxGroups || rows > kMaxExtent || n > kMaxExtent || k > kMaxExtent)
        return PURLIN_ERR_INVALID_ARG;
    lddy = lddy ? lddy : n;
    ldx = ldx ? ldx : k;
    lddw = lddw ? lddw : k;
    if (bad_ld(lddy, n) || bad_ld(ldx, k) || bad_ld(lddw, k)) return PURLIN_ERR_INVALID_ARG;
    if (n == 0 || k == 0 || groups == 0) return ctx ? PURLIN_OK : PURLIN_ERR_INVALID_ARG;
    if (dw == nullptr || (rows > 0 && (dy == nullptr || x == nullptr || begin == nullptr ||
                                       count == nullptr || misaligned(begin, 8) ||
                                       misaligned(count, 8))))
        return PURLIN_ERR_INVALID_ARG;
    if (misaligned(dw, 2) ||
        (rows > 0 && (misaligned(dy, 16) || misaligned(x, 16) || (lddy * 2) % 16 != 0 ||
                      (ldx * 2) % 16 != 0)))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix mw = matrix(dw, (size_t)groups * n, k, lddw, dtype);
    if (overlap(mw, matrix(dy, rows, n, lddy, dtype)) ||
        overlap(mw, matrix(x, rows, k, ldx, dtype)) || overlap(mw, group_array(begin, groups)) ||
        overlap(mw, group_array(count, groups)))
        return PURLIN_ERR_ALIAS;
    if (too_many_tiles(k, 0, n / kGroupedRowTile + 1, groups)) return PURLIN_ERR_UNSUPPORTED;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;
    if (rows == 0)
        return cudaMemset2DAsync(dw, lddw * 2, 0, k * 2, (size_t)groups * n, ctx->stream) ==
                       cudaSuccess
                   ? PURLIN_OK
                   : PURLIN_ERR_CUDA;

    GroupedArgs a;
    a.mode = kGroupedGrad;
    a.x = x;
    a.w = dy;
    a.y = dw;
    a.begin = begin;
    a.count = count;
    a.ldx = ldx;
    a.ldw = lddy;
    a.ldy = lddw;
    a.groups = groups;
    a.rows = rows;
    a.n = n;
    a.k = k;
    a.dtype = dtype;
    return run_grouped(ctx, a);
}

}  // extern "C"
