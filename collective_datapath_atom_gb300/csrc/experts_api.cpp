// experts_api.cpp -- host side of the router, the order by expert and the rows'
// way to the experts and back (include/purlin.h, "layer operators"; kernels in
// router.cu and expert_rows.cu): argument checks and the launches.
#include <cuda_runtime.h>

#include <cmath>

#include "checks.h"
#include "host.h"
#include "layers.h"

using namespace purlin;
using namespace purlin::host;

namespace {

// A device array of n 32-bit values.
Matrix words(const void *p, size_t n) { return matrix(p, 1, n, n, PURLIN_F32); }

// The router's fields, checked, as launch arguments.
purlin_status read_router(const purlin_router *r, purlin_dtype dtype, RouteArgs *a) {
    if (dtype != PURLIN_F32 && dtype != PURLIN_BF16)
        return dtype == PURLIN_E4M3 ? PURLIN_ERR_UNSUPPORTED : PURLIN_ERR_INVALID_ARG;
    if (r == nullptr || r->experts < 1 || r->experts > PURLIN_MAX_GROUPS || r->top_k < 1 ||
        (r->scores != PURLIN_SOFTMAX && r->scores != PURLIN_SIGMOID) || r->groups < 0 ||
        r->group_top < 0 || (r->renormalise != 0 && r->renormalise != 1) ||
        !std::isfinite(r->scale))
        return PURLIN_ERR_INVALID_ARG;
    const int groups = r->groups > 1 ? r->groups : 1;
    const int top_groups = groups > 1 ? r->top_groups : 1;
    if (r->experts % groups != 0 || top_groups < 1 || top_groups > groups ||
        r->top_k > r->experts / groups * top_groups)
        return PURLIN_ERR_INVALID_ARG;
    if (r->top_k > kMaxChoices || groups > kMaxExpertGroups || r->group_top > 2)
        return PURLIN_ERR_UNSUPPORTED;
    a->experts = r->experts;
    a->top_k = r->top_k;
    a->groups = groups;
    a->top_groups = top_groups;
    a->group_top = r->group_top == 2 ? 2 : 1;
    a->sigmoid = r->scores == PURLIN_SIGMOID;
    a->renormalise = r->renormalise == 1;
    a->scale = r->scale == 0 ? 1.f : r->scale;
    a->dtype = dtype;
    return PURLIN_OK;
}

bool too_many_slots(size_t tokens, int top_k) { return tokens > kMaxExtent / (size_t)top_k; }

// What the three calls that move rows have in common.
purlin_status rows_ranges(size_t tokens, int top_k, size_t cols, size_t n_rows) {
    if (top_k < 1 || top_k > kMaxChoices || too_many_slots(tokens, top_k) || cols > kMaxExtent ||
        n_rows > kMaxExtent)
        return PURLIN_ERR_INVALID_ARG;
    return PURLIN_OK;
}

purlin_status f32_or_bf16(purlin_dtype dtype) {
    if (dtype == PURLIN_E4M3) return PURLIN_ERR_UNSUPPORTED;
    return dtype == PURLIN_F32 || dtype == PURLIN_BF16 ? PURLIN_OK : PURLIN_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

purlin_status purlin_route(purlin_ctx *ctx, const void *logits, size_t ld, const float *bias,
                           float *weights, int32_t *chosen, size_t tokens,
                           const purlin_router *router, purlin_dtype dtype) {
    RouteArgs a;
    const purlin_status st = read_router(router, dtype, &a);
    if (st != PURLIN_OK) return st;
    const size_t experts = (size_t)a.experts, slots = tokens * (size_t)a.top_k;
    ld = ld ? ld : experts;
    if (bad_ld(ld, experts) || too_many_slots(tokens, a.top_k)) return PURLIN_ERR_INVALID_ARG;
    if (tokens == 0) return ctx ? PURLIN_OK : PURLIN_ERR_INVALID_ARG;
    if (logits == nullptr || weights == nullptr || chosen == nullptr) return PURLIN_ERR_INVALID_ARG;
    if (misaligned(logits, (size_t)size_of(dtype)) || misaligned(bias, 4) ||
        misaligned(weights, 4) || misaligned(chosen, 4))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix ml = matrix(logits, tokens, experts, ld, dtype), mb = words(bias, experts);
    const Matrix mw = words(weights, slots), mc = words(chosen, slots);
    if (any_overlap(mw, {ml, mb, mc}) || any_overlap(mc, {ml, mb})) return PURLIN_ERR_ALIAS;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;
    a.logits = logits;
    a.bias = bias;
    a.weights = weights;
    a.chosen = chosen;
    a.ld = ld;
    a.tokens = tokens;
    a.stream = ctx->stream;
    return done(launch_route(a));
}

purlin_status purlin_route_backward(purlin_ctx *ctx, const float *dweights, const void *logits,
                                    size_t ld, const int32_t *chosen, void *dlogits, size_t ldd,
                                    size_t tokens, const purlin_router *router,
                                    purlin_dtype dtype) {
    RouteArgs a;
    const purlin_status st = read_router(router, dtype, &a);
    if (st != PURLIN_OK) return st;
    const size_t experts = (size_t)a.experts, slots = tokens * (size_t)a.top_k;
    ld = ld ? ld : experts;
    ldd = ldd ? ldd : experts;
    if (bad_ld(ld, experts) || bad_ld(ldd, experts) || too_many_slots(tokens, a.top_k))
        return PURLIN_ERR_INVALID_ARG;
    if (tokens == 0) return ctx ? PURLIN_OK : PURLIN_ERR_INVALID_ARG;
    if (dweights == nullptr || logits == nullptr || chosen == nullptr || dlogits == nullptr)
        return PURLIN_ERR_INVALID_ARG;
    const size_t es = (size_t)size_of(dtype);
    if (misaligned(logits, es) || misaligned(dlogits, es) || misaligned(dweights, 4) ||
        misaligned(chosen, 4))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix ml = matrix(logits, tokens, experts, ld, dtype);
    const Matrix md = matrix(dlogits, tokens, experts, ldd, dtype);
    if (any_overlap(md, {words(dweights, slots), words(chosen, slots)}) ||
        (overlap(md, ml) && !same(md, ml)))
        return PURLIN_ERR_ALIAS;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;
    a.logits = logits;
    a.dweights = dweights;
    a.chosen = const_cast<int32_t *>(chosen);
    a.dlogits = dlogits;
    a.ld = ld;
    a.ldd = ldd;
    a.tokens = tokens;
    a.stream = ctx->stream;
    return done(launch_route_backward(a));
}

purlin_status purlin_expert_order(purlin_ctx *ctx, const int32_t *chosen, int32_t *place,
                                  int64_t *begin, int64_t *count, size_t slots, int groups,
                                  size_t capacity) {
    if (groups < 0 || groups > kMaxGroups || slots > kMaxExtent || capacity > kMaxExtent ||
        (size_t)groups * capacity > kMaxExtent)
        return PURLIN_ERR_INVALID_ARG;
    if ((slots > 0 && (chosen == nullptr || place == nullptr)) ||
        (groups > 0 && (begin == nullptr || count == nullptr)))
        return PURLIN_ERR_INVALID_ARG;
    if (misaligned(chosen, 4) || misaligned(place, 4) || misaligned(begin, 8) ||
        misaligned(count, 8))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix mi = words(slots ? chosen : nullptr, slots);
    const Matrix mp = words(slots ? place : nullptr, slots);
    const Matrix mb = words(begin, 2 * (size_t)groups), mc = words(count, 2 * (size_t)groups);
    if (any_overlap(mp, {mi, mb, mc}) || any_overlap(mb, {mi, mc}) || overlap(mc, mi))
        return PURLIN_ERR_ALIAS;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;
    if (slots == 0 && groups == 0) return PURLIN_OK;
    OrderArgs a;
    a.chosen = chosen;
    a.place = place;
    a.begin = begin;
    a.count = count;
    a.slots = slots;
    a.capacity = capacity;
    a.groups = groups;
    a.sms = ctx->sms;
    a.stream = ctx->stream;
    if (const size_t bytes = expert_order_workspace(a)) {
        void *work = nullptr;
        const purlin_status st = workspace(ctx, bytes, &work);
        if (st != PURLIN_OK) return st;
        a.partial = static_cast<int *>(work);
    }
    return done(launch_expert_order(a));
}

purlin_status purlin_dispatch_rows(purlin_ctx *ctx, const void *x, size_t ldx,
                                   const float *scales, const int32_t *place, void *out,
                                   size_t ldo, float *out_scales, size_t tokens, int top_k,
                                   size_t cols, size_t out_rows, purlin_dtype dtype) {
    if (dtype != PURLIN_F32 && dtype != PURLIN_BF16 && dtype != PURLIN_E4M3)
        return PURLIN_ERR_INVALID_ARG;
    const purlin_status st = rows_ranges(tokens, top_k, cols, out_rows);
    if (st != PURLIN_OK) return st;
    ldx = ldx ? ldx : cols;
    ldo = ldo ? ldo : cols;
    if (bad_ld(ldx, cols) || bad_ld(ldo, cols)) return PURLIN_ERR_INVALID_ARG;
    if (tokens == 0 || cols == 0) return ctx ? PURLIN_OK : PURLIN_ERR_INVALID_ARG;
    // (arrays of no rows may be missing)
    if (x == nullptr || place == nullptr || (scales == nullptr && out_scales != nullptr) ||
        (out_rows > 0 && (out == nullptr || (scales != nullptr) != (out_scales != nullptr))))
        return PURLIN_ERR_INVALID_ARG;
    const size_t es = (size_t)size_of(dtype), slots = tokens * (size_t)top_k;
    if (misaligned(x, es) || misaligned(out, es) || misaligned(place, 4) ||
        misaligned(scales, 4) || misaligned(out_scales, 4))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix mx = matrix(x, tokens, cols, ldx, dtype), ms = words(scales, tokens);
    const Matrix mp = words(place, slots), mo = matrix(out, out_rows, cols, ldo, dtype);
    const Matrix mt = words(out_rows ? out_scales : nullptr, out_rows);
    if (any_overlap(mo, {mx, ms, mp, mt}) || any_overlap(mt, {mx, ms, mp})) return PURLIN_ERR_ALIAS;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;
    if (out_rows == 0) return PURLIN_OK;
    RowsArgs a;
    a.x = x;
    a.scales = scales;
    a.place = place;
    a.out = out;
    a.out_scales = out_scales;
    a.ldx = ldx;
    a.ldo = ldo;
    a.tokens = tokens;
    a.cols = cols;
    a.n_rows = out_rows;
    a.top_k = top_k;
    a.dtype = dtype;
    a.sms = ctx->sms;
    a.stream = ctx->stream;
    return done(launch_dispatch_rows(a));
}

purlin_status purlin_combine_rows(purlin_ctx *ctx, const void *rows, size_t ldr,
                                  const float *weights, const int32_t *place, const void *shared,
                                  size_t lds, void *y, size_t ldy, size_t tokens, int top_k,
                                  size_t cols, size_t n_rows, purlin_dtype dtype) {
    purlin_status st = f32_or_bf16(dtype);
    if (st == PURLIN_OK) st = rows_ranges(tokens, top_k, cols, n_rows);
    if (st != PURLIN_OK) return st;
    ldr = ldr ? ldr : cols;
    lds = lds ? lds : cols;
    ldy = ldy ? ldy : cols;
    if (bad_ld(ldr, cols) || bad_ld(lds, cols) || bad_ld(ldy, cols)) return PURLIN_ERR_INVALID_ARG;
    if (tokens == 0 || cols == 0) return ctx ? PURLIN_OK : PURLIN_ERR_INVALID_ARG;
    if (place == nullptr || y == nullptr || (rows == nullptr && n_rows > 0))
        return PURLIN_ERR_INVALID_ARG;
    const size_t es = (size_t)size_of(dtype), slots = tokens * (size_t)top_k;
    if (misaligned(rows, es) || misaligned(shared, es) || misaligned(y, es) ||
        misaligned(place, 4) || misaligned(weights, 4))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix mr = matrix(rows, n_rows, cols, ldr, dtype);
    const Matrix ms = matrix(shared, tokens, cols, lds, dtype);
    const Matrix my = matrix(y, tokens, cols, ldy, dtype);
    if (any_overlap(my, {mr, words(place, slots), words(weights, slots)}) ||
        (overlap(my, ms) && !same(my, ms)))
        return PURLIN_ERR_ALIAS;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;
    RowsArgs a;
    a.rows = rows;
    a.weights = weights;
    a.place = place;
    a.shared = shared;
    a.out = y;
    a.ldr = ldr;
    a.lds = lds;
    a.ldo = ldy;
    a.tokens = tokens;
    a.cols = cols;
    a.n_rows = n_rows;
    a.top_k = top_k;
    a.dtype = dtype;
    a.sms = ctx->sms;
    a.stream = ctx->stream;
    return done(launch_combine_rows(a));
}

purlin_status purlin_combine_rows_backward(purlin_ctx *ctx, const void *dy, size_t lddy,
                                           const void *rows, size_t ldr, const float *weights,
                                           const int32_t *place, void *drows, size_t lddr,
                                           float *dweights, size_t tokens, int top_k, size_t cols,
                                           size_t n_rows, purlin_dtype dtype) {
    purlin_status st = f32_or_bf16(dtype);
    if (st == PURLIN_OK) st = rows_ranges(tokens, top_k, cols, n_rows);
    if (st != PURLIN_OK) return st;
    lddy = lddy ? lddy : cols;
    ldr = ldr ? ldr : cols;
    lddr = lddr ? lddr : cols;
    if (bad_ld(lddy, cols) || bad_ld(ldr, cols) || bad_ld(lddr, cols))
        return PURLIN_ERR_INVALID_ARG;
    if (tokens == 0) return ctx ? PURLIN_OK : PURLIN_ERR_INVALID_ARG;
    if (dweights == nullptr || place == nullptr || weights == nullptr ||
        (cols > 0 && (dy == nullptr || (n_rows > 0 && (rows == nullptr || drows == nullptr)))))
        return PURLIN_ERR_INVALID_ARG;
    const size_t es = (size_t)size_of(dtype), slots = tokens * (size_t)top_k;
    if (misaligned(dy, es) || misaligned(rows, es) || misaligned(drows, es) ||
        misaligned(dweights, 4) || misaligned(place, 4) || misaligned(weights, 4))
        return PURLIN_ERR_ALIGNMENT;
    const Matrix mdy = matrix(dy, tokens, cols, lddy, dtype);
    const Matrix mr = matrix(rows, n_rows, cols, ldr, dtype);
    const Matrix md = matrix(drows, n_rows, cols, lddr, dtype);
    const Matrix mp = words(place, slots), mw = words(weights, slots), mg = words(dweights, slots);
    if (any_overlap(md, {mdy, mp, mw, mg}) || any_overlap(mg, {mdy, mr, mp, mw}) ||
        (overlap(md, mr) && !same(md, mr)))
        return PURLIN_ERR_ALIAS;
    if (ctx == nullptr) return PURLIN_ERR_INVALID_ARG;
    RowsArgs a;
    a.x = dy;
    a.rows = rows;
    a.weights = weights;
    a.place = place;
    a.out = drows;
    a.out_scales = dweights;
    a.ldx = lddy;
    a.ldr = ldr;
    a.ldo = lddr;
    a.tokens = tokens;
    a.cols = cols;
    a.n_rows = n_rows;
    a.top_k = top_k;
    a.dtype = dtype;
    a.sms = ctx->sms;
    a.stream = ctx->stream;
    return done(launch_combine_rows_backward(a));
}

}  // extern "C"
