// router.cu -- which experts a token goes to, and with what weights: scores of its
// logits (softmax or sigmoid), a bias for balance, groups of experts, the top k, and
// their renormalised weights; and the weights' gradient with respect to the logits.
//
// A warp has a token.  Its lanes are dealt out to the groups of experts, 32 / P lanes
// a group (P: the groups, rounded up to a power of two), and each lane holds
// consecutive experts of its group, so that a lower lane holds lower experts: an
// expert's key is its choice value as an ordered 32-bit number, the largest key of the
// warp is one reduction, and of equal keys the lowest lane's is the lowest expert.
//
// The choice is that of exact values.  Without a bias the scores rise with the logits,
// and the logits themselves are compared, exactly.  With one, binary32 values c carry
// an error of at most `tol`, and where two that matter to the answer (neighbours among
// the chosen, the last of them and what is left, the last group kept and the rest) are
// no further apart than that, and not of the same logit and bias, what is near the
// border is computed again in binary64 and ranked by that: about two rows in a thousand.
// What binary64 does not tell apart, as scores of logits above 37 with a bias, are equal
// values.
//
// Bound by the issue of instructions, about a thousand a token of 256 experts in eight
// groups (16384 tokens, sigmoid, bias, four groups, top 8: 25 us, 72 % of the issue
// slots; the logits' bytes are 2.6; bf16 the same).  Fewer lanes a token, 8 or 16, leave more experts to
// a lane and the work of its second best among the chosen: 32 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "layers.h"

namespace purlin {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kMaxFinite = 3.40282347e38f;
constexpr int kRouteWarps = 8;   // tokens of a block

__device__ __forceinline__ float minus_infinity() { return __int_as_float(0xff800000); }

struct RouteParams {
    const void *logits;
    const float *bias, *dweights;
    float *weights;
    int32_t *chosen;
    void *dlogits;
    size_t ld, ldd, tokens;
    int experts, top_k, groups, top_groups, group_top;
    int each;    // experts of a group
    int lanes, lane_bits;   // lanes of a group, a power of two
    int held;    // experts of a lane
    bool sigmoid, renormalise;
    float scale;
};

__device__ __forceinline__ float value_of(const float *p) { return *p; }
__device__ __forceinline__ float value_of(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// A logit as it counts: +inf is the largest finite value, -0 is 0, NaN is NaN.
__device__ __forceinline__ float counted(float l) { return (l > kMaxFinite ? kMaxFinite : l) + 0.f; }

// Numbers in the order of the values; 0 is left for "none".
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
}

__device__ __forceinline__ float sigmoid_of(float l) {
    const float z = expf(-fabsf(l));
    return (l >= 0.f ? 1.f : z) / (1.f + z);
}

// The same for the choice alone, by the approximate 2^x and 1 / x: off by 2 + 1.2 |l|
// ulp of the exponential, which is as many of the score where that is small, and next
// to none where it is near 1 (16384 x 256: with exp and a division 2 us more).
__device__ __forceinline__ float choice_sigmoid(float l) {
    float z, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(l * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + z));
    return s;
}

// The choice value in binary64: a score and the bias.
struct Exact {
    bool sigmoid;
    double most, sum;   // softmax: the largest logit, and the sum of exp(l - most)
    __device__ __noinline__ double operator()(float l, float b) const {
        const double d = (double)l;
        if (sigmoid) {
            const double z = exp(-fabs(d));
            return (d >= 0 ? 1.0 : z) / (1.0 + z) + (double)b;
        }
        return exp(d - most) / sum + (double)b;
    }
};

// One row's experts as a lane holds them: `n` of them from `first` on.
template <typename T, int HELD>
struct Row {
    const T *logits;
    const float *bias;
    int first, n;
    __device__ __forceinline__ float logit(int e) const { return counted(value_of(logits + e)); }
    __device__ __forceinline__ float bias_at(int e) const { return bias ? bias[e] + 0.f : 0.f; }
};

// HELD consecutive values from 16-byte boundaries (fewer bytes where there are fewer).
template <int HELD>
__device__ __forceinline__ void load_held(float (&v)[HELD], const float *p) {
    if constexpr (HELD % 4 == 0) {
#pragma unroll
        for (int i = 0; i < HELD / 4; ++i) {
            const float4 u = reinterpret_cast<const float4 *>(p)[i];
            v[4 * i] = u.x;
            v[4 * i + 1] = u.y;
            v[4 * i + 2] = u.z;
            v[4 * i + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < HELD; ++i) v[i] = p[i];
    }
}
template <int HELD>
__device__ __forceinline__ void load_held(float (&v)[HELD], const __nv_bfloat16 *p) {
    if constexpr (HELD % 8 == 0) {
#pragma unroll
        for (int i = 0; i < HELD / 8; ++i) {
            const uint4 u = reinterpret_cast<const uint4 *>(p)[i];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < HELD; ++i) v[i] = __bfloat162float(p[i]);
    }
}

// A lane's two largest keys and their places; experts that were taken are out of it.
template <int HELD>
struct Best {
    using Mask = std::conditional_t<HELD <= 32, uint32_t, uint64_t>;
    uint32_t key = 0, second = 0;
    int at = 0, second_at = 0;
    Mask taken = 0;
    template <bool FIRST>
    __device__ __forceinline__ void scan(const uint32_t (&keys)[HELD]) {
        key = second = 0;
        at = second_at = 0;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const uint32_t k = !FIRST && (taken >> i & 1) ? 0 : keys[i];
            const bool most = k > key, more = k > second;
            second_at = most ? at : more ? i : second_at;
            second = max(second, min(key, k));
            at = most ? i : at;
            key = max(key, k);
        }
    }
    // The largest is taken; a lane that has given two looks for the rest again.
    __device__ __forceinline__ void take(const uint32_t (&keys)[HELD]) {
        taken |= (Mask)1 << at;
        if (second != 0) {
            key = second;
            at = second_at;
            second = 0;
            fresh = false;
        } else if (!fresh) {
            scan<false>(keys);
            fresh = true;
        } else {
            key = 0;
        }
    }
    bool fresh = true;   // the second largest is known, or there is none
};

// Binary64's denominators of a row's scores.
template <typename T, int HELD>
__device__ __noinline__ Exact exact_scores(const Row<T, HELD> &row, bool sigmoid, float most) {
    Exact x{sigmoid, (double)most, 1.0};
    if (!sigmoid) {
        double s = 0;
        for (int i = 0; i < row.n; ++i) {
            const float l = row.logit(row.first + i);
            if (l >= -kMaxFinite) s += exp((double)l - x.most);
        }
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        x.sum = s;
    }
    return x;
}

// Whether this lane's group is kept, by binary64 values.  `least`: experts of the group
// with smaller keys are none of its two largest.
template <typename T, int HELD>
__device__ __noinline__ bool exact_groups(const Row<T, HELD> &row, const uint32_t (&key)[HELD], uint32_t least,
                                          const Exact &exact, const RouteParams &p, int lane) {
    double a = -INFINITY, b = -INFINITY;   // the lane's two largest
    uint64_t left = 0;
#pragma unroll
    for (int i = 0; i < HELD; ++i) left |= (uint64_t)(key[i] != 0 && key[i] >= least) << i;
    while (left != 0) {
        const int i = __ffsll(left) - 1;
        left &= left - 1;
        const double d = exact(row.logit(row.first + i), row.bias_at(row.first + i));
        if (d > a) {
            b = a;
            a = d;
        } else if (d > b) {
            b = d;
        }
    }
    __syncwarp();
    for (int o = 1; o < p.lanes; o <<= 1) {
        const double oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
    }
    const double v = p.group_top == 2 && b > -INFINITY ? a + b : a;
    int rank = 0;
    const int g = lane / p.lanes;
    for (int h = 0; h < p.groups; ++h) {
        const double o = __shfl_sync(kAll, v, h * p.lanes);
        rank += o > v || (o == v && h < g);
    }
    return g < p.groups && rank < p.top_groups && a > -INFINITY;
}

// VECTOR: every lane holds HELD experts, on 16-byte boundaries.
template <typename T, int HELD, bool VECTOR>
__global__ void __launch_bounds__(32 * kRouteWarps)
route_kernel(const __grid_constant__ RouteParams p) {
    const int lane = threadIdx.x & 31;
    const size_t token = (size_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (token >= p.tokens) return;   // whole warps
    const int g = lane >> p.lane_bits, sub = lane & (p.lanes - 1);
    Row<T, HELD> row;
    row.logits = static_cast<const T *>(p.logits) + token * p.ld;
    row.bias = p.bias;
    row.first = g * p.each + sub * p.held;
    row.n = VECTOR ? HELD : g < p.groups ? max(0, min(p.held, p.each - sub * p.held)) : 0;

    float l[HELD], b[HELD];
    if constexpr (VECTOR) {
        load_held<HELD>(l, row.logits + row.first);
        if (p.bias) load_held<HELD>(b, p.bias + row.first);
    } else {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            l[i] = i < row.n ? value_of(row.logits + row.first + i) : minus_infinity();
            if (p.bias) b[i] = i < row.n ? p.bias[row.first + i] : 0.f;
        }
    }
    bool bad = false;   // a NaN in the row
    float most = minus_infinity();
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        bad |= l[i] != l[i];
        most = fmaxf(most, l[i]);   // (not a NaN)
    }
    bad = __any_sync(kAll, bad);
    most = counted(warp_max(most));
    float inv = 0.f;   // softmax: 1 / the sum of exp(l - most)
    if (!p.sigmoid && most >= -kMaxFinite && (p.bias || !p.renormalise || p.group_top == 2)) {
        float s = 0.f, e[HELD];
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            e[i] = expf(counted(l[i]) - most);
            s += bad && l[i] != l[i] ? 0.f : e[i];   // (without NaNs the choice is of the rest)
        }
        inv = 1.f / warp_sum(s);
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < HELD; ++i) l[i] = l[i] >= -kMaxFinite ? e[i] * inv : minus_infinity();
        }
    }
    // an error of the choice values: of the scores, none above the largest one's (l e^-l
    // falls), and of a sum's rounding.  Softmax: the exponential, the quotient and HELD + 5
    // additions
    const float largest = p.sigmoid ? choice_sigmoid(most) : inv;
    const float tol = largest * (p.sigmoid ? 4.f + 1.2f * fminf(fmaxf(-most, 0.f), 200.f) : (float)(HELD + 16)) * 0x1p-22f + 0x1p-120f;
    auto near = [&](float hi, float lo, float by) {   // not told apart, infinities too
        return !(hi - lo > by + fabsf(hi) * 0x1p-22f);
    };
    auto score = [&](float v) { return p.sigmoid ? choice_sigmoid(v) : expf(v - most) * inv; };
    uint32_t key[HELD];
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        float c = l[i];
        if (!p.bias) c = counted(c);
        else if (p.sigmoid) c = choice_sigmoid(c) + b[i];
        else c += b[i];
        key[i] = l[i] >= -kMaxFinite && c > minus_infinity() ? key_of(c) : 0;
    }
    Best<HELD> best;
    best.template scan<true>(key);

    if (p.top_groups < p.groups) {
        uint32_t a = best.key, c = best.second;   // the group's two largest keys
        for (int o = 1; o < p.lanes; o <<= 1) {
            const uint32_t oa = __shfl_xor_sync(kAll, a, o), oc = __shfl_xor_sync(kAll, c, o);
            c = max(min(a, oa), max(c, oc));
            a = max(a, oa);
        }
        float v = of_key(a), size = 0.f;   // size: of what v adds up
        const bool exactly = !p.bias && p.group_top == 1;   // logits, nothing to tell apart
        if (!exactly) {
            if (!p.bias) v = score(v);
            size = fabsf(v);
            if (p.group_top == 2 && c != 0) {
                const float second = p.bias ? of_key(c) : score(of_key(c));
                v += second;
                size += fabsf(second);
            }
        }
        const uint32_t mine = a != 0 ? key_of(v) : 0;
        int rank = 0;
#pragma unroll 4
        for (int h = 0; h < p.groups; ++h) {
            const uint32_t o = __shfl_sync(kAll, mine, h * p.lanes);
            rank += o > mine || (o == mine && h < g);
        }
        const bool there = g < p.groups && mine != 0;
        bool keep = there && rank < p.top_groups;
        if (!exactly) {
            // each value is off by its two choices' errors and the sum's, which go by the
            // choices' sizes (with opposite signs the sum has none); where one kept may lie
            // below one that is left, and they are not the like of the last one kept
            const float off = fabsf(v) <= kMaxFinite ? 2.f * tol + size * 0x1.8p-23f : 0.f;
            const uint32_t low = key_of(v - off), high = key_of(v + off);
            const uint32_t kept = __reduce_min_sync(kAll, keep ? low : 0xffffffffu);
            const uint32_t left = __reduce_max_sync(kAll, there && !keep ? high : 0);
            const bool unsure = keep ? low <= left : there && high >= kept;
            if (__any_sync(kAll, unsure)) {
                const int at = __ffs(__ballot_sync(kAll, there && rank == p.top_groups - 1)) - 1;
                const uint32_t ea = __shfl_sync(kAll, a, at), ec = __shfl_sync(kAll, c, at);
                const bool alike = !p.bias && a == ea && c == ec;
                if (__any_sync(kAll, unsure && !alike)) {
                    const uint32_t edge_key = p.group_top == 2 && c != 0 ? c : a;
                    const float edge_c = of_key(edge_key);
                    const float under = edge_c - (2.f * tol + fabsf(edge_c) * 0x1p-22f);
                    const uint32_t least = !p.bias ? edge_key : under == under ? key_of(under) : 1;
                    keep = exact_groups(row, key, least, exact_scores(row, p.sigmoid, most), p, lane);
                }
            }
        }
        if (!keep) {
            best.key = best.second = 0;
#pragma unroll
            for (int i = 0; i < HELD; ++i) key[i] = 0;
        }
    }

    // the largest key of the warp, top_k times; lane j keeps the j-th
    uint32_t my_key = 0;
    int my_e = -1, n = 0;
    auto take = [&] {
        const uint32_t top = __reduce_max_sync(kAll, best.key);
        if (top == 0) return false;
        const int from = __ffs(__ballot_sync(kAll, best.key == top)) - 1;
        const int e = __shfl_sync(kAll, row.first + best.at, from);
        if (lane == n) {
            my_key = top;
            my_e = e;
        }
        ++n;
        if (lane == from) best.take(key);
        return true;
    };
    while (n < p.top_k && take()) {
    }
    float my_l = my_e >= 0 ? row.logit(my_e) : minus_infinity();

    if (p.bias && n > 0) {
        const float my_b = my_e >= 0 ? row.bias_at(my_e) : 0.f;
        const float c = of_key(my_key);
        const float next_c = __shfl_down_sync(kAll, c, 1);
        const float edge = __shfl_sync(kAll, c, n - 1);
        const bool tight = lane + 1 < n && near(c, next_c, 2.f * tol);
        const bool crowd = best.key != 0 && near(edge, of_key(best.key), 2.f * tol);
        if (__any_sync(kAll, tight || crowd)) {
            // near, but perhaps of the same logit and bias: then the order is right
            const float next_l = __shfl_down_sync(kAll, my_l, 1), next_b = __shfl_down_sync(kAll, my_b, 1);
            const float edge_l = __shfl_sync(kAll, my_l, n - 1), edge_b = __shfl_sync(kAll, my_b, n - 1);
            bool unsure = tight && !(my_l == next_l && my_b == next_b);
            int close = 0;   // of what is left, as near to the last one chosen
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                if (best.taken >> i & 1) key[i] = 0;
                if (key[i] != 0 && near(edge, of_key(key[i]), 2.f * tol)) {
                    ++close;
                    unsure |= !(row.logit(row.first + i) == edge_l && row.bias_at(row.first + i) == edge_b);
                }
            }
            if (__any_sync(kAll, unsure)) {
                const Exact exact = exact_scores(row, p.sigmoid, most);
                const int chosen = n, all = chosen + __reduce_add_sync(kAll, close);
                if (all <= 32) {
                    // a candidate a lane, each at its rank among them
                    while (n < all && take()) {
                    }
                    const double d = my_e >= 0 ? exact(row.logit(my_e), row.bias_at(my_e)) : -INFINITY;
                    int rank = 0;
                    for (int i = 0; i < n; ++i) {
                        const double o = __shfl_sync(kAll, d, i);
                        const int oe = __shfl_sync(kAll, my_e, i);
                        rank += o > d || (o == d && oe < my_e);
                    }
                    int e = -1;
                    for (int i = 0; i < n; ++i) {
                        const int r = __shfl_sync(kAll, rank, i), oe = __shfl_sync(kAll, my_e, i);
                        if (r == lane) e = oe;
                    }
                    my_e = lane < chosen ? e : -1;
                } else {
                    // every expert that is left, by binary64 values, one after another
                    for (int j = 0; j < chosen; ++j) {
                        const int e = __shfl_sync(kAll, my_e, j);
#pragma unroll
                        for (int i = 0; i < HELD; ++i)
                            if (i < row.n && row.first + i == e) key[i] = 1;
                    }
                    for (int j = 0; j < chosen; ++j) {
                        double most_d = -INFINITY;
                        int at = 0x7fffffff;
#pragma unroll 1
                        for (int i = 0; i < row.n; ++i) {
                            bool in = false;
#pragma unroll
                            for (int q = 0; q < HELD; ++q) in |= q == i && key[q] != 0;
                            if (!in) continue;
                            const double d = exact(row.logit(row.first + i), row.bias_at(row.first + i));
                            if (at == 0x7fffffff || d > most_d) {
                                most_d = d;
                                at = row.first + i;
                            }
                        }
                        for (int o = 16; o > 0; o >>= 1) {
                            const double od = __shfl_xor_sync(kAll, most_d, o);
                            const int oa = __shfl_xor_sync(kAll, at, o);
                            if (od > most_d || (od == most_d && oa < at)) {
                                most_d = od;
                                at = oa;
                            }
                        }
                        if (lane == j) my_e = at;
#pragma unroll
                        for (int i = 0; i < HELD; ++i)
                            if (i < row.n && row.first + i == at) key[i] = 0;
                    }
                }
                n = chosen;
                my_l = my_e >= 0 ? row.logit(my_e) : minus_infinity();
            }
        }
    }

    const bool mine = lane < n;
    float w = 0.f;
    if (p.renormalise) {
        // over the chosen logits alone, by a factor that keeps the largest from being small
        const float top = warp_max(mine ? my_l : minus_infinity());
        if (p.sigmoid) {
            if (mine) w = expf(fminf(my_l, 0.f) - fminf(top, 0.f)) / (1.f + expf(-fabsf(my_l)));
        } else if (mine) {
            w = expf(my_l - top);
        }
        const float s = warp_sum(w);
        w = s > 0.f ? w / s : 0.f;
    } else if (mine) {
        w = p.sigmoid ? sigmoid_of(my_l) : expf(my_l - most) * inv;
    }
    if (lane < p.top_k) {
        const size_t at = token * p.top_k + lane;
        p.weights[at] = bad ? __int_as_float(0x7fffffff) : w * p.scale;
        p.chosen[at] = mine ? my_e : -1;
    }
}

// ---------------------------------------------------------------- backward --

// A warp a token: the chosen experts' shares in the lanes, then the row.  Without
// renormalisation a softmax has a gradient for every expert, and a lane holds every 32nd
// of the row (HELD of them); else the row is zeros but for the chosen ones.
template <typename T, int HELD>
__global__ void __launch_bounds__(32 * kRouteWarps)
route_backward_kernel(const __grid_constant__ RouteParams p) {
    const int lane = threadIdx.x & 31;
    const size_t token = (size_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (token >= p.tokens) return;   // whole warps
    const T *row = static_cast<const T *>(p.logits) + token * p.ld;
    T *out = static_cast<T *>(p.dlogits) + token * p.ldd;
    const bool dense = !p.sigmoid && !p.renormalise;
    float d[HELD];
    if (dense) {
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            d[i] = lane + 32 * i < p.experts ? counted(value_of(row + lane + 32 * i)) : minus_infinity();
    }
    int e = -1;
    float l = minus_infinity(), g = 0.f;
    if (lane < p.top_k) {
        const size_t at = token * p.top_k + lane;
        e = p.chosen[at];
        if ((unsigned)e < (unsigned)p.experts) {
            l = counted(value_of(row + e));
            g = p.scale * p.dweights[at];
        } else {
            e = -1;
        }
    }
    const bool real = e >= 0 && l >= -kMaxFinite;
    float v = 0.f, total = 0.f, share = 0.f;
    if (p.renormalise) {
        const float top = warp_max(real ? l : minus_infinity());
        float n = 0.f;
        if (real)
            n = p.sigmoid ? expf(fminf(l, 0.f) - fminf(top, 0.f)) / (1.f + expf(-fabsf(l)))
                          : expf(l - top);
        const float s = warp_sum(n);
        share = s > 0.f ? n / s : 0.f;
        const float mean = warp_sum(real ? g * share : 0.f);
        if (real) v = share * (g - mean) * (p.sigmoid ? sigmoid_of(-l) : 1.f);
    } else if (p.sigmoid) {
        if (real) v = g * sigmoid_of(l) * sigmoid_of(-l);
    } else {
        float most = minus_infinity(), s = 0.f;
#pragma unroll
        for (int i = 0; i < HELD; ++i) most = fmaxf(most, d[i]);
        most = fmaxf(warp_max(most), -kMaxFinite);   // (an empty row: exp(-inf) each)
#pragma unroll
        for (int i = 0; i < HELD; ++i) s += d[i] = expf(d[i] - most);
        s = warp_sum(s);
        const float inv = s == 0.f ? 0.f : 1.f / s;   // (NaN for a row with a NaN)
        share = real ? expf(l - most) * inv : 0.f;
        v = real ? g * share : 0.f;
        total = warp_sum(v);
#pragma unroll
        for (int i = 0; i < HELD; ++i) d[i] *= -(inv * total);
    }
    // an expert that occurs twice: its shares' sum, in both of its lanes
    const unsigned alike = __match_any_sync(kAll, e);
    if (__any_sync(kAll, e >= 0 && __popc(alike) > 1)) {
        float sum = 0.f;
        for (int i = 0; i < p.top_k; ++i) {
            const float o = __shfl_sync(kAll, v, i);
            if (alike >> i & 1) sum += o;
        }
        v = sum;
    }
    v -= share * total;   // (0 but where the row is dense)
    __syncwarp();         // dlogits may be logits: every lane has read its chosen one
    if (dense) {
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (lane + 32 * i < p.experts) put(out + lane + 32 * i, d[i]);
    } else {
        for (int i = lane; i < p.experts; i += 32) put(out + i, 0.f);
    }
    __syncwarp();
    if (e >= 0) put(out + e, v);
}

RouteParams params(const RouteArgs &a) {
    RouteParams p{};
    p.logits = a.logits;
    p.bias = a.bias;
    p.dweights = a.dweights;
    p.weights = a.weights;
    p.chosen = a.chosen;
    p.dlogits = a.dlogits;
    p.ld = a.ld;
    p.ldd = a.ldd;
    p.tokens = a.tokens;
    p.experts = a.experts;
    p.top_k = a.top_k;
    p.groups = a.groups;
    p.top_groups = a.top_groups;
    p.group_top = a.groups > 1 && a.top_groups < a.groups ? a.group_top : 1;
    p.each = a.experts / a.groups;
    int pow2 = 1;
    while (pow2 < a.groups) pow2 *= 2;
    p.lanes = 32 / pow2;
    while (1 << p.lane_bits < p.lanes) ++p.lane_bits;
    p.held = (p.each + p.lanes - 1) / p.lanes;
    p.sigmoid = a.sigmoid;
    p.renormalise = a.renormalise;
    p.scale = a.scale;
    return p;
}

template <typename T, int HELD>
void route_held(const RouteArgs &a, const RouteParams &p) {
    const unsigned grid = (unsigned)((a.tokens + kRouteWarps - 1) / kRouteWarps);
    constexpr size_t kBytes = HELD * sizeof(T) < 16 ? HELD * sizeof(T) : 16;
    constexpr bool kWhole = HELD >= 4 && kBytes == 16;   // (below, scalar loads are as good)
    if constexpr (kWhole) {
        if (p.lanes * p.held == p.each && p.held == HELD && p.lanes * p.groups == 32 &&
            reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.ld * sizeof(T) % 16 == 0 &&
            reinterpret_cast<uintptr_t>(a.bias) % 16 == 0) {
            route_kernel<T, HELD, true><<<grid, 32 * kRouteWarps, 0, a.stream>>>(p);
            return;
        }
    }
    route_kernel<T, HELD, false><<<grid, 32 * kRouteWarps, 0, a.stream>>>(p);
}

template <typename T>
cudaError_t route_typed(const RouteArgs &a) {
    const RouteParams p = params(a);
    if (p.held <= 1) route_held<T, 1>(a, p);
    else if (p.held <= 2) route_held<T, 2>(a, p);
    else if (p.held <= 4) route_held<T, 4>(a, p);
    else if (p.held <= 8) route_held<T, 8>(a, p);
    else if (p.held <= 16) route_held<T, 16>(a, p);
    else if (p.held <= 32) route_held<T, 32>(a, p);
    else route_held<T, 64>(a, p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t route_backward_typed(const RouteArgs &a) {
    const RouteParams p = params(a);
    const unsigned grid = (unsigned)((a.tokens + kRouteWarps - 1) / kRouteWarps);
    const int held = a.sigmoid || a.renormalise ? 1 : (a.experts + 31) / 32;
    constexpr int kBlock = 32 * kRouteWarps;
    if (held <= 1) route_backward_kernel<T, 1><<<grid, kBlock, 0, a.stream>>>(p);
    else if (held <= 2) route_backward_kernel<T, 2><<<grid, kBlock, 0, a.stream>>>(p);
    else if (held <= 4) route_backward_kernel<T, 4><<<grid, kBlock, 0, a.stream>>>(p);
    else if (held <= 8) route_backward_kernel<T, 8><<<grid, kBlock, 0, a.stream>>>(p);
    else if (held <= 16) route_backward_kernel<T, 16><<<grid, kBlock, 0, a.stream>>>(p);
    else route_backward_kernel<T, 32><<<grid, kBlock, 0, a.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a) {
    return a.dtype == PURLIN_F32 ? route_typed<float>(a) : route_typed<__nv_bfloat16>(a);
}

cudaError_t launch_route_backward(const RouteArgs &a) {
    return a.dtype == PURLIN_F32 ? route_backward_typed<float>(a) : route_backward_typed<__nv_bfloat16>(a);
}

}  // namespace purlin
