// expert_rows.cu -- the order of slots by expert, the copies of tokens' rows to their
// places in it, their weighted sum on the way back, and that sum's gradients.
//
// The order is a counting sort that keeps the slots' own order: a slot's place is its
// expert's first row, and the slots of that expert before it.  Slots are cut into one
// piece a block, pieces into one run a warp; counts of the runs, added up over the runs
// and pieces before, are where each run begins, and within 32 slots at a time the lanes
// of one expert rank themselves by a match over the warp.  Integers alone: the same
// places every time.
//
// The rows' kernels are bound by bytes.  A thread has windows of 16 bytes of a token's
// row and all of the token's places: dispatch loads once and stores top_k times, combine
// adds up the rows in their order in binary32, with many threads an SM for the loads in
// flight.  16384 tokens of eight places: dispatch of 7168 bytes and a scale 158 us (6.7
// TB/s) and the order 8.6 on the device, 13 with its two launches; combine of 7168 bf16 348
// us (6.1 TB/s); its backward pass of 4096 bf16 356 us (6.4 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "layers.h"

namespace purlin {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ------------------------------------------------------------------- order --

constexpr int kOrderThreads = 256, kOrderWarps = kOrderThreads / 32;
// Least slots of a block.  Fewer are more blocks, each of which adds up all the others'
// counts (131072 slots of 256 experts 8.6 us on the device, with 1024 10.0, with 4096 10.6;
// 4096 slots 6.9, 6.2 and 7.6; 2048, one launch, 4.5, 5.6 and 4.6).
constexpr int kOrderSlots = 2048;

struct OrderParams {
    const int32_t *chosen;
    int32_t *place;
    int64_t *begin, *count;
    int *partial;     // blocks x groups counts
    size_t slots;
    size_t capacity;
    int groups;
    int run;          // slots of a warp, a multiple of 32
};

// 32 kBatch slots of a warp's run, loaded together: -1 where there is none.
constexpr int kBatch = 8;

__device__ __forceinline__ void load_slots(const OrderParams &p, size_t from, int left, int (&e)[kBatch]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const size_t s = from + 32 * k + lane;
        const int v = 32 * k < left && s < p.slots ? p.chosen[s] : -1;
        e[k] = (unsigned)v < (unsigned)p.groups ? v : -1;
    }
}

// Counts of this warp's run into its row of `hist`, which is zero.
__device__ __forceinline__ void count_run(const OrderParams &p, int *hist) {
    const size_t from = ((size_t)blockIdx.x * kOrderWarps + (threadIdx.x >> 5)) * p.run;
    for (int i = 0; i < p.run; i += 32 * kBatch) {
        int e[kBatch];
        load_slots(p, from + i, p.run - i, e);
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (e[k] >= 0) atomicAdd(&hist[e[k]], 1);
    }
}

__global__ void __launch_bounds__(kOrderThreads)
order_count_kernel(const __grid_constant__ OrderParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the places may be launched
    extern __shared__ int hist[];
    for (int e = threadIdx.x; e < p.groups; e += kOrderThreads) hist[e] = 0;
    __syncthreads();
    count_run(p, hist);
    __syncthreads();
    for (int e = threadIdx.x; e < p.groups; e += kOrderThreads)
        p.partial[(size_t)blockIdx.x * p.groups + e] = hist[e];
}

// Shared memory: kOrderWarps x groups counts, then totals and counts of the blocks before.
// The first kOrderWarps warps have slots; where there are many blocks, as many more help
// to add up their counts, eight loads at once (64 blocks of 256 threads, a thread an
// expert, took 14 us over it).
constexpr int kPlaceThreads = 1024, kAtOnce = 8;

__global__ void __launch_bounds__(kPlaceThreads)
order_place_kernel(const __grid_constant__ OrderParams p) {
    extern __shared__ int hist[];
    __shared__ long long warp_total[kOrderWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = p.groups, threads = (int)blockDim.x;
    int *total = hist + kOrderWarps * groups, *earlier = total + groups;
    int *own = hist + warp * groups;
    for (int e = threadIdx.x; e < (kOrderWarps + 2) * groups; e += threads) hist[e] = 0;
    __syncthreads();
    if (warp < kOrderWarps) count_run(p, own);
    // launched while the other blocks' counts are still being taken: wait for all of them
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (gridDim.x > 1) {
        const int blocks = (int)gridDim.x, pieces = (blocks + kAtOnce - 1) / kAtOnce;
        for (int i = threadIdx.x; i < groups * pieces; i += threads) {
            const int piece = i / groups, e = i - piece * groups;
            int c[kAtOnce], before = 0, sum = 0;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int b = min(piece * kAtOnce + k, blocks - 1);
                c[k] = p.partial[(size_t)b * groups + e];
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int b = piece * kAtOnce + k;
                sum += b < blocks ? c[k] : 0;
                before += b < (int)blockIdx.x ? c[k] : 0;
            }
            atomicAdd(&total[e], sum);   // (whole numbers: in any order)
            atomicAdd(&earlier[e], before);
        }
    }
    __syncthreads();
    // the run's counts become the slots of the expert before it
    for (int e = threadIdx.x; e < groups; e += threads) {
        int before = earlier[e];
        for (int w = 0; w < kOrderWarps; ++w) {
            const int c = hist[w * groups + e];
            hist[w * groups + e] = before;
            before += c;
        }
        if (gridDim.x == 1) total[e] = before;
    }
    __syncthreads();
    // the experts' first rows: capacities, or the totals before, a piece of them a thread
    const int each = (groups + kOrderThreads - 1) / kOrderThreads;
    const int first = min(groups, (int)threadIdx.x * each), last = min(groups, first + each);
    long long sum = 0;
    for (int e = first; e < last; ++e) sum += total[e];
    long long scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(kAll, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31 && warp < kOrderWarps) warp_total[warp] = scan;
    __syncthreads();
    long long at = scan - sum;
    for (int w = 0; w < min(warp, kOrderWarps); ++w) at += warp_total[w];
    for (int e = first; e < last; ++e) {
        const int n = total[e];
        const long long row = p.capacity ? (long long)e * (long long)p.capacity : at;
        if (blockIdx.x == 0) {
            p.begin[e] = row;
            p.count[e] = p.capacity && n > (long long)p.capacity ? (long long)p.capacity : n;
        }
        total[e] = (int)row;
        at += n;
    }
    __syncthreads();
    if (warp >= kOrderWarps) return;
    const size_t from = ((size_t)blockIdx.x * kOrderWarps + warp) * p.run;
    for (int i = 0; i < p.run; i += 32 * kBatch) {
        int e[kBatch];
        unsigned alike[kBatch];
        load_slots(p, from + i, p.run - i, e);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) alike[k] = __match_any_sync(kAll, e[k]);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int rank = e[k] >= 0 ? own[e[k]] + __popc(alike[k] & ((1u << lane) - 1)) : 0;
            __syncwarp();
            if (e[k] >= 0 && (alike[k] >> lane) == 1) own[e[k]] = rank + 1;   // the last lane of its expert
            __syncwarp();
            const size_t s = from + i + 32 * k + lane;
            if (i + 32 * k < p.run && s < p.slots)
                p.place[s] = e[k] >= 0 && (p.capacity == 0 || rank < (long long)p.capacity) ? total[e[k]] + rank : -1;
        }
    }
}

int order_blocks(const OrderArgs &a) {
    const size_t pieces = (a.slots + kOrderSlots - 1) / kOrderSlots;
    return (int)std::max<size_t>(1, std::min<size_t>(pieces, (size_t)a.sms));
}

// -------------------------------------------------------------------- rows --

// Rows are read and written in windows of W bytes, 16, 8 or 4, the most that pointers,
// pitches and columns allow.  W 0, where that is too little: windows of 16 bytes on the
// boundaries of the row that is written; a row that is read is put in step from two loads,
// whose second another thread's first brought into the cache.  At a row's ends they bring
// bytes of the rows beside it, which go nowhere; at the matrix's own ends windows are read
// element by element, and at a row's written word by word and byte by byte.
// What is too little was measured, 16384 tokens of eight places: windows of 4 bytes lose in
// combine (2050 bf16 162 us, out of step 134; 1021 f32 150 and 129) and in copies of bf16
// and f32 (8000 x 4098 135 and 121), and win in copies of bytes (1020 50 and 81) and in the
// backward pass, which has two rows to put in step (2050 bf16 355 and 477); windows of 8
// win or are level.  Element by element bf16 of 1021 columns took 134 us (now 75), backward
// 290 (239).
template <int W>
struct Words {
    uint32_t w[W ? W / 4 : 4];
};

struct RowsParams {
    const char *x, *rows, *shared;
    const char *x_end, *rows_end, *shared_end;   // of the matrices
    const float *scales, *weights;
    const int32_t *place;
    char *out;
    float *out_scales;
    size_t ldx, ldr, lds, ldo;   // bytes
    size_t n_rows, tokens;
    int top_k, parts;            // parts: blocks of a token (backward: places of a block)
    int64_t row_bytes;
    uint32_t windows;            // of a row, at the worst place
};

__device__ __forceinline__ bool inside(int place, size_t rows) {
    return place >= 0 && (size_t)place < rows;
}

// Bytes from a row's start to its window i, on the boundaries of `row`.
template <int W>
__device__ __forceinline__ int64_t window_at(const char *row, uint32_t i) {
    if constexpr (W == 0) return (int64_t)i * 16 - (int64_t)(reinterpret_cast<uintptr_t>(row) & 15);
    return (int64_t)i * W;
}

template <int W>
__device__ __forceinline__ Words<W> load_words(const char *p) {
    Words<W> v;
    if constexpr (W == 16 || W == 0) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
    } else if constexpr (W == 8) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        v.w[0] = u.x, v.w[1] = u.y;
    } else {
        v.w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
    return v;
}

// A window of a row from `at` on; ES bytes an element.  W 0: of a matrix from `base` to
// `end`; what lies outside the row is not said.
template <int W, int ES>
__device__ __forceinline__ Words<W> read_window(const char *row, int64_t at, int64_t bytes, const char *base,
                                                const char *end) {
    if constexpr (W != 0) {
        return load_words<W>(row + at);
    } else {
        const int off = (int)(reinterpret_cast<uintptr_t>(row + at) & 15);
        const char *p = row + at - off;
        uint32_t w[8] = {};
        if (p >= base && p + 32 <= end) {
            const Words<W> a = load_words<W>(p), b = load_words<W>(p + 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = a.w[i];
                w[i + 4] = b.w[i];
            }
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (off & 3) * 8);
        } else {
#pragma unroll
            for (int j = 0; j < 16 / ES; ++j) {
                const int64_t e = at + j * ES;
                if (e < 0 || e >= bytes) continue;
                uint32_t v;
                if constexpr (ES == 4) v = *reinterpret_cast<const uint32_t *>(row + e);
                else if constexpr (ES == 2) v = *reinterpret_cast<const uint16_t *>(row + e);
                else v = *reinterpret_cast<const uint8_t *>(row + e);
                w[j * ES / 4] |= v << (j * ES % 4 * 8);
            }
        }
        return Words<W>{{w[0], w[1], w[2], w[3]}};
    }
}

template <int W, int ES>
__device__ __forceinline__ void write_window(char *row, int64_t at, int64_t bytes, const Words<W> &v) {
    if constexpr (W == 8) {
        *reinterpret_cast<uint2 *>(row + at) = make_uint2(v.w[0], v.w[1]);
    } else if constexpr (W == 4) {
        *reinterpret_cast<uint32_t *>(row + at) = v.w[0];
    } else if (W == 16 || (at >= 0 && at + 16 <= bytes)) {
        *reinterpret_cast<uint4 *>(row + at) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    } else if constexpr (W == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t word = at + 4 * q;
            if (word >= 0 && word + 4 <= bytes) {
                *reinterpret_cast<uint32_t *>(row + word) = v.w[q];
                continue;
            }
            if constexpr (ES == 4) continue;
#pragma unroll
            for (int j = 0; j < 4 / ES; ++j) {
                const int64_t e = word + j * ES;
                if (e < 0 || e >= bytes) continue;
                if constexpr (ES == 2) *reinterpret_cast<uint16_t *>(row + e) = (uint16_t)(v.w[q] >> (16 * j));
                else *reinterpret_cast<uint8_t *>(row + e) = (uint8_t)(v.w[q] >> (8 * j));
            }
        }
    }
}

// blockDim.y tokens a block, or `parts` blocks a token; EACH windows a thread, a block
// apart.  A place's share of the row is stored at once, place after place, so that the
// stores of a block run along a row.  In step, x is loaded once for all of the places.
template <int W, int ES, int EACH>
__global__ void dispatch_kernel(const __grid_constant__ RowsParams p) {
    const uint32_t unit = blockIdx.x / p.parts, part = blockIdx.x - unit * p.parts;
    const size_t token = (size_t)unit * blockDim.y + threadIdx.y;
    if (token >= p.tokens) return;
    const uint32_t first = part * blockDim.x * EACH + threadIdx.x;
    const int32_t *place = p.place + token * p.top_k;
    const char *x = p.x + token * p.ldx;
    if (p.scales && part == 0)
        for (int j = threadIdx.x; j < p.top_k; j += (int)blockDim.x)
            if (inside(place[j], p.n_rows)) p.out_scales[place[j]] = p.scales[token];
    Words<W> v[EACH];
    if constexpr (W != 0) {
#pragma unroll
        for (int u = 0; u < EACH; ++u)
            if (first + u * blockDim.x < p.windows)
                v[u] = read_window<W, ES>(x, window_at<W>(x, first + u * blockDim.x), p.row_bytes, p.x, p.x_end);
    }
    for (int j = 0; j < p.top_k; ++j) {
        const int to = place[j];
        if (!inside(to, p.n_rows)) continue;
        char *out = p.out + (size_t)to * p.ldo;
        if constexpr (W == 0) {
#pragma unroll
            for (int u = 0; u < EACH; ++u)
                v[u] = read_window<W, ES>(x, window_at<W>(out, first + u * blockDim.x), p.row_bytes, p.x, p.x_end);
        }
#pragma unroll
        for (int u = 0; u < EACH; ++u)
            if (first + u * blockDim.x < p.windows)
                write_window<W, ES>(out, window_at<W>(out, first + u * blockDim.x), p.row_bytes, v[u]);
    }
}

// A window's values.
template <typename T, int W>
__device__ __forceinline__ void unpack(const Words<W> &u, float *f) {
#pragma unroll
    for (int q = 0; q < (int)(sizeof(u.w) / 4); ++q) {
        if constexpr (sizeof(T) == 4) {
            f[q] = __uint_as_float(u.w[q]);
        } else {
            f[2 * q] = __uint_as_float(u.w[q] << 16);
            f[2 * q + 1] = __uint_as_float(u.w[q] & 0xFFFF0000u);
        }
    }
}
template <typename T, int W>
__device__ __forceinline__ Words<W> pack(const float *f) {
    Words<W> u;
#pragma unroll
    for (int q = 0; q < (int)(sizeof(u.w) / 4); ++q) {
        if constexpr (sizeof(T) == 4) {
            u.w[q] = __float_as_uint(f[q]);
        } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
            u.w[q] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
    return u;
}

// A thread a window of y; tokens and blocks as above.  (Loads of four rows at a time, ahead
// of their sums, are slower: 16384 x 7168 bf16 of eight places 434 us, so 348.)
template <typename T, int W>
__global__ void combine_kernel(const __grid_constant__ RowsParams p) {
    constexpr int ES = sizeof(T), N = sizeof(Words<W>) / ES;
    const uint32_t unit = blockIdx.x / p.parts, part = blockIdx.x - unit * p.parts;
    const size_t token = (size_t)unit * blockDim.y + threadIdx.y;
    const uint32_t i = part * blockDim.x + threadIdx.x;
    if (token >= p.tokens || i >= p.windows) return;
    char *out = p.out + token * p.ldo;
    const int64_t at = window_at<W>(out, i);
    float sum[N] = {};
    if (p.shared) unpack<T>(read_window<W, ES>(p.shared + token * p.lds, at, p.row_bytes, p.shared, p.shared_end), sum);
    for (int j = 0; j < p.top_k; ++j) {
        const int place = p.place[token * p.top_k + j];
        if (!inside(place, p.n_rows)) continue;
        const float w = p.weights ? p.weights[token * p.top_k + j] : 1.f;
        float f[N];
        unpack<T>(read_window<W, ES>(p.rows + (size_t)place * p.ldr, at, p.row_bytes, p.rows, p.rows_end), f);
#pragma unroll
        for (int q = 0; q < N; ++q) sum[q] = fmaf(w, f[q], sum[q]);
    }
    write_window<W, ES>(out, at, p.row_bytes, pack<T, W>(sum));
}

// For a place: the row's gradient and the product with dy.  A block has a token, which
// reads dy once, or a place where there are too few tokens for the SMs (64 tokens of eight
// places x 4096 bf16 5.8 us, a block a token 10.5); `parts` places a block.
template <typename T, int W>
__global__ void combine_backward_kernel(const __grid_constant__ RowsParams p) {
    constexpr int ES = sizeof(T), N = sizeof(Words<W>) / ES;
    __shared__ float sums[2][32];   // places that are there take turns
    int turn = 0;
    const int warps = blockDim.x >> 5;
    for (int j = 0; j < p.parts; ++j) {
        const size_t slot = (size_t)blockIdx.x * p.parts + j;
        const char *dy = p.x + slot / p.top_k * p.ldx;
        const int place = p.place[slot];
        if (!inside(place, p.n_rows)) {
            if (threadIdx.x == 0) p.out_scales[slot] = 0.f;
            continue;
        }
        const float w = p.weights[slot];
        const char *row = p.rows + (size_t)place * p.ldr;
        char *out = p.out + (size_t)place * p.ldo;
        float dot = 0.f;
        for (uint32_t i = threadIdx.x; i < p.windows; i += blockDim.x) {
            const int64_t at = window_at<W>(out, i);
            float d[N], v[N];
            unpack<T>(read_window<W, ES>(dy, at, p.row_bytes, p.x, p.x_end), d);
            unpack<T>(read_window<W, ES>(row, at, p.row_bytes, p.rows, p.rows_end), v);
            if (W == 0 && (at < 0 || at + 16 > p.row_bytes)) {
#pragma unroll
                for (int q = 0; q < N; ++q)
                    if (at + q * ES < 0 || at + q * ES >= p.row_bytes) d[q] = v[q] = 0.f;
            }
#pragma unroll
            for (int q = 0; q < N; ++q) {
                dot = fmaf(d[q], v[q], dot);
                d[q] *= w;
            }
            write_window<W, ES>(out, at, p.row_bytes, pack<T, W>(d));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
        if ((threadIdx.x & 31) == 0) sums[turn][threadIdx.x >> 5] = dot;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int k = 1; k < warps; ++k) dot += sums[turn][k];
            p.out_scales[slot] = dot;
        }
        turn ^= 1;
    }
}

// A launch's parameters; the windows' bytes, 0 where they would be fewer than `least`.
int params(const RowsArgs &a, size_t es, int least, RowsParams *p) {
    *p = RowsParams{};
    p->x = static_cast<const char *>(a.x);
    p->rows = static_cast<const char *>(a.rows);
    p->shared = static_cast<const char *>(a.shared);
    p->scales = a.scales;
    p->weights = a.weights;
    p->place = a.place;
    p->out = static_cast<char *>(a.out);
    p->out_scales = a.out_scales;
    p->ldx = a.x ? a.ldx * es : 0;
    p->ldr = a.rows ? a.ldr * es : 0;
    p->lds = a.shared ? a.lds * es : 0;
    p->ldo = a.ldo * es;
    p->n_rows = a.n_rows;
    p->tokens = a.tokens;
    p->top_k = a.top_k;
    const size_t bytes = a.cols * es;
    p->x_end = p->x + (a.tokens - 1) * p->ldx + bytes;
    p->shared_end = p->shared + (a.tokens - 1) * p->lds + bytes;
    p->rows_end = p->rows + (a.n_rows ? a.n_rows - 1 : 0) * p->ldr + bytes;
    size_t all = 16 | bytes | p->ldx | p->ldr | p->lds | p->ldo;
    for (const void *q : {a.x, a.rows, a.shared, (const void *)a.out}) all |= reinterpret_cast<uintptr_t>(q);
    const int most = (int)(all & (~all + 1)), width = most >= least ? most : 0;
    p->row_bytes = (int64_t)bytes;
    p->windows = (uint32_t)(width ? bytes / width : (bytes + 30) / 16);
    return width;
}

// `each` windows a thread: the tokens of a block, or the blocks of a token.
bool spread(RowsParams &p, uint32_t each, unsigned *grid, dim3 *block) {
    const uint32_t most = 256 * each;
    p.parts = (int)((p.windows + most - 1) / most);
    uint32_t x = (p.windows + p.parts * each - 1) / (p.parts * each);
    if (x > 16) {
        x = (x + 31) / 32 * 32;
    } else {   // parts of a warp
        uint32_t pow2 = 1;
        while (pow2 < x) pow2 *= 2;
        x = pow2;
    }
    *block = dim3(x, 256 / x);
    const size_t units = (p.tokens + block->y - 1) / block->y;
    *grid = (unsigned)(units * p.parts);
    return units * p.parts <= 0x7FFFFFFFu;   // (else they have more bytes than the GPU)
}

template <int ES, int LEAST, typename F>
cudaError_t by_width(int width, F run) {
    if (width == 16) return run(std::integral_constant<int, 16>());
    if (width == 8) return run(std::integral_constant<int, 8>());
    if constexpr (LEAST <= 4)
        if (width == 4) return run(std::integral_constant<int, 4>());
    if constexpr (LEAST > ES) return run(std::integral_constant<int, 0>());
    return cudaErrorInvalidValue;
}

template <int ES>
cudaError_t dispatch_typed(const RowsArgs &a) {
    constexpr int kLeast = ES == 1 ? 4 : 8;
    RowsParams p;
    return by_width<ES, kLeast>(params(a, ES, kLeast, &p), [&](auto width) {
        constexpr int W = decltype(width)::value;
        // four windows a thread where blocks are many and rows fill them: a token's places
        // are read once for four times the bytes (16384 x 7168 e4m3 to one place each 37.6 us,
        // a window a thread 41.1; two places 55.3 and 55.5; eight 164 and 162; 128 tokens of
        // eight 6.2 and 4.2)
        const bool many = a.tokens * p.windows >= (size_t)a.sms * 8192 && p.windows >= 256;
        unsigned grid;
        dim3 block;
        if (!spread(p, many ? 4 : 1, &grid, &block)) return cudaErrorInvalidConfiguration;
        if (many) dispatch_kernel<W, ES, 4><<<grid, block, 0, a.stream>>>(p);
        else dispatch_kernel<W, ES, 1><<<grid, block, 0, a.stream>>>(p);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t combine_typed(const RowsArgs &a) {
    RowsParams p;
    return by_width<sizeof(T), 8>(params(a, sizeof(T), 8, &p), [&](auto width) {
        unsigned grid;
        dim3 block;
        if (!spread(p, 1, &grid, &block)) return cudaErrorInvalidConfiguration;
        combine_kernel<T, decltype(width)::value><<<grid, block, 0, a.stream>>>(p);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t combine_backward_typed(const RowsArgs &a) {
    RowsParams p;
    return by_width<sizeof(T), 4>(params(a, sizeof(T), 4, &p), [&](auto width) {
        p.parts = a.tokens < 4 * (size_t)a.sms ? 1 : a.top_k;
        const unsigned grid = (unsigned)(a.tokens * a.top_k / p.parts);
        const unsigned block = std::min(256u, std::max(32u, (p.windows + 31) / 32 * 32));
        combine_backward_kernel<T, decltype(width)::value><<<grid, block, 0, a.stream>>>(p);
        return cudaGetLastError();
    });
}

}  // namespace

size_t expert_order_workspace(const OrderArgs &a) {
    const int blocks = order_blocks(a);
    return blocks > 1 ? (size_t)blocks * a.groups * sizeof(int) : 0;
}

cudaError_t launch_expert_order(const OrderArgs &a) {
    const int blocks = order_blocks(a);
    const size_t runs = (size_t)blocks * kOrderWarps;
    const size_t run = ((a.slots + runs - 1) / runs + 31) / 32 * 32;
    const OrderParams p{a.chosen, a.place, a.begin, a.count, a.partial, a.slots, a.capacity, a.groups, (int)run};
    const int smem = (kOrderWarps + 2) * a.groups * (int)sizeof(int);   // 40 KiB at most
    if (blocks > 1) {
        order_count_kernel<<<blocks, kOrderThreads, a.groups * sizeof(int), a.stream>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    // its launch overlaps the counts' kernel, which every kernel before it precedes
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)blocks);
    c.blockDim = dim3(blocks > 1 ? kPlaceThreads : kOrderThreads);
    c.dynamicSmemBytes = (size_t)smem;
    c.stream = a.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = blocks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&c, order_place_kernel, p);
}

cudaError_t launch_dispatch_rows(const RowsArgs &a) {
    return a.dtype == PURLIN_F32    ? dispatch_typed<4>(a)
           : a.dtype == PURLIN_BF16 ? dispatch_typed<2>(a)
                                    : dispatch_typed<1>(a);
}

cudaError_t launch_combine_rows(const RowsArgs &a) {
    return a.dtype == PURLIN_F32 ? combine_typed<float>(a) : combine_typed<__nv_bfloat16>(a);
}

cudaError_t launch_combine_rows_backward(const RowsArgs &a) {
    if (a.cols == 0)
        return cudaMemsetAsync(a.out_scales, 0, a.tokens * (size_t)a.top_k * sizeof(float), a.stream);
    return a.dtype == PURLIN_F32 ? combine_backward_typed<float>(a)
                                 : combine_backward_typed<__nv_bfloat16>(a);
}

}  // namespace purlin
