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
// The rows' kernels are bound by bytes.  A thread has one access of a token's row (16
// bytes where pointers, pitches and columns allow, else the largest power of two that
// they do) and all of the token's places: dispatch loads once and stores top_k times,
// combine has top_k loads in flight and adds them up in their order in binary32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "layers.h"

namespace purlin {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ------------------------------------------------------------------- order --

constexpr int kOrderThreads = 256, kOrderWarps = kOrderThreads / 32;
constexpr int kOrderSlots = 2048;   // least slots of a block

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

// An access of W bytes.
template <int W>
struct Access;
template <>
struct Access<16> { using type = uint4; };
template <>
struct Access<8> { using type = uint2; };
template <>
struct Access<4> { using type = uint32_t; };
template <>
struct Access<2> { using type = uint16_t; };
template <>
struct Access<1> { using type = uint8_t; };

struct RowsParams {
    const char *x, *rows, *shared;
    const float *scales, *weights;
    const int32_t *place;
    char *out;
    float *out_scales;
    size_t ldx, ldr, lds, ldo;   // bytes
    size_t n_rows;
    int top_k, parts;            // parts: blocks of a token
    uint32_t accesses;           // of a row
};

__device__ __forceinline__ bool inside(int place, size_t rows) {
    return place >= 0 && (size_t)place < rows;
}

// EACH accesses a thread, a block apart; a place's share of the row is stored at once,
// place after place, so that the stores of a block run along a row.
template <int W, int EACH>
__global__ void dispatch_kernel(const __grid_constant__ RowsParams p) {
    using A = typename Access<W>::type;
    const size_t token = blockIdx.x / p.parts;
    const uint32_t part = blockIdx.x - (uint32_t)token * p.parts;
    const uint32_t first = part * blockDim.x * EACH + threadIdx.x;
    const int32_t *place = p.place + token * p.top_k;
    if (p.scales && part == 0 && threadIdx.x < p.top_k && inside(place[threadIdx.x], p.n_rows))
        p.out_scales[place[threadIdx.x]] = p.scales[token];
    A v[EACH];
#pragma unroll
    for (int u = 0; u < EACH; ++u)
        if (first + u * blockDim.x < p.accesses)
            v[u] = reinterpret_cast<const A *>(p.x + token * p.ldx)[first + u * blockDim.x];
    for (int j = 0; j < p.top_k; ++j) {
        const int to = place[j];
        if (!inside(to, p.n_rows)) continue;
        A *out = reinterpret_cast<A *>(p.out + (size_t)to * p.ldo);
#pragma unroll
        for (int u = 0; u < EACH; ++u)
            if (first + u * blockDim.x < p.accesses) out[first + u * blockDim.x] = v[u];
    }
}

// The N values of type T in an access.
template <typename T, int N>
struct Values {
    T v[N];
};

template <typename T>
__device__ __forceinline__ float as_float(T v);
template <>
__device__ __forceinline__ float as_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float as_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T, int W>
__device__ __forceinline__ void load(float (&f)[W / sizeof(T)], const char *row, uint32_t i) {
    using A = typename Access<W>::type;
    union {
        A a;
        T v[W / sizeof(T)];
    } u;
    u.a = reinterpret_cast<const A *>(row)[i];
#pragma unroll
    for (int q = 0; q < W / (int)sizeof(T); ++q) f[q] = as_float<T>(u.v[q]);
}
template <typename T, int W>
__device__ __forceinline__ void store(char *row, uint32_t i, const float (&f)[W / sizeof(T)]) {
    using A = typename Access<W>::type;
    union {
        A a;
        T v[W / sizeof(T)];
    } u;
#pragma unroll
    for (int q = 0; q < W / (int)sizeof(T); ++q) u.v[q] = rounded<T>(f[q]);
    reinterpret_cast<A *>(row)[i] = u.a;
}

template <typename T, int W>
__global__ void combine_kernel(const __grid_constant__ RowsParams p) {
    constexpr int N = W / sizeof(T);
    const size_t token = blockIdx.x / p.parts;
    const uint32_t part = blockIdx.x - (uint32_t)token * p.parts;
    const uint32_t i = part * blockDim.x + threadIdx.x;
    if (i >= p.accesses) return;
    float sum[N] = {};
    if (p.shared) load<T, W>(sum, p.shared + token * p.lds, i);
    for (int j = 0; j < p.top_k; ++j) {
        const int place = p.place[token * p.top_k + j];
        if (!inside(place, p.n_rows)) continue;
        const float w = p.weights ? p.weights[token * p.top_k + j] : 1.f;
        float v[N];
        load<T, W>(v, p.rows + (size_t)place * p.ldr, i);
#pragma unroll
        for (int q = 0; q < N; ++q) sum[q] = fmaf(w, v[q], sum[q]);
    }
    store<T, W>(p.out + token * p.ldo, i, sum);
}

// A block a token: for each of its places the row's gradient and the product with dy.
template <typename T, int W>
__global__ void combine_backward_kernel(const __grid_constant__ RowsParams p) {
    constexpr int N = W / sizeof(T);
    __shared__ float sums[2][32];   // places that are there take turns
    int turn = 0;
    const size_t token = blockIdx.x;
    const char *dy = p.x + token * p.ldx;
    const int warps = blockDim.x >> 5;
    for (int j = 0; j < p.top_k; ++j) {
        const size_t slot = token * p.top_k + j;
        const int place = p.place[slot];
        if (!inside(place, p.n_rows)) {
            if (threadIdx.x == 0) p.out_scales[slot] = 0.f;
            continue;
        }
        const float w = p.weights[slot];
        const char *row = p.rows + (size_t)place * p.ldr;
        float dot = 0.f;
        for (uint32_t i = threadIdx.x; i < p.accesses; i += blockDim.x) {
            float d[N], v[N];
            load<T, W>(d, dy, i);
            load<T, W>(v, row, i);
#pragma unroll
            for (int q = 0; q < N; ++q) {
                dot = fmaf(d[q], v[q], dot);
                d[q] *= w;
            }
            store<T, W>(p.out + (size_t)place * p.ldo, i, d);
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

// The largest access that the rows of every operand allow.
int width_of(const RowsParams &p, size_t row_bytes) {
    size_t all = 16 | row_bytes;
    for (const void *q : {(const void *)p.x, (const void *)p.rows, (const void *)p.shared, (const void *)p.out})
        all |= reinterpret_cast<uintptr_t>(q);
    for (size_t ld : {p.ldx, p.ldr, p.lds, p.ldo}) all |= ld;
    return (int)(all & (~all + 1));
}

RowsParams params(const RowsArgs &a, size_t es) {
    RowsParams p{};
    p.x = static_cast<const char *>(a.x);
    p.rows = static_cast<const char *>(a.rows);
    p.shared = static_cast<const char *>(a.shared);
    p.scales = a.scales;
    p.weights = a.weights;
    p.place = a.place;
    p.out = static_cast<char *>(a.out);
    p.out_scales = a.out_scales;
    p.ldx = a.x ? a.ldx * es : 0;
    p.ldr = a.rows ? a.ldr * es : 0;
    p.lds = a.shared ? a.lds * es : 0;
    p.ldo = a.ldo * es;
    p.n_rows = a.n_rows;
    p.top_k = a.top_k;
    return p;
}

// `each` accesses a thread: the blocks of a token, and their threads.
void spread(RowsParams &p, size_t tokens, uint32_t each, unsigned *grid, unsigned *block) {
    const uint32_t most = 256 * each;
    p.parts = (int)((p.accesses + most - 1) / most);
    if ((size_t)p.parts * tokens > 0x7FFFFFFFu) p.parts = 0;   // (more bytes than the GPU has)
    *block = p.parts ? ((p.accesses + p.parts * each - 1) / (p.parts * each) + 31) / 32 * 32 : 0;
    *grid = (unsigned)((size_t)p.parts * tokens);
}

size_t size_of(int dtype) { return dtype == PURLIN_F32 ? 4 : dtype == PURLIN_BF16 ? 2 : 1; }

template <typename T, typename F>
cudaError_t by_width(int width, F run) {
    if (width >= 16) return run(std::integral_constant<int, 16>());
    if (width == 8) return run(std::integral_constant<int, 8>());
    if constexpr (sizeof(T) <= 4)
        if (width == 4) return run(std::integral_constant<int, 4>());
    if constexpr (sizeof(T) <= 2)
        if (width == 2) return run(std::integral_constant<int, 2>());
    if constexpr (sizeof(T) == 1) return run(std::integral_constant<int, 1>());
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t combine_typed(const RowsArgs &a) {
    RowsParams p = params(a, sizeof(T));
    return by_width<T>(width_of(p, a.cols * sizeof(T)), [&](auto w) {
        constexpr int W = decltype(w)::value;
        p.accesses = (uint32_t)(a.cols * sizeof(T) / W);
        unsigned grid, block;
        spread(p, a.tokens, 1, &grid, &block);
        if (grid == 0) return cudaErrorInvalidConfiguration;
        combine_kernel<T, W><<<grid, block, 0, a.stream>>>(p);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t combine_backward_typed(const RowsArgs &a) {
    RowsParams p = params(a, sizeof(T));
    return by_width<T>(width_of(p, a.cols * sizeof(T)), [&](auto w) {
        constexpr int W = decltype(w)::value;
        p.accesses = (uint32_t)(a.cols * sizeof(T) / W);
        const unsigned block = std::min(256u, std::max(32u, (p.accesses + 31) / 32 * 32));
        combine_backward_kernel<T, W><<<(unsigned)a.tokens, block, 0, a.stream>>>(p);
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
    RowsParams p = params(a, size_of(a.dtype));
    const size_t row_bytes = a.cols * size_of(a.dtype);
    return by_width<char>(width_of(p, row_bytes), [&](auto w) {
        constexpr int W = decltype(w)::value;
        p.accesses = (uint32_t)(row_bytes / W);
        unsigned grid, block;
        const bool many = a.tokens * p.accesses >= (size_t)a.sms * 8192;
        spread(p, a.tokens, many ? 4 : 1, &grid, &block);
        if (grid == 0) return cudaErrorInvalidConfiguration;
        if (many) dispatch_kernel<W, 4><<<grid, block, 0, a.stream>>>(p);
        else dispatch_kernel<W, 1><<<grid, block, 0, a.stream>>>(p);
        return cudaGetLastError();
    });
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
