// grouped.cu -- matrix products grouped by expert with ragged row counts.
//
// out[j][i] = sum over k of A[i][k] B[j][k] for every group; layers.h names
// what A, B, i, j and k are in each mode.  Groups are (first row, row count)
// pairs in device memory, so the tiles of a launch are found on the device.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "layers.h"
#include "snac.cuh"

namespace purlin {
namespace {

struct GroupTable {
    int tiles[kMaxGroups + 1];   // tiles before group g
    int begin[kMaxGroups];
    int count[kMaxGroups];
    int bad;
};

// Read and check the groups; tiles[g] = tiles before group g, from
// tiles_of(count).  Every thread of the block calls it; false if a group lies
// outside the rows or the groups hold more rows than there are (so some
// overlap).
template <typename F>
__device__ bool read_groups(GroupTable &t, const int64_t *begin, const int64_t *count, int groups,
                            long long rows, F tiles_of) {
    if (threadIdx.x == 0) t.bad = 0;
    __syncthreads();
    for (int g = threadIdx.x; g < groups; g += blockDim.x) {
        const long long b = begin[g], c = count[g];
        // c > rows first: b + c does not overflow
        if (c < 0 || b < 0 || c > rows || b > rows - c) t.bad = 1;
        t.begin[g] = (int)b;
        t.count[g] = (int)c;
    }
    __syncthreads();
    if (t.bad) return false;
    if (threadIdx.x < 32) {
        int before = 0;
        long long held = 0;
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int g = g0 + (int)threadIdx.x;
            int v = g < groups ? tiles_of(t.count[g]) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if ((int)threadIdx.x >= o) v += u;
            }
            if (g < groups) {
                t.tiles[g + 1] = before + v;
                held += t.count[g];
            }
            before += __shfl_sync(0xffffffffu, v, 31);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) held += __shfl_xor_sync(0xffffffffu, held, o);
        if (threadIdx.x == 0) {
            t.tiles[0] = 0;
            if (held > rows) t.bad = 1;
        }
    }
    __syncthreads();
    return !t.bad;
}

// The group whose tiles include tile `t` (groups without tiles are skipped).
__device__ __forceinline__ int group_of(const GroupTable &t, int groups, int tile) {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (t.tiles[mid + 1] > tile) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

struct SimpleParams {
    const void *x, *w;
    void *y;
    const float *x_scales, *w_scales;
    const int64_t *begin, *count;
    size_t ldx, ldw, ldy;
    long long rows;
    int groups, n, k;
    unsigned long long *err;
};

template <typename T>
__device__ __forceinline__ float value(T v);
template <>
__device__ __forceinline__ float value<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float value<__nv_fp8_e4m3>(__nv_fp8_e4m3 v) { return (float)v; }

constexpr int kTile = 64, kStep = 16;

// 64 x 64 outputs a block at a time, 4 x 4 a thread, binary32 products.
template <typename T, int MODE>
__global__ void __launch_bounds__(256) grouped_simple_kernel(const __grid_constant__ SimpleParams p) {
    __shared__ GroupTable table;
    __shared__ float as[kStep][kTile + 1], bs[kStep][kTile + 1];
    const int ni = MODE == kGroupedGrad ? p.k : p.n;   // i extent
    const int i_tiles = (ni + kTile - 1) / kTile;
    const bool ok = read_groups(table, p.begin, p.count, p.groups, p.rows, [&](int c) {
        return (MODE == kGroupedGrad ? (p.n + kTile - 1) / kTile : (c + kTile - 1) / kTile) * i_tiles;
    });
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            snac::record_error(p.err, PURLIN_ERR_INVALID_ARG, snac::kSiteGroups, 0);
        return;
    }
    const T *x = static_cast<const T *>(p.x), *w = static_cast<const T *>(p.w);
    const int total = table.tiles[p.groups];
    const int ti = threadIdx.x & 15, tj = threadIdx.x >> 4;
    for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
        const int g = group_of(table, p.groups, tile);
        const int local = tile - table.tiles[g];
        const int i0 = (local % i_tiles) * kTile, j0 = (local / i_tiles) * kTile;
        const long long row0 = table.begin[g];
        const int nj = MODE == kGroupedGrad ? p.n : table.count[g];
        const int nk = MODE == kGroupedGrad ? table.count[g] : p.k;
        float acc[4][4] = {};
        for (int k0 = 0; k0 < nk; k0 += kStep) {
            for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
                // neighbouring threads along the axis that is contiguous in memory
                const int ka = MODE == kGroupedNK ? e % kStep : e / kTile;
                const int ia = MODE == kGroupedNK ? e / kStep : e % kTile;
                float a = 0.f;
                if (k0 + ka < nk && i0 + ia < ni) {
                    if constexpr (MODE == kGroupedNK)
                        a = value<T>(w[((size_t)g * p.n + i0 + ia) * p.ldw + k0 + ka]);
                    else if constexpr (MODE == kGroupedKN)
                        a = value<T>(w[((size_t)g * p.k + k0 + ka) * p.ldw + i0 + ia]);
                    else
                        a = value<T>(x[(size_t)(row0 + k0 + ka) * p.ldx + i0 + ia]);
                }
                as[ka][ia] = a;
                const int kb = MODE == kGroupedGrad ? e / kTile : e % kStep;
                const int jb = MODE == kGroupedGrad ? e % kTile : e / kStep;
                float b = 0.f;
                if (k0 + kb < nk && j0 + jb < nj) {
                    if constexpr (MODE == kGroupedGrad)
                        b = value<T>(w[(size_t)(row0 + k0 + kb) * p.ldw + j0 + jb]);
                    else
                        b = value<T>(x[(size_t)(row0 + j0 + jb) * p.ldx + k0 + kb]);
                }
                bs[kb][jb] = b;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kStep; ++k)
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        acc[u][v] = fmaf(as[k][ti + 16 * v], bs[k][tj + 16 * u], acc[u][v]);
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int i = i0 + ti + 16 * v, j = j0 + tj + 16 * u;
                if (i >= ni || j >= nj) continue;
                float o = acc[u][v];
                if constexpr (sizeof(T) == 1)
                    o = o * p.x_scales[row0 + j] * p.w_scales[(size_t)g * p.n + i];
                const size_t at = MODE == kGroupedGrad ? ((size_t)g * p.n + j) * p.ldy + i
                                                       : (size_t)(row0 + j) * p.ldy + i;
                static_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(o);
            }
    }
}

}  // namespace

cudaError_t launch_grouped(const GroupedArgs &a) {
    SimpleParams p{a.x,   a.w,   a.y,   a.x_scales, a.w_scales, a.begin, a.count, a.ldx, a.ldw,
                   a.ldy, (long long)a.rows, a.groups, (int)a.n, (int)a.k, a.err};
    const int grid = a.sms * 4;
    if (a.dtype == PURLIN_E4M3)
        grouped_simple_kernel<__nv_fp8_e4m3, kGroupedNK><<<grid, 256, 0, a.stream>>>(p);
    else if (a.mode == kGroupedNK)
        grouped_simple_kernel<__nv_bfloat16, kGroupedNK><<<grid, 256, 0, a.stream>>>(p);
    else if (a.mode == kGroupedKN)
        grouped_simple_kernel<__nv_bfloat16, kGroupedKN><<<grid, 256, 0, a.stream>>>(p);
    else
        grouped_simple_kernel<__nv_bfloat16, kGroupedGrad><<<grid, 256, 0, a.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace purlin
