// grouped.cu -- matrix products grouped by expert with ragged row counts.
//
// out[j][i] = sum over k of A[i][k] B[j][k] for every group; layers.h names
// what A, B, i, j and k are in each mode.  Groups are (first row, row count)
// pairs in device memory, so the tiles of a launch are found on the device.
//
// One persistent CTA an SM.  A tile is 128 i by up to 256 j: the weights'
// channels take the tensor core's 128-lane side and the group's rows the other,
// whose width is a field of the instruction, so a group of 5 rows costs a
// 16-column product, not a padded one, and the same code serves one token and a
// prefill.  A warp brings 128-byte-wide boxes of both operands into a ring of
// shared-memory stages (TMA, 128-byte swizzle), a warp issues tcgen05.mma from
// them into one of two accumulators in tensor memory, and four warps write the
// other accumulator out meanwhile.
//
// With fewer tiles than SMs (decode) K is split over the idle CTAs: each
// writes its binary32 accumulator to a workspace, and the last of a tile's CTAs
// to arrive adds them in split order, so the result does not depend on which
// came last.
//
// kGroupedGrad sums over a group's rows: both operands then lie along M or N in
// memory (MN-major), and the last block of rows is cut at the group's end by
// clearing its rows in shared memory, since rows of no group may hold anything.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "layers.h"
#include "snac.cuh"
#include "tensor.cuh"

namespace purlin {
namespace {

struct GroupTable {
    int tiles[kMaxGroups + 1];   // tiles before group g
    int begin[kMaxGroups];
    int count[kMaxGroups];
    int most;                    // rows of the largest group
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
        int most = 0;
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
                most = max(most, t.count[g]);
            }
            before += __shfl_sync(0xffffffffu, v, 31);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            held += __shfl_xor_sync(0xffffffffu, held, o);
            most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        }
        if (threadIdx.x == 0) {
            t.tiles[0] = 0;
            t.most = most;
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

constexpr int kStages = 4;
constexpr int kTileI = 128, kTileJ = 256;
constexpr int kRowBytes = 128;                    // a stage's extent along a swizzled row
constexpr int kABytes = kTileI * kRowBytes;       // 16 KiB a stage
constexpr int kBBytes = kTileJ * kRowBytes;       // 32 KiB a stage
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kBoxJ = 32;                         // rows of a K-major box of B
constexpr int kBoxBytes = 64 * kRowBytes;         // MN-major box: 64 elements by 64 k
constexpr int kMaxSplits = 16;
constexpr int kThreads = 192;
constexpr uint32_t kSmem = kStages * kStageBytes + 1024;

struct TcParams {
    CUtensorMap a, b;
    __nv_bfloat16 *out;
    const float *x_scales, *w_scales;
    const int64_t *begin, *count;
    float *partial;       // gridDim.x accumulators of kTileJ x kTileI
    unsigned *arrived;    // gridDim.x, zero between launches
    size_t ldy;
    long long rows;
    int groups, ni, n, k;
    unsigned long long *err;
};

struct TcShared {
    GroupTable table;
    snac::Ctl ctl;
    uint64_t full[kStages], empty[kStages];   // stage loaded; stage consumed
    uint64_t done[2], free[2];                // accumulator complete; accumulator read
    uint64_t drain;
    uint32_t tmem;
    int last;
};

// One CTA's share of a tile: blocks [kb0, kb1) of the K axis.
struct Unit {
    int g, i0, j0, nj;   // nj: valid columns, up to kTileJ
    int row0;            // first row of the group
    int nk;              // K extent
    int kb0, kb1;
    int tile, split;
};

template <int MODE, int BK>
__device__ __forceinline__ Unit unit_at(const TcParams &p, const GroupTable &t, int u, int splits,
                                        int i_tiles) {
    Unit q;
    q.tile = u / splits;
    q.split = u - q.tile * splits;
    q.g = group_of(t, p.groups, q.tile);
    const int local = q.tile - t.tiles[q.g];
    const int jt = local / i_tiles;
    q.i0 = (local - jt * i_tiles) * kTileI;
    q.j0 = jt * kTileJ;
    q.row0 = t.begin[q.g];
    q.nj = min(kTileJ, (MODE == kGroupedGrad ? p.n : t.count[q.g]) - q.j0);
    q.nk = MODE == kGroupedGrad ? t.count[q.g] : p.k;
    const int blocks = (q.nk + BK - 1) / BK;
    q.kb0 = (int)((long long)blocks * q.split / splits);
    q.kb1 = (int)((long long)blocks * (q.split + 1) / splits);
    return q;
}

template <int MODE, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
grouped_tc_kernel(const __grid_constant__ TcParams p) {
    constexpr int BK = BF16 ? 64 : 128;        // K elements a stage
    constexpr int KSTEP = BF16 ? 16 : 32;      // K elements an instruction
    constexpr bool A_MN = MODE != kGroupedNK, B_MN = MODE == kGroupedGrad;
    extern __shared__ unsigned char raw[];
    __shared__ TcShared s;
    const uint32_t stage0 = (atom::smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0 && lane == 0) {
        tensor::prefetch_map(&p.a);
        tensor::prefetch_map(&p.b);
        for (int i = 0; i < kStages; ++i) {
            atom::mbar_init(&s.full[i], 1);
            atom::mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            atom::mbar_init(&s.done[i], 1);
            atom::mbar_init(&s.free[i], 4);
        }
        atom::mbar_init(&s.drain, 1);
        atom::mbar_init_fence();
        s.ctl.abort = 0;
    }
    const int i_tiles = (p.ni + kTileI - 1) / kTileI;
    const bool ok = read_groups(s.table, p.begin, p.count, p.groups, p.rows, [&](int c) {
        return ((MODE == kGroupedGrad ? p.n : c) + kTileJ - 1) / kTileJ * i_tiles;
    });
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            snac::record_error(p.err, PURLIN_ERR_INVALID_ARG, snac::kSiteGroups, 0);
        return;
    }
    const int tiles = s.table.tiles[p.groups];
    // Splits of K: as many as the grid has CTAs for, at least four blocks each.
    const int blocks = ((MODE == kGroupedGrad ? s.table.most : p.k) + BK - 1) / BK;
    const int splits =
        tiles == 0 ? 1
                   : max(1, min(min((int)gridDim.x / tiles, kMaxSplits), blocks / 4));
    const int units = tiles * splits;
    if ((int)blockIdx.x >= units) return;

    if (warp == 1) tensor::tmem_alloc(&s.tmem, 512);
    tensor::fence_before_sync();
    __syncthreads();
    tensor::fence_after_sync();
    const uint32_t tmem = s.tmem;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return snac::ring_wait(bar, parity, &s.ctl, p.err, snac::kSiteGroupedWait, true);
    };
    // one answer for the warp, whichever lanes saw the wait expire
    auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    uint32_t filled = 0;   // stages that warp 0's lane 0 has filled

    if (warp == 0) {
        // ---- load
        if (lane == 0) {
            uint32_t &it = filled;
            bool run = true;
            for (int u = blockIdx.x; u < units && run; u += gridDim.x) {
                const Unit q = unit_at<MODE, BK>(p, s.table, u, splits, i_tiles);
                const int boxes = B_MN ? (q.nj + 63) / 64 : (q.nj + kBoxJ - 1) / kBoxJ;
                const uint32_t bytes = kABytes + boxes * (B_MN ? kBoxBytes : kBoxJ * kRowBytes);
                for (int kb = q.kb0; kb < q.kb1; ++kb, ++it) {
                    const uint32_t st = it % kStages;
                    if (!wait(&s.empty[st], ((it / kStages) & 1) ^ 1)) {
                        run = false;
                        break;
                    }
                    const uint32_t bar = atom::smem_u32(&s.full[st]);
                    const uint32_t a = stage0 + st * kStageBytes, b = a + kABytes;
                    atom::mbar_arrive_expect_tx(&s.full[st], bytes);
                    if constexpr (MODE == kGroupedNK) {
                        tensor::load_box_3d(a, &p.a, kb * BK, q.i0, q.g, bar);
                    } else if constexpr (MODE == kGroupedKN) {
                        for (int h = 0; h < 2; ++h)
                            tensor::load_box_3d(a + h * kBoxBytes, &p.a, q.i0 + 64 * h, kb * BK,
                                                q.g, bar);
                    } else {
                        for (int h = 0; h < 2; ++h)
                            tensor::load_box_2d(a + h * kBoxBytes, &p.a, q.i0 + 64 * h,
                                                q.row0 + kb * BK, bar);
                    }
                    for (int h = 0; h < boxes; ++h) {
                        if constexpr (B_MN)
                            tensor::load_box_2d(b + h * kBoxBytes, &p.b, q.j0 + 64 * h,
                                                q.row0 + kb * BK, bar);
                        else
                            tensor::load_box_2d(b + h * kBoxJ * kRowBytes, &p.b, kb * BK,
                                                q.row0 + q.j0 + kBoxJ * h, bar);
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ---- multiply
        uint32_t it = 0, acc = 0;
        bool run = true;
        for (int u = blockIdx.x; u < units && run; u += gridDim.x) {
            const Unit q = unit_at<MODE, BK>(p, s.table, u, splits, i_tiles);
            if (q.kb0 == q.kb1) continue;   // an empty group, or a split with no block
            const uint32_t buf = acc & 1;
            if (!wait_warp(&s.free[buf], ((acc >> 1) & 1) ^ 1)) break;
            ++acc;
            tensor::fence_after_sync();
            const uint32_t d = tmem + buf * kTileJ;
            const uint32_t idesc =
                tensor::instr_desc(BF16 ? 1 : 0, A_MN, B_MN, kTileI, (q.nj + 15) & ~15);
            for (int kb = q.kb0; kb < q.kb1; ++kb, ++it) {
                const uint32_t st = it % kStages;
                if (!wait_warp(&s.full[st], (it / kStages) & 1)) {
                    run = false;
                    break;
                }
                tensor::fence_after_sync();
                const uint32_t a = stage0 + st * kStageBytes, b = a + kABytes;
                const int left = min(BK, q.nk - kb * BK);
                const int steps = (left + KSTEP - 1) / KSTEP;
                if constexpr (MODE == kGroupedGrad) {
                    // rows past the group's end inside the last instruction's 16
                    if (left < steps * KSTEP) {
                        const int quads = (steps * KSTEP - left) * (kRowBytes / 16);
                        const int boxes = 2 + (q.nj + 63) / 64;
                        for (int e = lane; e < quads * boxes; e += 32) {
                            const int box = e / quads, at = e - box * quads;
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             a + box * kBoxBytes + left * kRowBytes + at * 16),
                                         "r"(0)
                                         : "memory");
                        }
                        tensor::fence_async_shared();
                        __syncwarp();
                    }
                }
                if (lane == 0) {
                    const uint64_t da = tensor::operand_desc(a, kBoxBytes);
                    const uint64_t db = tensor::operand_desc(b, kBoxBytes);
                    for (int k = 0; k < steps; ++k) {
                        // K-major: 32 bytes on along the row; MN-major: 16 rows on
                        const uint64_t oa = (uint64_t)k * (A_MN ? 16 * kRowBytes : 32) >> 4;
                        const uint64_t ob = (uint64_t)k * (B_MN ? 16 * kRowBytes : 32) >> 4;
                        tensor::mma<BF16>(d, da + oa, db + ob, idesc, kb > q.kb0 || k > 0);
                    }
                    tensor::commit(atom::smem_u32(&s.empty[st]));
                    if (kb + 1 == q.kb1) tensor::commit(atom::smem_u32(&s.done[buf]));
                }
                __syncwarp();
            }
        }
    } else {
        // ---- write out; warp w reads lanes 32 (w % 4) on of the accumulator
        const int quarter = warp & 3;
        uint32_t acc = 0;
        for (int u = blockIdx.x; u < units; u += gridDim.x) {
            const Unit q = unit_at<MODE, BK>(p, s.table, u, splits, i_tiles);
            const int i = q.i0 + quarter * 32 + lane;
            const bool live = i < p.ni;
            const bool empty = q.kb0 == q.kb1;
            const uint32_t buf = acc & 1;
            bool good = true;
            if (!empty) {
                good = wait_warp(&s.done[buf], (acc >> 1) & 1);
                if (!good && splits == 1) break;   // with splits: on to the barriers below
                ++acc;
                tensor::fence_after_sync();
            }
            const size_t row = MODE == kGroupedGrad ? (size_t)q.g * p.n + q.j0
                                                    : (size_t)q.row0 + q.j0;
            __nv_bfloat16 *out = p.out + row * p.ldy + i;
            float ws = 1.f;
            if constexpr (!BF16) ws = live ? p.w_scales[(size_t)q.g * p.n + i] : 0.f;
            float *mine = p.partial + (size_t)u * kTileJ * kTileI + quarter * 32 + lane;
            auto put = [&](int j, float v, float xs) {
                if constexpr (!BF16) v = v * xs * ws;
                out[(size_t)j * p.ldy] = __float2bfloat16_rn(v);
            };
            for (int c = 0; c < q.nj && good; c += 32) {
                uint32_t v[32];
                __syncwarp();
                if (!empty) {
                    tensor::tmem_load32(tmem + buf * kTileJ + c + ((uint32_t)quarter << 21), v);
                    tensor::tmem_wait_loads();
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) v[x] = 0;
                }
                const int width = min(32, q.nj - c);
                if (splits == 1) {
                    float xs = 0.f;
                    if constexpr (!BF16)
                        if (lane < width) xs = p.x_scales[row + c + lane];
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        const float sx = BF16 ? 1.f : __shfl_sync(0xffffffffu, xs, x);
                        if (x < width && live) put(c + x, __uint_as_float(v[x]), sx);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (x < width) __stcg(mine + (size_t)(c + x) * kTileI, __uint_as_float(v[x]));
                }
            }
            if (!empty) {
                tensor::fence_before_sync();
                __syncwarp();
                if (lane == 0) atom::mbar_arrive(&s.free[buf]);
            }
            if (splits > 1) {
                // the last of the tile's CTAs adds the accumulators in split order
                __threadfence();
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (warp == 2 && lane == 0) {
                    const unsigned before = atomicAdd(&p.arrived[q.tile], 1u);
                    s.last = before + 1 == (unsigned)splits;
                    if (s.last) p.arrived[q.tile] = 0;
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (s.last && live && good) {
                    __threadfence();
                    const float *all = p.partial + (size_t)q.tile * splits * kTileJ * kTileI +
                                       quarter * 32 + lane;
                    for (int j = 0; j < q.nj; ++j) {
                        float v = 0.f;
                        for (int k = 0; k < splits; ++k)
                            v += __ldcg(all + ((size_t)k * kTileJ + j) * kTileI);
                        put(j, v, BF16 ? 1.f : p.x_scales[row + j]);
                    }
                }
            }
        }
    }
    tensor::fence_before_sync();
    __syncthreads();
    tensor::fence_after_sync();
    if (s.ctl.abort) {
        // a wait expired: let the copies and products in flight end before the exit
        if (warp == 0 && lane == 0)
            for (uint32_t o = filled > kStages ? filled - kStages : 0; o < filled; ++o)
                snac::ring_wait(&s.full[o % kStages], (o / kStages) & 1, &s.ctl, p.err,
                                snac::kSiteGroupedWait, false);
        if (warp == 1) {
            if (lane == 0) tensor::commit(atom::smem_u32(&s.drain));
            snac::ring_wait(&s.drain, 0, &s.ctl, p.err, snac::kSiteGroupedWait, false);
        }
        __syncthreads();
    }
    if (warp == 1) tensor::tmem_free(tmem, 512);
}

// ------------------------------------------------------------------- host --

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// A tensor of rank 2 or 3 with rows `ld` elements apart, read in boxes of
// box0 x box1 elements in 128-byte swizzled rows; reads outside it give zeros.
bool make_map(CUtensorMap *m, const void *p, int dtype, int rank, size_t d0, size_t d1, size_t d2,
              size_t ld, uint32_t box0, uint32_t box1) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const size_t es = dtype == PURLIN_BF16 ? 2 : 1;
    const cuuint64_t dims[3] = {d0, d1, d2};
    const cuuint64_t strides[2] = {ld * es, d1 * ld * es};
    const cuuint32_t box[3] = {box0, box1, 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return f(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
             (cuuint32_t)rank, const_cast<void *>(p), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, bool BF16>
cudaError_t launch_tc(const GroupedArgs &a, TcParams &p) {
    static const cudaError_t ready = cudaFuncSetAttribute(
        grouped_tc_kernel<MODE, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (ready != cudaSuccess) return ready;
    grouped_tc_kernel<MODE, BF16><<<a.sms, kThreads, kSmem, a.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t grouped_workspace(int sms) { return (size_t)sms * kTileI * kTileJ * sizeof(float); }

cudaError_t launch_grouped(const GroupedArgs &a) {
    TcParams p;
    const size_t bk = a.dtype == PURLIN_BF16 ? 64 : 128;
    bool ok;
    if (a.mode == kGroupedNK)
        ok = make_map(&p.a, a.w, a.dtype, 3, a.k, a.n, (size_t)a.groups, a.ldw, (uint32_t)bk, kTileI) &&
             make_map(&p.b, a.x, a.dtype, 2, a.k, a.rows, 1, a.ldx, (uint32_t)bk, kBoxJ);
    else if (a.mode == kGroupedKN)
        ok = make_map(&p.a, a.w, a.dtype, 3, a.n, a.k, (size_t)a.groups, a.ldw, 64, 64) &&
             make_map(&p.b, a.x, a.dtype, 2, a.k, a.rows, 1, a.ldx, 64, kBoxJ);
    else
        ok = make_map(&p.a, a.x, a.dtype, 2, a.k, a.rows, 1, a.ldx, 64, 64) &&
             make_map(&p.b, a.w, a.dtype, 2, a.n, a.rows, 1, a.ldw, 64, 64);
    if (!ok) return cudaErrorInvalidValue;
    p.out = static_cast<__nv_bfloat16 *>(a.y);
    p.x_scales = a.x_scales;
    p.w_scales = a.w_scales;
    p.begin = a.begin;
    p.count = a.count;
    p.partial = a.partial;
    p.arrived = a.arrived;
    p.ldy = a.ldy;
    p.rows = (long long)a.rows;
    p.groups = a.groups;
    p.ni = (int)(a.mode == kGroupedGrad ? a.k : a.n);
    p.n = (int)a.n;
    p.k = (int)a.k;
    p.err = a.err;
    if (a.dtype == PURLIN_E4M3) return launch_tc<kGroupedNK, false>(a, p);
    if (a.mode == kGroupedNK) return launch_tc<kGroupedNK, true>(a, p);
    if (a.mode == kGroupedKN) return launch_tc<kGroupedKN, true>(a, p);
    return launch_tc<kGroupedGrad, true>(a, p);
}

}  // namespace purlin
