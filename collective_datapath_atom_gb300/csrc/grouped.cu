// grouped.cu -- matrix products grouped by expert with ragged row counts.
//
// out[j][i] = sum over k of A[i][k] B[j][k] for every group; layers.h names
// what A, B, i, j and k are in each mode.  Groups are (first row, row count)
// pairs in device memory, so the tiles of a launch are found on the device.
//
// Persistent CTAs, one an SM, alone or in pairs that share a tile.  A tile is
// 128 i (256 for a pair) by up to 256 j: the weights' channels take the tensor
// core's 128-lane side and the group's rows the other, whose width is a field of
// the instruction, so a group of 5 rows costs a 16-column product, not a padded
// one, and the same code serves one token and a prefill.  A warp brings
// 128-byte-wide boxes of both operands into a ring of shared-memory stages (TMA,
// 128-byte swizzle), a warp issues tcgen05.mma from them into one of two
// accumulators in tensor memory, and eight warps write the other accumulator out
// meanwhile.
//
// Tiles go round the CTAs; fewer tiles than CTAs (decode) are cut into equal runs
// of K blocks instead, one a CTA.  A run's partial tiles go to a workspace in
// binary32, and the last of a tile's CTAs to arrive adds them in K order, so the
// result does not depend on which came last.
//
// kGroupedGrad sums over a group's rows: both operands then lie along M or N in
// memory (MN-major), and the last block of rows is cut at the group's end by
// clearing its rows in shared memory, since rows of no group may hold anything.
//
// Sums are binary32 in tensor memory, rounded once to bf16 on the way out.
//
// Bound by the tensor cores at prefill sizes: 16384 x 7168 x 2048 bf16 in one
// group takes 246 us in a short burst and 278 in long runs at the card's power limit
// (1.73 PFLOP/s; one cuBLAS product 288 there), over 8 Zipf groups 282 and 316, the
// tensor pipe 80% active; e4m3 at twice the channels 275 and 317 (3.5 and 3.0
// PFLOP/s); data gradient 260, weight gradient 297 us alone.  Bound by the weights'
// bytes at decode sizes: 8 rows on 5 of 8 experts, 147 MB, 31 us; 128 rows on 64
// experts, e4m3, 269 MB, 47 us (5.7 TB/s), of which about 5 us are the launch, the
// plan, the first load's latency and the join.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "layers.h"
#include "snac.cuh"
#include "tensor.cuh"

namespace purlin {
namespace {

constexpr int kTileI = 128, kTileJ = 256;
constexpr int kRowBytes = 128;                    // a stage's extent along a swizzled row
constexpr int kABytes = kTileI * kRowBytes;       // 16 KiB a stage
constexpr int kBoxJ = 32;                         // rows of a K-major box of B
constexpr int kBoxBytes = 64 * kRowBytes;         // MN-major box: 64 elements by 64 k
constexpr int kWriters = 8;                       // warps that write accumulators out
constexpr int kCutter = 2 + kWriters;             // the warp that cuts stages (kGroupedGrad)
constexpr int threads_of(int mode) { return 32 * (kCutter + (mode == kGroupedGrad ? 1 : 0)); }
constexpr int kSlotFloats = kTileI * kTileJ;      // one partial accumulator
constexpr int kWidths = 8;                        // row-tile widths to choose from: 32, 64, ... 256

constexpr uint32_t kRingBytes = 192 * 1024, kSmem = kRingBytes + 1024;
constexpr int kMaxStages = 9;

// Bytes of a stage: A's and the CTA's share of B.  A narrow tile leaves room for
// more stages, which a stream of weights needs.
template <bool B_MN, int CG>
__device__ __forceinline__ uint32_t stage_bytes(int width) {
    const int mine = width / CG;
    return kABytes + (B_MN ? (mine + 63) / 64 * kBoxBytes
                           : (mine + kBoxJ - 1) / kBoxJ * kBoxJ * kRowBytes);
}

struct TcParams {
    CUtensorMap a, b;
    __nv_bfloat16 *out;
    const float *x_scales, *w_scales;
    const int64_t *begin, *count;
    float *partial;       // two accumulators a CTA
    unsigned *arrived;    // a counter a tile, CTA and writer, zero between launches
    size_t ldy;
    long long rows;
    int groups, ni, n, k;
    int wide;             // rows of out start on 16-byte boundaries
    unsigned long long *err;
};

// The launch's tiles, found from the groups by every CTA.
struct Plan {
    int tiles[kMaxGroups + 1];           // tiles before group g
    long long cost[kMaxGroups + 1];      // cost of those tiles (block_cost)
    int begin[kMaxGroups];
    int count[kMaxGroups];
    int width;                           // of a row tile
    int whole;                           // tiles that go round whole: all or none
    int runs;                            // CTAs that share all of them instead
    long long left;                      // cost of those
    int bad;
};

// a / b of two that are not negative; 64-bit division is several times dearer, and
// a decode step's numbers are small.
__device__ __forceinline__ long long divide(long long a, long long b) {
    return (unsigned long long)(a | b) >> 32 == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The group whose entry of a running total includes `at` (groups that add
// nothing are skipped).
template <typename T>
__device__ __forceinline__ int group_of(const T *before, int groups, T at) {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (before[mid + 1] > at) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// Cost of a K block of a tile with nj columns: its loads, in KiB (A's 16 and an
// eighth a column).
constexpr int kMostCost = 16 + kTileJ / 8;
__device__ __forceinline__ int block_cost(int nj) { return 16 + (nj + 7) / 8; }

// The same in clocks of an SM: the products, or the fill of shared memory (about
// 65 bytes a clock).
template <int CG>
__device__ __forceinline__ float block_clocks(int width) {
    return fmaxf(2.f * width, (kABytes + (float)(width * kRowBytes / CG)) / 65.f);
}

// A run's join costs about this many K blocks of time.
constexpr int kJoinBlocks = 12;

// One group's tiles: `full` row tiles of the plan's width, then maybe a narrower
// one, each of them i_tiles tiles.
template <int MODE, int BK>
struct GroupTiles {
    int i_tiles, width, rest, blocks;
    int full;                          // tiles of the whole width
    long long full_cost, rest_cost;    // of one tile
    __device__ GroupTiles(const TcParams &p, int count, int width, int i_tiles)
        : i_tiles(i_tiles), width(width) {
        const int nj = MODE == kGroupedGrad ? p.n : count;
        blocks = max(1, ((MODE == kGroupedGrad ? count : p.k) + BK - 1) / BK);   // empty sums too
        const int down = nj / width;
        rest = nj - down * width;
        full = down * i_tiles;
        full_cost = (long long)blocks * block_cost(width);
        rest_cost = (long long)blocks * block_cost(rest);
    }
    __device__ int tiles() const { return full + (rest > 0 ? i_tiles : 0); }
    __device__ long long cost() const { return before(tiles()); }
    __device__ long long before(int local) const {
        return min(local, full) * full_cost + max(0, local - full) * rest_cost;
    }
    __device__ int tile_at(long long cost) const {
        return cost < full * full_cost ? (int)divide(cost, full_cost)
                                       : full + (int)divide(cost - full * full_cost, rest_cost);
    }
    __device__ int unit(int local) const { return block_cost(local < full ? width : rest); }
};

// Whether group (b, c) lies in the rows.
__device__ __forceinline__ bool group_bad(long long b, long long c, long long rows) {
    return c < 0 || b < 0 || c > rows || b > rows - c;   // c > rows first: b + c does not overflow
}

// Warp 0: check the groups and lay out the tiles.  More than 32 groups are in the
// plan already (`bad`: one of them lies outside the rows).  Groups that hold more
// rows than there are overlap, and are refused too; a plan of bad groups has no
// tiles.  This stands before the first load of every CTA, so it is one warp's
// work with one block barrier behind it, and sums by redux: by the block, with
// shared atomics, it took several times as long.
template <int MODE, int BK, int CG>
__device__ void lay_out(Plan &t, const TcParams &p, int i_tiles, int ctas, bool bad) {
    const int lane = threadIdx.x;
    if (p.groups <= 32 && lane < p.groups) {
        const long long b = p.begin[lane], c = p.count[lane];
        bad = group_bad(b, c, p.rows);
        t.begin[lane] = (int)b;
        t.count[lane] = (int)c;
    }
    bad = __any_sync(0xffffffffu, bad);
    long long held = 0;
    int most = 0;
    int down[kWidths] = {};   // row tiles at each width
    if (!bad) {
        unsigned low = 0, high = 0;
        for (int g = lane; g < p.groups; g += 32) {
            const int c = t.count[g];
            low += (unsigned)c & 0xFFFFu;
            high += (unsigned)c >> 16;
            most = max(most, c);
            if constexpr (MODE != kGroupedGrad) {
#pragma unroll
                for (int w = 0; w < kWidths; ++w) down[w] += (c + 32 * w + 31) / (32 * w + 32);
            }
        }
        held = ((long long)__reduce_add_sync(0xffffffffu, high) << 16) +
               __reduce_add_sync(0xffffffffu, low);
        most = __reduce_max_sync(0xffffffffu, most);
        bad = held > p.rows;
    }
    if (bad) {
        if (lane == 0) {
            t.bad = 1;
            t.width = 32;
            t.whole = 0;
            t.left = 0;
            t.runs = 1;
        }
        return;
    }
    // the width that costs least, the wider of two that cost about the same; groups
    // of a few rows leave no choice
    int width = 32;
    if (MODE == kGroupedGrad || most > 32) {
        int mine = 0;
#pragma unroll
        for (int w = 0; w < kWidths; ++w) {
            const int v = MODE == kGroupedGrad ? (p.n + 32 * w + 31) / (32 * w + 32) * p.groups
                                               : __reduce_add_sync(0xffffffffu, down[w]);
            if (lane == w) mine = v;
        }
        unsigned key = 0xFFFFFFFFu;
        if (lane < kWidths) {
            const int w = 32 * lane + 32;
            const float tiles = (float)mine * i_tiles;
            const float blocks = MODE == kGroupedGrad
                                     ? fmaxf(1.f, (float)held / (BK * (float)p.groups))
                                     : (float)((p.k + BK - 1) / BK);
            const float even = tiles / ctas, waves = ceilf(even);
            const float cost = (even >= 1.f ? waves * blocks : fminf(blocks, even * blocks + kJoinBlocks)) *
                                   block_clocks<CG>(w) + 12.f * w;
            key = (__float_as_uint(cost) & ~7u) | (unsigned)(kWidths - 1 - lane);
        }
        width = 32 * (kWidths - (int)(__reduce_min_sync(0xffffffffu, key) & 7u));
    }
    int tiles = 0;
    long long spent = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
        const int g = g0 + lane;
        const GroupTiles<MODE, BK> of(p, g < p.groups ? t.count[g] : 0, width, i_tiles);
        int v = g < p.groups ? of.tiles() : 0;
        long long k = g < p.groups ? of.cost() : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            const long long q = __shfl_up_sync(0xffffffffu, k, o);
            if (lane >= o) {
                v += u;
                k += q;
            }
        }
        if (g < p.groups) {
            t.tiles[g + 1] = tiles + v;
            t.cost[g + 1] = spent + k;
        }
        tiles += __shfl_sync(0xffffffffu, v, 31);
        spent += __shfl_sync(0xffffffffu, k, 31);
    }
    if (lane != 0) return;
    t.bad = 0;
    t.tiles[0] = 0;
    t.cost[0] = 0;
    t.width = width;
    // Fewer tiles than CTAs: runs of K blocks, where the time that idle CTAs would
    // waste is more than a join's.  (More tiles go round whole: CTAs in step share
    // what they read of the weights; with the last wave cut into runs they
    // read them twice, and products of a few waves took half as long again.)
    const long long idle = ctas - tiles;
    const bool cut = tiles > 0 && idle > 0 &&
                     idle * spent >= (long long)kJoinBlocks * ctas * block_cost(width) * tiles;
    t.whole = cut ? 0 : tiles;
    t.left = cut ? spent : 0;
    // at least four of the dearest blocks a run: a block begins in each
    t.runs = (int)max(1ll, min((long long)ctas, t.left / (4 * kMostCost)));
}

struct TcShared {
    Plan plan;
    snac::Ctl ctl;
    uint64_t full[kMaxStages];    // stage loaded; the leader's counts both CTAs' loads
    uint64_t empty[kMaxStages];   // stage consumed
    // kGroupedGrad, in place of full where a stage is to be cut at the group's end:
    uint64_t whole[kMaxStages];   // loaded in this CTA
    uint64_t cut[kMaxStages];     // cut in both (leader)
    uint64_t done[2], free[2];    // accumulator complete; accumulator read
    uint64_t drain;
    uint32_t tmem;
    alignas(16) __nv_bfloat16 turn[kWriters][16 * 32];   // 16 rows of 32 channels a warp
    float row_scales[2][kTileJ];                         // of the tile at hand, and the next
};

// What a CTA (or pair) does next: K blocks [kb0, kb1) of a tile.
struct Unit {
    int g, i0, j0, nj;   // nj: valid columns, up to the width
    int row0;            // first row of the group
    int nk;              // K extent
    int kb0, kb1;        // kb0 == kb1: the sum over nothing
    int tile;
    int c0, c1;          // the tile's runs, first and last; equal where nobody shares it
    int head;            // the first run's slot for the tile; the others begin in it: 2 run
};

// The runs split the cost evenly; a block belongs to the run it begins in.
__device__ __forceinline__ long long run_begin(const Plan &t, int c) { return divide(t.left * c, t.runs); }

__device__ __forceinline__ int run_of(const Plan &t, long long at) {
    return (int)divide((at + 1) * t.runs - 1, t.left);
}

// Walks the units of one CTA (or pair) `c` of `ctas`.
template <int MODE, int BK, int CG>
struct Walk {
    const TcParams &p;
    const Plan &t;
    int i_tiles, c, ctas;
    int tile;             // next whole tile
    long long at, end;    // the run's share of the cost still to do
    __device__ Walk(const TcParams &p, const Plan &t, int i_tiles, int c, int ctas)
        : p(p), t(t), i_tiles(i_tiles), c(c), ctas(ctas), tile(c) {
        at = end = 0;
        if (t.left > 0 && c < t.runs) {
            at = run_begin(t, c);
            end = run_begin(t, c + 1);
        }
    }
    __device__ bool next(Unit &q) {
        if (tile < t.whole) {
            q.tile = tile;
            tile += ctas;
            q.g = group_of(t.tiles, p.groups, q.tile);
            place(q);
            q.kb0 = 0;
            q.kb1 = (q.nk + BK - 1) / BK;
            q.c0 = q.c1 = c;
            return true;
        }
        while (at < end) {
            q.g = group_of(t.cost, p.groups, at);
            const GroupTiles<MODE, BK> of(p, t.count[q.g], t.width, i_tiles);
            const int local = of.tile_at(at - t.cost[q.g]), unit = of.unit(local);
            q.tile = t.tiles[q.g] + local;
            const long long begin = t.cost[q.g] + of.before(local);
            q.kb0 = (int)divide(at - begin + unit - 1, unit);
            q.kb1 = (int)min((long long)of.blocks, divide(end - begin + unit - 1, unit));
            at = begin + (long long)of.blocks * unit;
            if (q.kb0 >= q.kb1) continue;   // the run begins inside the tile's last block
            q.c0 = run_of(t, begin);
            q.c1 = run_of(t, begin + (long long)(of.blocks - 1) * unit);
            q.head = 2 * q.c0 + (run_begin(t, q.c0) < begin ? 1 : 0);
            place(q);
            if (q.nk == 0) q.kb1 = q.kb0;
            return true;
        }
        return false;
    }
    __device__ void place(Unit &q) const {
        const int local = q.tile - t.tiles[q.g];
        const int jt = local / i_tiles;
        q.i0 = (local - jt * i_tiles) * (kTileI * CG);
        q.j0 = jt * t.width;
        q.row0 = t.begin[q.g];
        q.nj = min(t.width, (MODE == kGroupedGrad ? p.n : t.count[q.g]) - q.j0);
        q.nk = MODE == kGroupedGrad ? t.count[q.g] : p.k;
    }
};

// Columns of the instruction for nj valid ones: what its shape allows.
template <int CG>
__device__ __forceinline__ int columns_of(int nj) {
    return (nj + 16 * CG - 1) / (16 * CG) * (16 * CG);
}

// Wait for a barrier's phase, two seconds at most; `abortable`: give up as soon
// as another role of the CTA has.
__device__ bool bounded_wait(uint64_t *bar, uint32_t parity, volatile snac::Ctl *ctl,
                             unsigned long long *err, bool abortable) {
    uint64_t t0 = 0;   // the timer is slow to read: not before some 60 tries
    for (uint32_t it = 1;; ++it) {
        if (atom::mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (abortable && ctl->abort) return false;
            const uint64_t now = atom::globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > snac::kRingWaitNs) {
                snac::record_error(err, PURLIN_ERR_TIMEOUT, snac::kSiteGroupedWait, blockIdx.x);
                ctl->abort = 1;
                return false;
            }
        }
    }
}

template <int MODE, bool BF16, int CG>
__global__ void __launch_bounds__(threads_of(MODE), 1)
grouped_tc_kernel(const __grid_constant__ TcParams p) {
    constexpr int BK = BF16 ? 64 : 128;        // K elements a stage
    constexpr int KSTEP = BF16 ? 16 : 32;      // K elements an instruction
    constexpr bool A_MN = MODE != kGroupedNK, B_MN = MODE == kGroupedGrad;
    extern __shared__ unsigned char raw[];
    __shared__ TcShared s;
    const uint32_t stage0 = (atom::smem_u32(raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = CG == 1 ? 0 : (int)(blockIdx.x & 1);   // in the pair; 0 leads
    const int group = blockIdx.x / CG, groups = gridDim.x / CG;

    if (warp == 0 && lane == 0) {
        tensor::prefetch_map(&p.a);
        tensor::prefetch_map(&p.b);
        for (int i = 0; i < kMaxStages; ++i) {
            atom::mbar_init(&s.full[i], 1);
            atom::mbar_init(&s.empty[i], 1);
            atom::mbar_init(&s.whole[i], 1);
            atom::mbar_init(&s.cut[i], CG);
        }
        for (int i = 0; i < 2; ++i) {
            atom::mbar_init(&s.done[i], 1);
            atom::mbar_init(&s.free[i], kWriters * CG);
        }
        atom::mbar_init(&s.drain, 1);
        atom::mbar_init_fence();
        s.ctl.abort = 0;
    }
    const int i_tiles = (p.ni + kTileI * CG - 1) / (kTileI * CG);
    // Everything before this overlaps the end of the kernel before; nothing of its
    // memory is touched until it is done.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    Plan &plan = s.plan;
    // (not before the wait: the kernel before may still be taking tensor memory)
    if (warp == 1) tensor::tmem_alloc<CG>(&s.tmem, 512);
    bool bad = false;
    if (p.groups > 32) {
        for (int g = threadIdx.x; g < p.groups; g += blockDim.x) {
            const long long b = p.begin[g], c = p.count[g];
            bad |= group_bad(b, c, p.rows);
            plan.begin[g] = (int)b;
            plan.count[g] = (int)c;
        }
        bad = __syncthreads_or(bad);
    }
    if (warp == 0) lay_out<MODE, BK, CG>(plan, p, i_tiles, groups, bad);
    tensor::fence_before_sync();
    tensor::sync_ctas<CG>();
    tensor::fence_after_sync();
    if (plan.bad && blockIdx.x == 0 && threadIdx.x == 0)
        snac::record_error(p.err, PURLIN_ERR_INVALID_ARG, snac::kSiteGroups, 0);
    const uint32_t tmem = s.tmem;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return bounded_wait(bar, parity, &s.ctl, p.err, true);
    };
    // one answer for the warp, whichever lanes saw the wait expire
    auto wait_warp = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    Unit q;
    const uint32_t stage_size = stage_bytes<B_MN, CG>(plan.width);
    const uint32_t stages = min((uint32_t)kMaxStages, kRingBytes / stage_size);
    uint32_t st = 0, parity = 0;   // the next stage, and its ring's turn
    auto advance = [&] {
        if (++st == stages) {
            st = 0;
            parity ^= 1;
        }
    };
    // Phases of each stage's full (or whole and cut), one bit each: a stage's turn
    // uses the one or the others.  For the loading thread, those it counted on.
    uint32_t fulls = 0, cuts = 0, full_used = 0, cut_used = 0;
    // whether a K block of the weight gradient ends inside an instruction's rows
    auto cut_at = [&](int kb) {
        return MODE == kGroupedGrad && min(BK, q.nk - kb * BK) % KSTEP != 0;
    };
    Walk<MODE, BK, CG> walk(p, plan, i_tiles, group, groups);

    if (warp < 2) {
        // One thread loads, one multiplies: nothing but them on a stage's path.
        if (!tensor::elect()) {
        } else if (warp == 0) {
            // ---- load
            bool run = true;
            while (run && walk.next(q)) {
                const int half = columns_of<CG>(q.nj) / CG;
                const int mine = CG == 1 ? q.nj : half;   // columns of this CTA's share
                const int boxes = B_MN ? (mine + 63) / 64 : (mine + kBoxJ - 1) / kBoxJ;
                const uint32_t bytes = kABytes + boxes * (B_MN ? kBoxBytes : kBoxJ * kRowBytes);
                const int i0 = q.i0 + rank * kTileI, j0 = q.j0 + rank * half;
                for (int kb = q.kb0; kb < q.kb1; ++kb, advance()) {
                    if (!wait(&s.empty[st], parity ^ 1)) {
                        run = false;
                        break;
                    }
                    // the leader's barrier counts both CTAs' bytes
                    uint32_t bar = atom::smem_u32(&s.full[st]);
                    if (cut_at(kb)) {
                        bar = atom::smem_u32(&s.whole[st]);
                        atom::mbar_arrive_expect_tx(&s.whole[st], bytes);
                        cuts ^= 1u << st;
                        cut_used |= 1u << st;
                    } else if (rank == 0) {
                        atom::mbar_arrive_expect_tx(&s.full[st], CG * bytes);
                        fulls ^= 1u << st;
                        full_used |= 1u << st;
                    } else {
                        bar = tensor::in_cta(bar, 0);
                    }
                    const uint32_t a = stage0 + st * stage_size, b = a + kABytes;
                    if constexpr (MODE == kGroupedNK) {
                        tensor::load_box_3d<CG>(a, &p.a, kb * BK, i0, q.g, bar);
                    } else if constexpr (MODE == kGroupedKN) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            tensor::load_box_3d<CG>(a + h * kBoxBytes, &p.a, i0 + 64 * h, kb * BK,
                                                    q.g, bar);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            tensor::load_box_2d<CG>(a + h * kBoxBytes, &p.a, i0 + 64 * h,
                                                    q.row0 + kb * BK, bar);
                    }
                    for (int h = 0; h < boxes; ++h) {
                        if constexpr (B_MN)
                            tensor::load_box_2d<CG>(b + h * kBoxBytes, &p.b, j0 + 64 * h,
                                                    q.row0 + kb * BK, bar);
                        else
                            tensor::load_box_2d<CG>(b + h * kBoxJ * kRowBytes, &p.b, kb * BK,
                                                    q.row0 + j0 + kBoxJ * h, bar);
                    }
                }
            }
        } else {
            // ---- multiply: the pair's leader
            uint32_t acc = 0;
            bool run = rank == 0;
            while (run && walk.next(q)) {
                if (q.kb0 == q.kb1) continue;   // a sum over nothing
                const uint32_t buf = acc & 1;
                if (!wait(&s.free[buf], ((acc >> 1) & 1) ^ 1)) break;
                tensor::fence_after_sync();
                ++acc;
                const uint32_t d = tmem + buf * kTileJ;
                const uint32_t idesc = tensor::instr_desc(BF16 ? 1 : 0, A_MN, B_MN, kTileI * CG,
                                                          columns_of<CG>(q.nj));
                for (int kb = q.kb0; kb < q.kb1; ++kb, advance()) {
                    const bool cut = cut_at(kb);
                    if (!wait(cut ? &s.cut[st] : &s.full[st], (cut ? cuts : fulls) >> st & 1)) {
                        run = false;
                        break;
                    }
                    if (cut) {
                        cuts ^= 1u << st;
                        // the other CTA's writes, which the products read there
                        if constexpr (CG == 2) asm volatile("fence.acq_rel.cluster;" ::: "memory");
                    } else {
                        fulls ^= 1u << st;
                    }
                    const uint32_t a = stage0 + st * stage_size, b = a + kABytes;
                    const int left = min(BK, q.nk - kb * BK);
                    const int steps = (left + KSTEP - 1) / KSTEP;
                    tensor::fence_after_sync();
                    const uint64_t da = tensor::operand_desc(a, kBoxBytes);
                    const uint64_t db = tensor::operand_desc(b, kBoxBytes);
                    // K-major: 32 bytes on along the row; MN-major: 16 rows on
                    constexpr uint64_t kNextA = (A_MN ? 16 * kRowBytes : 32) >> 4;
                    constexpr uint64_t kNextB = (B_MN ? 16 * kRowBytes : 32) >> 4;
#pragma unroll
                    for (int k = 0; k < BK / KSTEP; ++k)
                        if (k < steps)
                            tensor::mma<BF16, CG>(d, da + k * kNextA, db + k * kNextB, idesc,
                                                  kb > q.kb0 || k > 0);
                    tensor::commit<CG>(atom::smem_u32(&s.empty[st]));
                    if (kb + 1 == q.kb1) tensor::commit<CG>(atom::smem_u32(&s.done[buf]));
                }
            }
        }
    } else if (warp == kCutter) {
        // ---- cut: clear the rows past a group's end inside the last instruction's 16
        bool run = true;
        while (run && walk.next(q)) {
            const int boxes = 2 + (columns_of<CG>(q.nj) / CG + 63) / 64;
            for (int kb = q.kb0; kb < q.kb1; ++kb, advance()) {
                if (!cut_at(kb)) continue;
                if (!wait_warp(&s.whole[st], cuts >> st & 1)) {
                    run = false;
                    break;
                }
                cuts ^= 1u << st;
                const int left = q.nk - kb * BK, past = (left + KSTEP - 1) / KSTEP * KSTEP;
                const int quads = (past - left) * (kRowBytes / 16);
                const uint32_t from = stage0 + st * stage_size + left * kRowBytes;
                for (int box = 0; box < boxes; ++box)
                    for (int e = lane; e < quads; e += 32)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                         from + box * kBoxBytes + e * 16),
                                     "r"(0)
                                     : "memory");
                tensor::fence_async_shared();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 1) atom::mbar_arrive(&s.cut[st]);
                    else tensor::arrive_cluster(tensor::in_cta(atom::smem_u32(&s.cut[st]), 0), true);
                }
            }
        }
    } else {
        // ---- write out; warp w reads lanes 32 (w % 4) on of the accumulator, and
        // every other 16 columns of them
        const int quarter = warp & 3;
        constexpr int kColStep = 16 * kWriters / 4;
        const int c_first = 16 * ((warp - 2) >> 2);
        const uint32_t turn = atom::smem_u32(s.turn[warp - 2]);
        // 16-byte pieces of a row of `turn` (32 channels) lie at a place that depends
        // on the row: eight rows of one piece, and four pieces of a row, meet no bank twice
        auto piece = [&](int r, int k) { return turn + r * 64 + ((k ^ (r >> 1)) & 3) * 16; };
        uint32_t acc = 0, tile = 0;
        bool dead = false;   // a wait expired: walk on, for the writers' barriers and counters
        while (walk.next(q)) {
            const int i0 = q.i0 + rank * kTileI + quarter * 32;   // the warp's first channel
            const bool shared = q.c0 != q.c1;
            const bool empty = q.kb0 == q.kb1;
            const uint32_t buf = acc & 1;
            const size_t row = MODE == kGroupedGrad ? (size_t)q.g * p.n + q.j0
                                                    : (size_t)q.row0 + q.j0;
            __nv_bfloat16 *out = p.out + row * p.ldy + i0;
            // scales, fetched while the products go on
            const float *xs = s.row_scales[tile++ & 1];
            float ws[4];
            if constexpr (!BF16) {
                const int j = (int)threadIdx.x - 64;
                if (j < q.nj) s.row_scales[(tile - 1) & 1][j] = p.x_scales[row + j];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int i = i0 + 8 * m + (lane >> 2);
                    ws[m] = i < p.ni ? p.w_scales[(size_t)q.g * p.n + i] : 0.f;
                }
                asm volatile("bar.sync 1, %0;" ::"n"(32 * kWriters) : "memory");
            }
            if (!empty && !dead) {
                dead = !wait_warp(&s.done[buf], (acc >> 1) & 1);
                ++acc;
                tensor::fence_after_sync();
            }
            // 16 columns of the accumulator from column c on, as fragments: r[0..7] of
            // the warp's lanes 0..15, r[8..15] of the others
            auto fetch = [&](int c, uint32_t (&r)[16]) {
                __syncwarp();
                if (!empty) {
                    const uint32_t at = tmem + buf * kTileJ + c + ((uint32_t)quarter << 21);
                    tensor::tmem_load_fragments(at, r);
                    tensor::tmem_load_fragments(at + (16u << 16), r + 8);
                } else {
#pragma unroll
                    for (int x = 0; x < 16; ++x) r[x] = 0;
                }
            };
            // Rows of out are columns of the accumulator: they turn in shared memory by
            // stmatrix, and leave as 16-byte stores where out's rows allow it.
            auto put = [&](int c, const uint32_t (&r)[16]) {
                __syncwarp();   // the rows before have left
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2 sx = {1.f, 1.f};
                    if constexpr (!BF16)
                        sx = *reinterpret_cast<const float2 *>(xs + c + 8 * h + 2 * (lane & 3));
                    uint32_t m[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {   // channels 8 k on
                        const int at = 8 * (k >> 1) + 4 * h + 2 * (k & 1);
                        float a = __uint_as_float(r[at]), b = __uint_as_float(r[at + 1]);
                        if constexpr (!BF16) {
                            a = a * sx.x * ws[k];
                            b = b * sx.y * ws[k];
                        }
                        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
                        m[k] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    tensor::store_transposed(piece(8 * h + (lane & 7), lane >> 3), m[0], m[1], m[2],
                                             m[3]);
                }
                __syncwarp();
                if (p.wide) {
                    const int k = lane & 3, room = p.ni - i0 - 8 * k;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int rr = 8 * t + (lane >> 2);
                        if (c + rr >= q.nj || room <= 0) continue;
                        uint4 v;
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                     : "r"(piece(rr, k))
                                     : "memory");
                        __nv_bfloat16 *to = out + 8 * k + (size_t)(c + rr) * p.ldy;
                        if (room >= 8) {
                            *reinterpret_cast<uint4 *>(to) = v;
                        } else {
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 7; ++e)
                                if (e < room)
                                    reinterpret_cast<unsigned short *>(to)[e] =
                                        (unsigned short)(w[e / 2] >> 16 * (e % 2));
                        }
                    }
                } else {
                    unsigned short *to =
                        reinterpret_cast<unsigned short *>(out) + lane + (size_t)c * p.ldy;
                    const int rows = i0 + lane < p.ni ? q.nj - c : 0;
                    unsigned short v[16];
#pragma unroll
                    for (int rr = 0; rr < 16; ++rr)
                        asm volatile("ld.shared.u16 %0, [%1];"
                                     : "=h"(v[rr])
                                     : "r"(piece(rr, lane >> 3) + (lane & 7) * 2)
                                     : "memory");
#pragma unroll
                    for (int rr = 0; rr < 16; ++rr, to += p.ldy)
                        if (rr < rows) *to = v[rr];
                }
            };
            // Where run r's partial of the tile lies (a run has two slots: for the tile it
            // begins in, and for the one it ends in if that is another):
            // [16 columns][quarter of the fragments][lane of 128] of float4.
            auto slot_of = [&](int r, int c) {
                return reinterpret_cast<float4 *>(p.partial) +
                       ((size_t)(r == q.c0 ? q.head : 2 * r) * CG + rank) * (kSlotFloats / 4) +
                       (size_t)(c / 16) * 4 * kTileI + quarter * 32 + lane;
            };
            uint32_t r[16], ahead[16];
            if (shared) {
                for (int c = c_first; c < q.nj && !dead; c += kColStep) {
                    fetch(c, r);
                    tensor::tmem_wait_loads(r);
                    float4 *mine = slot_of(group, c);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (x % 2 == 0 || c + 8 < q.nj)
                            __stcg(mine + x * kTileI,
                                   make_float4(__uint_as_float(r[4 * x]), __uint_as_float(r[4 * x + 1]),
                                               __uint_as_float(r[4 * x + 2]),
                                               __uint_as_float(r[4 * x + 3])));
                }
                // Warp by warp: the tile's last CTA to get here adds the accumulators, in K
                // order.  Nothing but this warp's counterparts to wait for.
                __threadfence();
                __syncwarp();
                int last = 0;
                if (lane == 0) {
                    unsigned *n = p.arrived + ((size_t)q.tile * CG + rank) * kWriters + warp - 2;
                    last = atomicAdd(n, 1u) == (unsigned)(q.c1 - q.c0);
                    if (last) *n = 0;
                }
                last = __shfl_sync(0xffffffffu, last, 0);
                if (last) __threadfence();
                for (int c = c_first; c < q.nj && !dead && last; c += kColStep) {
                    float4 sum[4] = {};
                    for (int k = q.c0; k <= q.c1; k += 3) {
                        float4 u[3][4];   // three runs' loads in flight
#pragma unroll
                        for (int y = 0; y < 3; ++y)
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                u[y][x] = k + y <= q.c1 && (x % 2 == 0 || c + 8 < q.nj)
                                              ? __ldcg(slot_of(k + y, c) + x * kTileI)
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int y = 0; y < 3; ++y)
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                sum[x].x += u[y][x].x;
                                sum[x].y += u[y][x].y;
                                sum[x].z += u[y][x].z;
                                sum[x].w += u[y][x].w;
                            }
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        r[4 * x] = __float_as_uint(sum[x].x);
                        r[4 * x + 1] = __float_as_uint(sum[x].y);
                        r[4 * x + 2] = __float_as_uint(sum[x].z);
                        r[4 * x + 3] = __float_as_uint(sum[x].w);
                    }
                    put(c, r);
                }
            } else if (!dead) {
                tensor::walk_columns(
                    c_first, kColStep, q.nj, [&](int c) { fetch(c, ahead); },
                    [&] {
                        tensor::tmem_wait_loads(ahead);
#pragma unroll
                        for (int x = 0; x < 16; ++x) r[x] = ahead[x];
                    },
                    [&](int c) { put(c, r); });
            }
            if (!empty && !dead) {
                tensor::fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    const uint32_t bar = atom::smem_u32(&s.free[buf]);
                    if constexpr (CG == 1) atom::mbar_arrive(&s.free[buf]);
                    else tensor::arrive_cluster(tensor::in_cta(bar, 0), false);
                }
            }
        }
    }
    tensor::fence_before_sync();
    __syncwarp();
    tensor::sync_ctas<CG>();
    tensor::fence_after_sync();
    if (s.ctl.abort) {
        // a wait expired: let the copies and products in flight end before the exit
        // (a pair's copies count at the leader, whose own wait expires with them)
        if (warp == 0)
            for (uint32_t i = 0; i < stages; ++i) {
                if (full_used >> i & 1)
                    bounded_wait(&s.full[i], (fulls >> i & 1) ^ 1, &s.ctl, p.err, false);
                if (cut_used >> i & 1)
                    bounded_wait(&s.whole[i], (cuts >> i & 1) ^ 1, &s.ctl, p.err, false);
            }
        if (warp == 1 && rank == 0) {
            if (tensor::elect()) tensor::commit<CG>(atom::smem_u32(&s.drain));
            bounded_wait(&s.drain, 0, &s.ctl, p.err, false);
        }
        __syncwarp();
    }
    tensor::sync_ctas<CG>();
    if (warp == 1) tensor::tmem_free<CG>(tmem, 512);
}

// ------------------------------------------------------------------- host --

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<void *> found{nullptr};   // not found: asked for again
    void *p = found.load(std::memory_order_acquire);
    if (p == nullptr) {
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            return nullptr;
        found.store(p, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(p);
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

template <int MODE, bool BF16, int CG>
cudaError_t launch_tc(const GroupedArgs &a, const TcParams &p) {
    static SharedMemoryLimit limit;
    const cudaError_t ready = limit.raise(grouped_tc_kernel<MODE, BF16, CG>, (int)kSmem);
    if (ready != cudaSuccess) return ready;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(a.sms / CG * CG));
    c.blockDim = dim3(threads_of(MODE));
    c.dynamicSmemBytes = kSmem;
    c.stream = a.stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim = {CG, 1, 1};
    c.attrs = at;
    c.numAttrs = CG;
    return cudaLaunchKernelEx(&c, grouped_tc_kernel<MODE, BF16, CG>, p);
}

template <int MODE, bool BF16>
cudaError_t launch_mode(const GroupedArgs &a, const TcParams &p) {
    // A pair halves what each CTA loads of B, and its tiles are twice as wide: it
    // pays once there is work for it.  Single CTAs against pairs, us, of equal groups:
    // 1024 rows in one, 2048 x 2048, 12.6 and 13.6; 2048 rows in 8, 1024 x 2048, 14.6
    // and 15.2, 7168 x 2048 54.8 and 51.6; 16384 rows in 64, 2048 x 2048, 123 and 114;
    // 16384 rows in 8, 2048 x 7168, 321 and 290.  Channels that fill a wider tile badly
    // stay with single CTAs (384: a third of it empty).
    // The counts are on the device: `rows` is what the buffer holds, an upper bound.  In
    // buffers of full capacity with few rows in them pairs lose a little: 128 rows on 64
    // experts of 1024 places, e4m3 1024 x 4096, 47.7 and 48.5, bf16 1024 x 2048 47.5 and
    // 48.2; 256 rows on 8 of 2048, 2048 x 7168, 41.9 and 42.5 (2000 rows 68.4 and 65.3);
    // 20 rows on 8 of 1024, 1024 x 1024, 7.3 and 8.2.
    const double work = (double)a.rows * (double)a.n * (double)a.k;
    const size_t wide = ((size_t)p.ni + 255) / 256 * 2, narrow = ((size_t)p.ni + 127) / 128;
    const bool pair = work >= 8e9 && 8 * wide <= 9 * narrow && a.sms >= 2;
    return pair ? launch_tc<MODE, BF16, 2>(a, p) : launch_tc<MODE, BF16, 1>(a, p);
}

}  // namespace

size_t grouped_workspace(int sms) { return 2 * (size_t)sms * kSlotFloats * sizeof(float); }

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
    p.wide = ((reinterpret_cast<uintptr_t>(a.y) | (a.ldy * sizeof(__nv_bfloat16))) & 15u) == 0;
    p.err = a.err;
    if (a.dtype == PURLIN_E4M3) return launch_mode<kGroupedNK, false>(a, p);
    if (a.mode == kGroupedNK) return launch_mode<kGroupedNK, true>(a, p);
    if (a.mode == kGroupedKN) return launch_mode<kGroupedKN, true>(a, p);
    return launch_mode<kGroupedGrad, true>(a, p);
}

}  // namespace purlin
