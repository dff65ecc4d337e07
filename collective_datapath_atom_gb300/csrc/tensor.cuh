// tensor.cuh -- the 5th-generation tensor cores' instructions as inline PTX:
// tensor-memory allocation, tcgen05.mma with shared-memory operands, its
// commit, the loads of an accumulator, tiled TMA loads, and the descriptors
// they take.  sm_103a only.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "atom.cuh"

namespace purlin {
namespace tensor {

// One thread of a converged warp, always the same one.  Instructions that take
// their operands from uniform registers (TMA, tcgen05) are issued under it: under
// a test of the lane's number the compiler cannot tell that one thread is active,
// and the product of a K block took twice its time.
__device__ __forceinline__ bool elect() {
    uint32_t one = 0;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t@p mov.u32 %0, 1;\n\t}"
        : "+r"(one));
    return one != 0;
}

// ------------------------------------------------------------------- TMA --

__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// One box of a tensor into shared memory, completion counted on `bar`.  CG 2:
// `bar` may be the pair's other CTA's (an address of in_cta).
#define PURLIN_LOAD_BOX(DIM, GROUP, COORDS, ...)                                   \
    asm volatile("cp.async.bulk.tensor." DIM                                       \
                 ".shared::cluster.global.tile.mbarrier::complete_tx::bytes" GROUP \
                 " [%0], [%1, " COORDS "], [%2];" ::"r"(smem),                     \
                 "l"(m), "r"(bar), __VA_ARGS__                                     \
                 : "memory")

template <int CG>
__device__ __forceinline__ void load_box_2d(uint32_t smem, const CUtensorMap *m, int c0, int c1,
                                            uint32_t bar) {
    if constexpr (CG == 1) PURLIN_LOAD_BOX("2d", "", "{%3, %4}", "r"(c0), "r"(c1));
    else PURLIN_LOAD_BOX("2d", ".cta_group::2", "{%3, %4}", "r"(c0), "r"(c1));
}

template <int CG>
__device__ __forceinline__ void load_box_3d(uint32_t smem, const CUtensorMap *m, int c0, int c1,
                                            int c2, uint32_t bar) {
    if constexpr (CG == 1) PURLIN_LOAD_BOX("3d", "", "{%3, %4, %5}", "r"(c0), "r"(c1), "r"(c2));
    else PURLIN_LOAD_BOX("3d", ".cta_group::2", "{%3, %4, %5}", "r"(c0), "r"(c1), "r"(c2));
}
#undef PURLIN_LOAD_BOX

// Writes of this thread to shared memory become visible to the async proxy.
__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// -------------------------------------------------------------- CTA pairs --

// The address, in the cluster's window, of what lies at `smem` in CTA `rank`.
__device__ __forceinline__ uint32_t in_cta(uint32_t smem, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
    return a;
}

// Arrive on a barrier of either CTA (an address of in_cta).  `published`: this
// thread's warp wrote shared memory that the other CTA's products read.  Without
// such writes the order within the CTA is enough: what the barrier guards was
// written by TMA or read by tcgen05.ld, and a release at cluster scope on every
// stage costs more than the stage (measured: twice the time of the whole product).
__device__ __forceinline__ void arrive_cluster(uint32_t bar, bool published) {
    if (published)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                     : "memory");
    else
        asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Every thread of the CTA, or of both CTAs of a pair.
template <int CG>
__device__ __forceinline__ void sync_ctas() {
    if constexpr (CG == 1) {
        __syncthreads();
    } else {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}

// ---------------------------------------------------------- tensor memory --

// Whole warp (of each CTA of the pair).  The column base goes to shared memory.
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t columns) {
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         atom::smem_u32(dst)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         atom::smem_u32(dst)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base),
                     "r"(columns)
                     : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base),
                     "r"(columns)
                     : "memory");
}

__device__ __forceinline__ void fence_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void fence_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Sixteen columns of sixteen lanes, as the fragments of 8 x 8 matrices: of columns
// 8 h on, thread t gets in r[4 h], r[4 h + 1] lane t / 4 of columns 2 (t % 4) and the
// next, in r[4 h + 2], r[4 h + 3] lane t / 4 + 8 of the same.
__device__ __forceinline__ void tmem_load_fragments(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(addr)
        : "memory");
}

// Wait for this thread's loads; r is theirs, and not used before.
__device__ __forceinline__ void tmem_wait_loads(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// Columns first, first + step, ... below `end` of an accumulator: the loads of the
// next ones are on their way while those that `wait` handed over are put away.
// Every load issued is waited for: one that is not may land in registers that hold
// something else by then, or read an accumulator that is given up already.  A warp
// without columns (a tile of 16 rows leaves half of them none) issues no load.
template <typename Fetch, typename Wait, typename Put>
__device__ __forceinline__ void walk_columns(int first, int step, int end, Fetch fetch, Wait wait,
                                             Put put) {
    if (first >= end) return;
    fetch(first);
#pragma unroll 1
    for (int c = first; c < end; c += step) {
        wait();
        if (c + step < end) fetch(c + step);
        put(c);
    }
}

// Four 8 x 8 matrices of 16-bit fragments, transposed: thread 8 m + i gives the
// address of 16 bytes for column i of matrix m.
__device__ __forceinline__ void store_transposed(uint32_t smem, uint32_t a, uint32_t b, uint32_t c,
                                                 uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem),
                 "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// ------------------------------------------------------------ descriptors --

// Shared-memory operand in 128-byte swizzled rows, in eight-row atoms of 1024
// bytes.  K-major: a row is 128 bytes of K, `block` is not used.  MN-major: a
// row is 64 elements of M or N at one k; atoms follow each other along K, and
// `block` is the distance in bytes to the next 64 elements of M or N.
__device__ __forceinline__ uint64_t operand_desc(uint32_t smem, uint32_t block) {
    return (uint64_t)((smem & 0x3FFFF) >> 4) | (uint64_t)(block >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// Instruction descriptor: binary32 accumulator; `format` 1 = bf16 (kind f16),
// 0 = e4m3 (kind f8f6f4); a_mn, b_mn: the operand is MN-major.
__host__ __device__ constexpr uint32_t instr_desc(uint32_t format, bool a_mn, bool b_mn, uint32_t m,
                                                  uint32_t n) {
    return 1u << 4 | format << 7 | format << 10 | (a_mn ? 1u << 15 : 0u) |
           (b_mn ? 1u << 16 : 0u) | (n >> 3) << 17 | (m >> 4) << 24;
}

#define PURLIN_MMA(CG, KIND)                                                        \
    asm volatile(                                                                   \
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"                             \
        "tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d), \
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)                       \
        : "memory")

// D (+)= A B, one thread.  CG 2: the pair's leader, for both CTAs; A's rows and
// B's columns lie half in each CTA's shared memory, at the same addresses.
template <bool BF16, int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                    bool accumulate) {
    if constexpr (BF16 && CG == 1) PURLIN_MMA("1", "f16");
    if constexpr (BF16 && CG == 2) PURLIN_MMA("2", "f16");
    if constexpr (!BF16 && CG == 1) PURLIN_MMA("1", "f8f6f4");
    if constexpr (!BF16 && CG == 2) PURLIN_MMA("2", "f8f6f4");
}
#undef PURLIN_MMA

// Arrive on `bar` (of each CTA of the pair) when the products issued so far by
// this thread are done.
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"((uint16_t)3)
            : "memory");
}

}  // namespace tensor
}  // namespace purlin
