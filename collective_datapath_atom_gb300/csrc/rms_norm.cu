// rms_norm.cu -- root-mean-square norm with the residual's addition, output
// in the input's type or in e4m3 with one scale a row, and its backward pass.
//
// Forward, a row at a time, in binary32:
//   t = x + residual,  r = 1 / sqrt(mean(t^2) + eps),  y = t r w.
// One pass over memory: a row's t stays in the registers of the threads that
// loaded it (a block, or one warp for short rows), so x and the residual are
// read once and total and y written once; two block sums (t^2, then max |y|
// for e4m3) separate the load from the store.  Bound by bytes, so the loads
// must not stop while a block waits for its sums.  Where a block has many rows
// to do it is persistent, and bulk copies bring its next rows into a ring in
// shared memory meanwhile; short rows, a warp's each, and launches of a few rows
// load into registers, the next row ahead.
//
// Backward, with g = dy w:
//   dx = r (g - t r^2 mean(g t)) + dtotal,  dweight = sum over rows of dy t r.
// The same walk: a thread owns the same columns in every row, so its share of
// dweight is a register sum, written once a block and added up over the blocks
// in a fixed order by a second kernel: no atomics, the same bits every time.
//
// Rows that start on no 16-byte boundary (an odd hidden size) are read and
// written in 16-byte windows all the same: a window starts `phase` elements
// before the row, and only the row's first and last windows go element by
// element.  The grid is a multiple of the windows' elements, so all of a
// block's rows have one phase and a thread's columns stay the same.  Operands at
// different phases go element by element (16384 x 7168 bf16 331 us instead of 158,
// backward 494 instead of 119).
//
// Both are bound by bytes.  16384 x 7168 bf16 with a residual to e4m3: 124 us, 6.6
// TB/s (99% of a copy's rate); backward of 32768 x 4096 bf16: 171 us, 6.3 TB/s.  A
// single row of 4096 is a launch and one round trip to memory, 4.5 us on the device.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "layers.h"
#include "snac.cuh"

namespace purlin {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kF32Max = 3.40282347e38f;      // the largest finite value
constexpr float kScaleMin = 1.17549435e-38f;   // 2^-126, the smallest normal value

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __nv_fp8_e4m3 from_f32<__nv_fp8_e4m3>(float v) {
    return __nv_fp8_e4m3(v);   // round to nearest even, saturating; NaN stays NaN
}

// Two values as bits of O, the first in the low half: one instruction a pair
// (a value at a time, the conversions were a fifth of the kernel's instructions).
template <typename O>
__device__ __forceinline__ uint32_t pair_bits(float a, float b) {
    if constexpr (sizeof(O) == 2) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&p);
    } else {
        return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    }
}

// V elements as one aligned memory access.
template <typename O, int V>
__device__ __forceinline__ void store(O *p, const float (&in)[V]) {
    if constexpr (V == 1) {
        *p = from_f32<O>(in[0]);
    } else if constexpr (sizeof(O) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(in[0], in[1], in[2], in[3]);
    } else if constexpr (sizeof(O) == 2) {
        *reinterpret_cast<uint4 *>(p) =
            make_uint4(pair_bits<O>(in[0], in[1]), pair_bits<O>(in[2], in[3]),
                       pair_bits<O>(in[4], in[5]), pair_bits<O>(in[6], in[7]));
    } else {
        uint32_t w[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            w[i] = pair_bits<O>(in[4 * i], in[4 * i + 1]) |
                   pair_bits<O>(in[4 * i + 2], in[4 * i + 3]) << 16;
        if constexpr (V == 4) *reinterpret_cast<uint32_t *>(p) = w[0];
        else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
}

// v / d from the reciprocal of d (rounded to nearest): the product, and one step
// with its exact remainder (P. Markstein, IBM J. Res. Dev. 34, 1990).  The product
// alone can be off by an ulp either way, which moves ties.  16384 x 7168 to e4m3:
// a division an element 229 us, this 124 (the product alone 135: the reads run
// further ahead of the writes).
__device__ __forceinline__ float quotient(float v, float d, float inv) {
    const float q = v * inv;
    return fmaf(fmaf(-q, d, v), inv, q);
}

// The mean of n values from their sum, inv = 1 / n; an infinite sum stays one.
__device__ __forceinline__ float mean_of(float sum, float n, float inv) {
    return fabsf(sum) <= kF32Max ? quotient(sum, n, inv) : sum;
}

// A row's values v over its e4m3 scale.
template <int ITEMS, int V>
__device__ __forceinline__ void divide_row(float (&v)[ITEMS][V], float scale) {
    // tiny rows: remainders would fall below the smallest value; both by 2^64, exactly
    if (scale < 0x1p-80f) {
        scale *= 0x1p64f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] *= 0x1p64f;
    }
    const float inv = 1.f / scale;
    const float d = scale <= kF32Max ? scale : 0.f;   // infinite: the products, 0 or NaN, stand
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = quotient(v[i][j], d, inv);
}

struct Sum {
    __device__ static float f(float a, float b) { return a + b; }
};
struct Max {
    __device__ static float f(float a, float b) { return fmaxf(a, b); }
};

// Reduction over the threads of a row: one warp, or the block through
// `shared` (32 floats, not reused before another barrier).  Every thread gets
// the result; the order is fixed.
template <typename Op>
__device__ __forceinline__ float reduce_row(float v, bool warp_only, float *shared) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = Op::f(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (warp_only) return v;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = shared[0];
    for (int w = 1; w < warps; ++w) v = Op::f(v, shared[w]);
    return v;
}

// Elements between a window's start and the row's, for the row at `row`.
template <int V>
__device__ __forceinline__ int phase_of(uint32_t phase, size_t ld, size_t row) {
    return V == 1 ? 0 : (int)((phase + (uint32_t)(ld % V) * (uint32_t)(row % V)) % V);
}

// V elements as 32-bit words, two bf16 in one: as an array of 16-bit values the
// compiler gave each a register of its own.
template <typename T, int V>
struct Window {
    static constexpr int kWords = (V * (int)sizeof(T) + 3) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ float at(int j) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        else return __uint_as_float(j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
    }
    __device__ __forceinline__ void set(int j, uint32_t bits) {   // of a cleared word
        if constexpr (sizeof(T) == 4) w[j] = bits;
        else w[j / 2] |= j % 2 ? bits << 16 : bits;
    }
};

__device__ __forceinline__ uint32_t bits_of(const float *p) { return __float_as_uint(*p); }
__device__ __forceinline__ uint32_t bits_of(const __nv_bfloat16 *p) {
    return *reinterpret_cast<const unsigned short *>(p);
}

// Window `e` of a row: elements e .. e + V of those in [0, hidden), zero outside.
// Without EDGE a window is in the row or outside it, never across an end.
template <typename T, int V, bool EDGE>
__device__ __forceinline__ Window<T, V> read_window(const T *row, int e, int hidden) {
    Window<T, V> k;
#pragma unroll
    for (int j = 0; j < k.kWords; ++j) k.w[j] = 0;
    if ((!EDGE || e >= 0) && e + V <= hidden) {
        if constexpr (V == 1) {
            k.w[0] = bits_of(row + e);
        } else {
            const uint4 u = *reinterpret_cast<const uint4 *>(row + e);
            k.w[0] = u.x;
            k.w[1] = u.y;
            k.w[2] = u.z;
            k.w[3] = u.w;
        }
    } else if constexpr (EDGE) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e + j >= 0 && e + j < hidden) k.set(j, bits_of(row + e + j));
    }
    return k;
}

template <typename O, int V, bool EDGE>
__device__ __forceinline__ void write_window(O *row, int e, int hidden, const float (&in)[V]) {
    if ((!EDGE || e >= 0) && e + V <= hidden) {
        store<O, V>(row + e, in);
    } else if constexpr (EDGE) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (e + j >= 0 && e + j < hidden) row[e + j] = from_f32<O>(in[j]);
    }
}

// The weight has an alignment of its own, and is read once a block.
template <typename T, int V, bool EDGE>
__device__ __forceinline__ Window<T, V> read_weight(const T *w, int e, int hidden) {
    if (!EDGE || (reinterpret_cast<uintptr_t>(w + e) & (sizeof(T) * V - 1)) == 0)
        return read_window<T, V, EDGE>(w, e, hidden);
    Window<T, V> k;
#pragma unroll
    for (int j = 0; j < k.kWords; ++j) k.w[j] = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (e + j >= 0 && e + j < hidden) k.set(j, bits_of(w + e + j));
    return k;
}

// ------------------------------------------------------------ staged rows --

constexpr int kMaxStages = 4;

// Wait for a stage, two seconds at most.
__device__ __forceinline__ bool bounded_row_wait(uint64_t *bar, uint32_t parity,
                                                 unsigned long long *err) {
    uint64_t t0 = 0;   // the timer is slow to read: not before some 60 tries
    for (uint32_t it = 1; !atom::mbar_try_wait(bar, parity); ++it) {
        if ((it & 63u) != 0) continue;
        const uint64_t now = atom::globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > snac::kRingWaitNs) {
            snac::record_error(err, PURLIN_ERR_TIMEOUT, snac::kSiteRowWait, blockIdx.x);
            return false;
        }
    }
    return true;
}

// A block's rows on their way through shared memory: `arrays` operands of a row
// a stage, the windows that lie wholly in the row brought by bulk copies, each
// at its place.  One thread issues; a stage is refilled after a block barrier
// behind which every thread is through with it.
template <typename T, int V, int ARRAYS>
struct RowRing {
    struct Shared {
        uint64_t full[kMaxStages];
    };
    Shared &s;
    unsigned char *base;
    uint32_t array_bytes;
    int stages, arrays, first, count;   // whole windows of a row: from, how many
    size_t row0, step, rows;
    int phase;
    uint32_t issued = 0;          // thread 0: rows fetched
    int fill = 0;                 // thread 0: the stage for the next one
    int st = 0;                   // the stage of the row at hand
    uint32_t parity = 0;
    const unsigned char *at;      // its start
    bool dead = false;            // a wait expired: no more of them
    const T *src[ARRAYS];
    size_t ld[ARRAYS];

    __device__ RowRing(Shared &s, unsigned char *base, int stages, int arrays, int hidden, int phase,
                       size_t row0, size_t step, size_t rows)
        : s(s), base(base), stages(stages), arrays(arrays), row0(row0), step(step), rows(rows),
          phase(phase), at(base) {
        first = phase > 0 ? 1 : 0;
        count = max(0, (phase + hidden) / V - first);
        array_bytes = (uint32_t)((hidden + 2 * (V - 1)) / V) * 16;
    }
    // Thread 0, before a block barrier.
    __device__ void init() {
        for (int i = 0; i < stages; ++i) atom::mbar_init(&s.full[i], 1);
        atom::mbar_init_fence();
    }
    // Thread 0: fill the next stage, if a row is left for it.
    __device__ void issue() {
        const size_t row = row0 + (size_t)issued * step;
        if (row >= rows || dead) return;
        uint64_t *bar = &s.full[fill];
        unsigned char *to = base + (size_t)fill * arrays * array_bytes + first * 16;
        ++issued;
        fill = fill + 1 == stages ? 0 : fill + 1;
        atom::mbar_arrive_expect_tx(bar, (uint32_t)(count * 16 * arrays));
        if (count == 0) return;
        // no cache hint: rows that share a line with the next fetched it twice (evict-first)
#pragma unroll
        for (int a = 0; a < ARRAYS; ++a)
            if (a < arrays)
                atom::bulk_load(to + a * array_bytes, src[a] + row * ld[a] + first * V - phase,
                                (uint32_t)count * 16, bar);
    }
    // Every thread: the row at hand is in its stage.  Two seconds at most.
    __device__ void wait(unsigned long long *err) {
        if (!dead && !bounded_row_wait(&s.full[st], parity, err)) dead = true;
    }
    // Every thread: on to the next row.
    __device__ void next() {
        if (++st == stages) {
            st = 0;
            parity ^= 1;
        }
        at = base + (size_t)st * arrays * array_bytes;
    }
    // Window `w` of array a of the row at hand, which is row `row`.
    template <bool EDGE>
    __device__ __forceinline__ Window<T, V> read(size_t row, int a, int w, int hidden) const {
        if ((!EDGE || w >= first) && w < first + count) {
            const uint4 u = *reinterpret_cast<const uint4 *>(at + a * array_bytes + w * 16);
            Window<T, V> k;
            k.w[0] = u.x;
            k.w[1] = u.y;
            k.w[2] = u.z;
            k.w[3] = u.w;
            return k;
        }
        if constexpr (EDGE) return read_window<T, V, EDGE>(src[a] + row * ld[a], w * V - phase, hidden);
        Window<T, V> k;
#pragma unroll
        for (int j = 0; j < k.kWords; ++j) k.w[j] = 0;
        return k;
    }
    // Thread 0, at the end: copies that a wait gave up on land before the exit.
    __device__ void drain(unsigned long long *err) {
        if (!dead) return;
        for (uint32_t n = issued > (uint32_t)stages ? issued - stages : 0; n < issued; ++n)
            bounded_row_wait(&s.full[n % (uint32_t)stages], (n / (uint32_t)stages) & 1, err);
    }
};

// The weight's windows of a block, each thread its own.
template <typename T, int V>
struct WeightStage {
    unsigned char *base;
    __device__ uint4 *at(int i) const {
        return reinterpret_cast<uint4 *>(base) + (size_t)i * blockDim.x + threadIdx.x;
    }
    __device__ void put(int i, const Window<T, V> &k) const {
        *at(i) = make_uint4(k.w[0], k.w[1], k.w[2], k.w[3]);
    }
    __device__ Window<T, V> get(int i) const {
        const uint4 u = *at(i);
        Window<T, V> k;
        k.w[0] = u.x;
        k.w[1] = u.y;
        k.w[2] = u.z;
        k.w[3] = u.w;
        return k;
    }
};

// Whether windows of V elements fit rows at p the way they fit rows at q: the
// same place within a window, row after row.
template <int V>
bool in_step(const void *p, size_t ldp, size_t esp, const void *q, size_t ldq, size_t esq) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) / esp % V ==
                                reinterpret_cast<uintptr_t>(q) / esq % V &&
                            ldp % V == ldq % V);
}

// How a launch covers its rows.
struct Shape {
    int items = 0;    // windows a thread; 0: the row does not fit the registers
    unsigned tx = 0, ty = 1, grid = 0;
    int stages = 0;   // of a staged launch, else 0
    size_t smem = 0;
};

// Windows of a row; with edges, at the worst phase.
template <int V>
size_t windows_of(size_t hidden, bool edge) {
    return edge ? (hidden + 2 * (V - 1)) / V : hidden / V;
}

unsigned warps_of(size_t windows, int items) {
    return (unsigned)((windows + items - 1) / items + 31) / 32 * 32;
}

}  // namespace
}  // namespace purlin

// What stands above, a row's windows, sums and ring, serves block_norm.cu too, which
// includes this file for it.
#ifndef PURLIN_ROWS_ONLY

namespace purlin {
namespace {

struct NormParams {
    const void *x, *residual, *weight;
    void *y, *total;
    float *scales;
    size_t ldx, ldr, ldy, ldt, rows;
    uint32_t hidden, phase;   // phase of row 0's first element in its window
    float eps;
    int stages;               // of a staged launch
    unsigned long long *err;
};

// Threads of a block: 1024 where a thread holds little, else the registers for it.
constexpr int norm_threads(int held) { return held <= 8 ? 1024 : 512; }
constexpr int kBackwardThreads = 512, kStagedThreads = 512;
constexpr int kShortRows = 8;   // rows of a block with a warp a row
// Backward, fewer rows a block and fewer blocks: less to join (4000 x 768 bf16 16.4
// us, with 8 rows and 1024 threads an SM 31.6; 32768 x 512 30.7 and 39.0).
constexpr int kBackwardShortRows = 4, kBackwardThreadsSm = 512;

// A thread holds ITEMS windows of V elements of its row.  blockDim.y rows a
// block; more than one only where blockDim.x is one warp.  Up to 64 bytes a
// thread the next row and the weight are kept in registers too.
template <typename T, typename O, int V, int ITEMS, bool EDGE>
__global__ void __launch_bounds__(norm_threads(ITEMS * V))
norm_kernel(const __grid_constant__ NormParams p) {
    constexpr bool AHEAD = ITEMS * V * sizeof(T) <= 64;
    __shared__ float sums[2][32], maxes[2][32];   // rows take turns: a barrier a sum
    const bool warp_only = blockDim.x == 32;
    const size_t step = (size_t)gridDim.x * blockDim.y;
    size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.rows) return;   // whole warps; blockDim.y > 1 has no block barrier
    const int hidden = (int)p.hidden, phase = EDGE ? phase_of<V>(p.phase, p.ldx, row) : 0;
    const int e0 = (int)threadIdx.x * V - phase, estep = (int)blockDim.x * V;
    const T *w = static_cast<const T *>(p.weight);
    Window<T, V> wk[ITEMS], xk[ITEMS], rk[ITEMS];
    auto fetch = [&](size_t at) {
        const T *x = static_cast<const T *>(p.x) + at * p.ldx;
        const T *res = static_cast<const T *>(p.residual) + at * p.ldr;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) xk[i] = read_window<T, V, EDGE>(x, e0 + i * estep, hidden);
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) rk[i] = read_window<T, V, EDGE>(res, e0 + i * estep, hidden);
        }
    };
    fetch(row);
    if constexpr (AHEAD) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) wk[i] = read_weight<T, V, EDGE>(w, e0 + i * estep, hidden);
    }
    for (int turn = 0; row < p.rows; row += step, turn ^= 1) {
        float t[ITEMS][V];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                t[i][j] = xk[i].at(j);
                if (p.residual) t[i][j] += rk[i].at(j);
                ss = fmaf(t[i][j], t[i][j], ss);
            }
        if constexpr (AHEAD) {
            if (row + step < p.rows) fetch(row + step);
        } else {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) wk[i] = read_weight<T, V, EDGE>(w, e0 + i * estep, hidden);
        }
        if (p.total) {
            T *total = static_cast<T *>(p.total) + row * p.ldt;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) write_window<T, V, EDGE>(total, e0 + i * estep, hidden, t[i]);
        }
        const float r = rsqrtf(reduce_row<Sum>(ss, warp_only, sums[turn]) / (float)p.hidden + p.eps);
        O *y = static_cast<O *>(p.y) + row * p.ldy;
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                // a window's elements outside the row are zero and stay out of the
                // maximum, unless r is infinite
                t[i][j] = t[i][j] * r * wk[i].at(j);
                most = fmaxf(most, fabsf(t[i][j]));
            }
            if constexpr (sizeof(O) != 1) write_window<O, V, EDGE>(y, e0 + i * estep, hidden, t[i]);
        }
        if constexpr (sizeof(O) == 1) {
            // fmaxf passes over NaN: the scale stays a number, the elements are NaN
            const float scale =
                fmaxf(reduce_row<Max>(most, warp_only, maxes[turn]) / kE4m3Max, kScaleMin);
            divide_row(t, scale);
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) write_window<O, V, EDGE>(y, e0 + i * estep, hidden, t[i]);
            if (threadIdx.x == 0) p.scales[row] = scale;
        }
        if constexpr (!AHEAD) {
            if (row + step < p.rows) fetch(row + step);
        }
    }
}

template <typename T, typename O, int V, int ITEMS, bool EDGE>
__global__ void __launch_bounds__(kStagedThreads, 2)
norm_staged_kernel(const __grid_constant__ NormParams p) {
    using Ring = RowRing<T, V, 2>;
    extern __shared__ __align__(128) unsigned char stage[];
    __shared__ typename Ring::Shared shared;
    __shared__ float sums[2][32], maxes[2][32];
    const int hidden = (int)p.hidden, phase = EDGE ? phase_of<V>(p.phase, p.ldx, blockIdx.x) : 0;
    Ring ring(shared, stage + ITEMS * blockDim.x * 16, p.stages, p.residual ? 2 : 1, hidden, phase, blockIdx.x, gridDim.x,
              p.rows);
    ring.src[0] = static_cast<const T *>(p.x);
    ring.ld[0] = p.ldx;
    ring.src[1] = static_cast<const T *>(p.residual);
    ring.ld[1] = p.ldr;
    if (threadIdx.x == 0) ring.init();
    __syncthreads();
    if (threadIdx.x == 0)
        for (int i = 0; i < p.stages; ++i) ring.issue();
    const int e0 = (int)threadIdx.x * V - phase, estep = (int)blockDim.x * V;
    // the weight's windows before the stages; a thread reads back what it wrote
    const WeightStage<T, V> weight{stage};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        weight.put(i, read_weight<T, V, EDGE>(static_cast<const T *>(p.weight), e0 + i * estep, hidden));
    const float inv_hidden = 1.f / (float)hidden;
    uint32_t n = 0;
    for (size_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++n, ring.next()) {
        ring.wait(p.err);
        float t[ITEMS][V];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int w = (int)threadIdx.x + i * (int)blockDim.x;
            const Window<T, V> xk = ring.template read<EDGE>(row, 0, w, hidden);
#pragma unroll
            for (int j = 0; j < V; ++j) t[i][j] = xk.at(j);
            if (p.residual) {
                const Window<T, V> rk = ring.template read<EDGE>(row, 1, w, hidden);
#pragma unroll
                for (int j = 0; j < V; ++j) t[i][j] += rk.at(j);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) ss = fmaf(t[i][j], t[i][j], ss);
        }
        if (p.total) {
            T *total = static_cast<T *>(p.total) + row * p.ldt;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) write_window<T, V, EDGE>(total, e0 + i * estep, hidden, t[i]);
        }
        const float r =
            rsqrtf(mean_of(reduce_row<Sum>(ss, false, sums[n & 1]), (float)hidden, inv_hidden) + p.eps);
        if (threadIdx.x == 0) ring.issue();   // the sum's barrier: every thread has read its share
        O *y = static_cast<O *>(p.y) + row * p.ldy;
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const Window<T, V> wk = weight.get(i);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                t[i][j] = t[i][j] * r * wk.at(j);
                most = fmaxf(most, fabsf(t[i][j]));
            }
            if constexpr (sizeof(O) != 1) write_window<O, V, EDGE>(y, e0 + i * estep, hidden, t[i]);
        }
        if constexpr (sizeof(O) == 1) {
            // fmaxf passes over NaN: the scale stays a number, the elements are NaN
            const float scale =
                fmaxf(reduce_row<Max>(most, false, maxes[n & 1]) / kE4m3Max, kScaleMin);
            divide_row(t, scale);
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) write_window<O, V, EDGE>(y, e0 + i * estep, hidden, t[i]);
            if (threadIdx.x == 0) p.scales[row] = scale;
        }
    }
    if (threadIdx.x == 0) ring.drain(p.err);
}

// Rows too long for the registers: x and the residual are read again (from
// the L2 cache mostly) for the output, and a third time for an e4m3 output.  More
// than 16384 elements, or 16384 with an edge in bf16, which is one window more than
// the threads hold: 4096 x 16384 bf16 with a weight off its boundary takes 233 us,
// aligned 92 (to e4m3 294 and 78, backward 258 and 86).
template <typename T, typename O>
__global__ void __launch_bounds__(1024) norm_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float sums[32], maxes[32];
    const size_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *res = p.residual ? static_cast<const T *>(p.residual) + row * p.ldr : nullptr;
    const T *w = static_cast<const T *>(p.weight);
    O *y = static_cast<O *>(p.y) + row * p.ldy;
    auto at = [&](uint32_t e) {
        return res ? to_f32<T>(x[e]) + to_f32<T>(res[e]) : to_f32<T>(x[e]);
    };
    float ss = 0.f;
    for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
        const float t = at(e);
        ss = fmaf(t, t, ss);
    }
    const float r = rsqrtf(reduce_row<Sum>(ss, false, sums) / (float)p.hidden + p.eps);
    float scale = 1.f;
    if constexpr (sizeof(O) == 1) {
        float most = 0.f;
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x)
            most = fmaxf(most, fabsf(at(e) * r * to_f32<T>(w[e])));
        scale = fmaxf(reduce_row<Max>(most, false, maxes) / kE4m3Max, kScaleMin);
        if (threadIdx.x == 0) p.scales[row] = scale;
    }
    for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
        // total may be x or the residual itself: each element is read before it is written
        const float t = at(e);
        if (p.total) static_cast<T *>(p.total)[row * p.ldt + e] = from_f32<T>(t);
        const float v = t * r * to_f32<T>(w[e]);
        y[e] = from_f32<O>(sizeof(O) == 1 ? v / scale : v);
    }
}

// ---------------------------------------------------------------- backward --

struct NormBackwardParams {
    const void *dy, *total, *weight, *dtotal;
    void *dx;
    float *partial;   // gridDim.x x hidden
    size_t lddy, ldt, lddt, lddx, rows;
    uint32_t hidden, phase;
    float eps;
    int stages;
    unsigned long long *err;
};

// blockDim.y rows a block, more than one only where blockDim.x is one warp: then
// the warps' shares of dweight are added up in shared memory, warp by warp.  WIDE:
// blocks of up to 1024 threads, whose 64 registers do not hold a row, its gradient
// and dweight's sums: 300 bytes a thread are spilled, and the weight is read again
// every row.  Still faster than the long kernel (`wide`, in backward_shape).
template <typename T, int V, int ITEMS, bool EDGE, bool WIDE = false>
__global__ void __launch_bounds__(WIDE ? 1024 : kBackwardThreads)
norm_backward_kernel(const __grid_constant__ NormBackwardParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be launched
    constexpr bool AHEAD = !WIDE && ITEMS * V * sizeof(T) <= 32;
    __shared__ float sums[2][2][32];   // rows take turns: one barrier a row
    __shared__ float joined[32 * ITEMS * V];
    const int hidden = (int)p.hidden;
    const size_t step = (size_t)gridDim.x * blockDim.y;
    size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int phase = EDGE ? phase_of<V>(p.phase, p.lddy, row) : 0;
    const int e0 = (int)threadIdx.x * V - phase, estep = (int)blockDim.x * V;
    float acc[ITEMS][V] = {};
    Window<T, V> wk[ITEMS], gk[ITEMS], tk[ITEMS], dk[ITEMS];
    auto fetch = [&](size_t at) {
        const T *dy = static_cast<const T *>(p.dy) + at * p.lddy;
        const T *t = static_cast<const T *>(p.total) + at * p.ldt;
        const T *d = static_cast<const T *>(p.dtotal) + at * p.lddt;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            gk[i] = read_window<T, V, EDGE>(dy, e0 + i * estep, hidden);
            tk[i] = read_window<T, V, EDGE>(t, e0 + i * estep, hidden);
        }
        if (!WIDE && p.dtotal) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) dk[i] = read_window<T, V, EDGE>(d, e0 + i * estep, hidden);
        }
    };
    if (row < p.rows) fetch(row);
    auto weight = [&](int i) {
        return read_weight<T, V, EDGE>(static_cast<const T *>(p.weight), e0 + i * estep, hidden);
    };
    if constexpr (!WIDE) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) wk[i] = weight(i);
    }
    const int warps = blockDim.x >> 5;
    int turn = 0;
    for (; row < p.rows; row += step, turn ^= 1) {   // one row a warp, or all of the block's one
        Window<T, V> g[ITEMS], t[ITEMS], d[ITEMS];
        float tt = 0.f, gt = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            g[i] = gk[i];
            t[i] = tk[i];
            d[i] = dk[i];
            if constexpr (WIDE) wk[i] = weight(i);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = t[i].at(j);
                tt = fmaf(u, u, tt);
                gt = fmaf(g[i].at(j) * wk[i].at(j), u, gt);
            }
        }
        if constexpr (AHEAD) {
            if (row + step < p.rows) fetch(row + step);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            tt += __shfl_xor_sync(0xffffffffu, tt, o);
            gt += __shfl_xor_sync(0xffffffffu, gt, o);
        }
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) {
                sums[turn][0][threadIdx.x >> 5] = tt;
                sums[turn][1][threadIdx.x >> 5] = gt;
            }
            __syncthreads();
            tt = gt = 0.f;
            for (int k = 0; k < warps; ++k) {
                tt += sums[turn][0][k];
                gt += sums[turn][1][k];
            }
        }
        const float inv_hidden = 1.f / (float)p.hidden;
        // (a division here: without its call the compiler keeps the row unpacked over the
        // sums, and four windows of bf16 spill 500 bytes)
        const float r = rsqrtf(tt / (float)p.hidden + p.eps);
        const float c = r * r * mean_of(gt, (float)p.hidden, inv_hidden);
        T *dx = static_cast<T *>(p.dx) + row * p.lddx;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            float o[V];
            if constexpr (WIDE) {
                wk[i] = weight(i);
                if (p.dtotal)
                    d[i] = read_window<T, V, EDGE>(static_cast<const T *>(p.dtotal) + row * p.lddt,
                                                   e0 + i * estep, hidden);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = t[i].at(j), y = g[i].at(j);
                acc[i][j] = fmaf(y, u * r, acc[i][j]);
                o[j] = r * fmaf(y, wk[i].at(j), -(u * c));
                if (p.dtotal) o[j] += d[i].at(j);
            }
            write_window<T, V, EDGE>(dx, e0 + i * estep, hidden, o);
        }
        if constexpr (!AHEAD) {
            if (row + step < p.rows) fetch(row + step);
        }
    }
    float *partial = p.partial + (size_t)blockIdx.x * p.hidden;
    if (blockDim.y > 1) {
        for (unsigned y = 0; y < blockDim.y; ++y) {
            if (threadIdx.y == y) {
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int e = e0 + i * estep + j;
                        if (e >= 0 && e < hidden) joined[e] = y == 0 ? acc[i][j] : joined[e] + acc[i][j];
                    }
            }
            __syncthreads();
        }
        for (int e = (int)(threadIdx.y * blockDim.x + threadIdx.x); e < hidden;
             e += (int)(blockDim.x * blockDim.y))
            partial[e] = joined[e];
        return;
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = e0 + i * estep + j;
            if (e >= 0 && e < hidden) partial[e] = acc[i][j];
        }
}

template <typename T, int V, int ITEMS, bool EDGE>
__global__ void __launch_bounds__(kStagedThreads)
norm_backward_staged_kernel(const __grid_constant__ NormBackwardParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be launched
    using Ring = RowRing<T, V, 3>;
    extern __shared__ __align__(128) unsigned char stage[];
    __shared__ typename Ring::Shared shared;
    __shared__ float sums[2][2][32];   // rows take turns: one barrier a row
    const int hidden = (int)p.hidden;
    const int phase = EDGE ? phase_of<V>(p.phase, p.lddy, blockIdx.x) : 0;
    Ring ring(shared, stage + ITEMS * blockDim.x * 16, p.stages, p.dtotal ? 3 : 2, hidden, phase, blockIdx.x, gridDim.x,
              p.rows);
    ring.src[0] = static_cast<const T *>(p.dy);
    ring.ld[0] = p.lddy;
    ring.src[1] = static_cast<const T *>(p.total);
    ring.ld[1] = p.ldt;
    ring.src[2] = static_cast<const T *>(p.dtotal);
    ring.ld[2] = p.lddt;
    if (threadIdx.x == 0) ring.init();
    __syncthreads();
    if (threadIdx.x == 0)
        for (int i = 0; i < p.stages; ++i) ring.issue();
    const int e0 = (int)threadIdx.x * V - phase, estep = (int)blockDim.x * V;
    float acc[ITEMS][V] = {};
    // the weight's windows before the stages; a thread reads back what it wrote
    const WeightStage<T, V> weight{stage};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        weight.put(i, read_weight<T, V, EDGE>(static_cast<const T *>(p.weight), e0 + i * estep, hidden));
    const int warps = blockDim.x >> 5;
    const float inv_hidden = 1.f / (float)hidden;
    uint32_t n = 0;
    for (size_t row = blockIdx.x; row < p.rows; row += gridDim.x, ++n, ring.next()) {
        ring.wait(p.err);
        float tt = 0.f, gt = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int w = (int)threadIdx.x + i * (int)blockDim.x;
            const Window<T, V> g = ring.template read<EDGE>(row, 0, w, hidden);
            const Window<T, V> t = ring.template read<EDGE>(row, 1, w, hidden), wk = weight.get(i);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = t.at(j);
                tt = fmaf(u, u, tt);
                gt = fmaf(g.at(j) * wk.at(j), u, gt);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            tt += __shfl_xor_sync(0xffffffffu, tt, o);
            gt += __shfl_xor_sync(0xffffffffu, gt, o);
        }
        if ((threadIdx.x & 31) == 0) {
            sums[n & 1][0][threadIdx.x >> 5] = tt;
            sums[n & 1][1][threadIdx.x >> 5] = gt;
        }
        __syncthreads();
        // behind the barrier every thread is through with the row before
        if (threadIdx.x == 0 && n > 0) ring.issue();
        tt = gt = 0.f;
        for (int k = 0; k < warps; ++k) {
            tt += sums[n & 1][0][k];
            gt += sums[n & 1][1][k];
        }
        const float r = rsqrtf(mean_of(tt, (float)hidden, inv_hidden) + p.eps);
        const float c = r * r * mean_of(gt, (float)hidden, inv_hidden);
        T *dx = static_cast<T *>(p.dx) + row * p.lddx;
        // the row is read again rather than held: the registers go to dweight's sums
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int w = (int)threadIdx.x + i * (int)blockDim.x;
            const Window<T, V> g = ring.template read<EDGE>(row, 0, w, hidden);
            const Window<T, V> t = ring.template read<EDGE>(row, 1, w, hidden), wk = weight.get(i);
            Window<T, V> d;
            if (p.dtotal) d = ring.template read<EDGE>(row, 2, w, hidden);
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = t.at(j), y = g.at(j);
                acc[i][j] = fmaf(y, u * r, acc[i][j]);
                o[j] = r * fmaf(y, wk.at(j), -(u * c));
                if (p.dtotal) o[j] += d.at(j);
            }
            write_window<T, V, EDGE>(dx, e0 + i * estep, hidden, o);
        }
    }
    if (threadIdx.x == 0) ring.drain(p.err);
    float *partial = p.partial + (size_t)blockIdx.x * p.hidden;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = e0 + i * estep + j;
            if (e >= 0 && e < hidden) partial[e] = acc[i][j];
        }
}

// dx of rows too long for the registers.
template <typename T>
__global__ void __launch_bounds__(1024)
norm_backward_long_kernel(const __grid_constant__ NormBackwardParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be launched
    __shared__ float sums[2][32];
    float *partial = p.partial + (size_t)blockIdx.x * p.hidden;
    for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) partial[e] = 0.f;
    const T *w = static_cast<const T *>(p.weight);
    for (size_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *dy = static_cast<const T *>(p.dy) + row * p.lddy;
        const T *t = static_cast<const T *>(p.total) + row * p.ldt;
        float tt = 0.f, gt = 0.f;
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
            const float u = to_f32<T>(t[e]);
            tt = fmaf(u, u, tt);
            gt = fmaf(to_f32<T>(dy[e]) * to_f32<T>(w[e]), u, gt);
        }
        tt = reduce_row<Sum>(tt, false, sums[0]);
        gt = reduce_row<Sum>(gt, false, sums[1]);
        __syncthreads();   // before the next row's sums
        const float r = rsqrtf(tt / (float)p.hidden + p.eps);
        const float c = r * r * (gt / (float)p.hidden);
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
            const float u = to_f32<T>(t[e]), d = to_f32<T>(dy[e]);
            float o = r * fmaf(d, to_f32<T>(w[e]), -(u * c));
            if (p.dtotal) o += to_f32<T>(static_cast<const T *>(p.dtotal)[row * p.lddt + e]);
            static_cast<T *>(p.dx)[row * p.lddx + e] = from_f32<T>(o);
            partial[e] = fmaf(d, u * r, partial[e]);
        }
    }
}

// dweight[e] = the blocks' partial sums: kJoinRows threads a column, each every
// kJoinRows-th block in order, then joined in order.
constexpr int kJoinRows = 32;

__global__ void __launch_bounds__(32 * kJoinRows)
norm_join_kernel(const float *partial, float *dweight, uint32_t hidden, int parts) {
    __shared__ float sums[kJoinRows][33];
    const uint32_t e = blockIdx.x * 32 + threadIdx.x;
    // launched while the rows are still being worked on: wait for all of them
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v = 0.f;
    if (e < hidden) {
#pragma unroll 8
        for (int b = threadIdx.y; b < parts; b += kJoinRows) v += partial[(size_t)b * hidden + e];
    }
    sums[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y != 0 || e >= hidden) return;
    v = sums[0][threadIdx.x];
#pragma unroll
    for (int k = 1; k < kJoinRows; ++k) v += sums[k][threadIdx.x];
    dweight[e] = v;
}

// Rows on the registers alone: the fewest windows a thread that `threads(items)`
// threads allow, which is the quickest for a block's first row.
template <int V, typename F>
Shape register_shape(size_t rows, size_t hidden, bool edge, int most_items, int sms,
                     int short_rows, int threads_sm, F threads) {
    Shape s;
    const size_t windows = windows_of<V>(hidden, edge);
    // a warp a row as soon as it can hold one: many short rows
    const int least = rows >= 8 * (size_t)sms && windows <= (size_t)32 * most_items ? most_items : 1;
    for (int items = least; items <= most_items; items *= 2) {
        const unsigned tx = warps_of(windows, items);
        if (tx > (unsigned)threads(items)) continue;
        s.items = items;
        s.tx = tx;
        break;
    }
    if (s.items == 0) return s;
    while (s.items > 1 && warps_of(windows, s.items / 2) == s.tx) s.items /= 2;
    s.ty = s.tx == 32 ? (unsigned)short_rows : 1;
    // a multiple of the windows' elements, so that a block's rows share their phase,
    // or a row a block
    const size_t blocks = std::max<size_t>(1, threads_sm / (s.tx * s.ty));
    const size_t grid = std::max<size_t>((size_t)sms * blocks / V * V, V);
    s.grid = (unsigned)std::min<size_t>((rows + s.ty - 1) / s.ty, grid);
    return s;
}

// Rows through shared memory.  items 0 where there are too few rows, or a row fits
// a warp, or the stages do not fit.  About 14 warps an SM and 96 KiB of
// rows on their way keep the memory busy; with twice that many the reads run so
// far ahead of the writes that it slows down (e4m3 from 7168 bf16 columns with a
// residual: two blocks of two stages 6.63 TB/s, of four 3.70; three of two 5.56, one
// of four 4.26).  `late`: a stage is refilled only a row later, so two of them leave
// gaps (32768 x 4096 bf16: three 170 us, two 198).
template <int V>
Shape staged_shape(size_t rows, size_t hidden, bool edge, int arrays, int sms, bool late) {
    Shape s;
    constexpr size_t kSmemSm = 227 * 1024, kReserved = 3 * 1024;   // an SM's; a block's own
    constexpr size_t kFlight = 96 * 1024;
    const size_t threads_sm = edge ? 640 : 448;   // edges take more instructions a row
    const size_t windows = windows_of<V>(hidden, edge);
    const size_t stage = (hidden + 2 * (V - 1)) / V * 16 * (size_t)arrays;   // as RowRing has it
    // a row that fits a warp's registers stays there; backward, where dweight's sums
    // need them, less of one does (32768 x 1024 bf16 55.4 us, from registers 61.5)
    if (V == 1 || windows <= (late ? 100 : 128)) return s;
    const int items = warps_of(windows, 4) <= (unsigned)kStagedThreads ? 4 : 8;
    const unsigned tx = warps_of(windows, items);
    if (items * V > 32 || tx > (unsigned)kStagedThreads) return s;
    const size_t weight = (size_t)items * tx * 16;
    for (size_t b = std::max<size_t>(2, threads_sm / tx); b >= 1; --b) {
        if (kSmemSm / b < kReserved + weight) continue;
        const size_t fit = std::min<size_t>((kSmemSm / b - kReserved - weight) / stage, kMaxStages);
        const size_t least = late && (b > 2 || tx >= 256) && b > 1 ? 3 : 2;
        if (fit < least) continue;
        const size_t stages =
            std::max(late ? std::min<size_t>(fit, 3) : least, std::min(fit, kFlight / (b * stage)));
        // forward, from a row an SM on (500 x 7168 to e4m3 8.2 us, from registers 12.3);
        // backward, where a block has two (509 x 1021 f32 10.3 us, from registers 7.5)
        if (rows < (late ? 2 * b : 1) * (size_t)sms) return s;
        s.items = items;
        s.tx = tx;
        s.stages = (int)(b == 1 ? fit : stages);
        s.smem = weight + (size_t)s.stages * stage;
        s.grid = (unsigned)std::min<size_t>(rows, std::max<size_t>((size_t)sms * b / V * V, V));
        break;
    }
    return s;
}

constexpr int kStagedSmem = 224 * 1024;   // most dynamic shared memory of a staged launch

template <typename T, typename O, int V, bool EDGE>
cudaError_t norm_typed(const NormArgs &a, NormParams &p) {
    if constexpr (V > 1) {
        const Shape s =
            staged_shape<V>(a.rows, a.hidden, EDGE, a.residual ? 2 : 1, a.sms, false);
        auto run = [&](auto kernel, SharedMemoryLimit &limit) {
            const cudaError_t ready = limit.raise(kernel, kStagedSmem);
            if (ready != cudaSuccess) return ready;
            kernel<<<s.grid, s.tx, s.smem, a.stream>>>(p);
            return cudaGetLastError();
        };
        p.stages = s.stages;
        if (s.items == 4) {
            static SharedMemoryLimit limit;
            return run(norm_staged_kernel<T, O, V, 4, EDGE>, limit);
        }
        if constexpr (V == 4) {
            if (s.items == 8) {
                static SharedMemoryLimit limit;
                return run(norm_staged_kernel<T, O, V, 8, EDGE>, limit);
            }
        }
    }
    constexpr int kMost = std::min(8, 32 / V);
    const Shape s = register_shape<V>(a.rows, a.hidden, EDGE, kMost, a.sms, kShortRows, 1024,
                                      [](int items) { return norm_threads(items * V); });
    const dim3 block(s.tx, s.ty);
    if (s.items == 1) norm_kernel<T, O, V, 1, EDGE><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == 2) norm_kernel<T, O, V, 2, EDGE><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == 4) norm_kernel<T, O, V, 4, EDGE><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == 8) {
        if constexpr (kMost >= 8) norm_kernel<T, O, V, 8, EDGE><<<s.grid, block, 0, a.stream>>>(p);
    } else
        norm_long_kernel<T, O><<<(unsigned)a.rows, 1024, 0, a.stream>>>(p);
    return cudaGetLastError();
}

template <typename T, typename O>
cudaError_t norm_any(const NormArgs &a) {
    constexpr int V = 16 / sizeof(T);
    constexpr size_t es = sizeof(T);
    NormParams p{a.x, a.residual, a.weight, a.y, a.total, a.scales, a.ldx, a.ldr, a.ldy, a.ldt,
                 a.rows, (uint32_t)a.hidden, (uint32_t)(reinterpret_cast<uintptr_t>(a.x) / es % V),
                 a.eps, 0, a.err};
    if (in_step<V>(a.residual, a.ldr, es, a.x, a.ldx, es) &&
        in_step<V>(a.total, a.ldt, es, a.x, a.ldx, es) &&
        in_step<V>(a.y, a.ldy, sizeof(O), a.x, a.ldx, es)) {
        if (p.phase == 0 && a.ldx % V == 0 && a.hidden % V == 0 &&
            reinterpret_cast<uintptr_t>(a.weight) % 16 == 0)
            return norm_typed<T, O, V, false>(a, p);
        return norm_typed<T, O, V, true>(a, p);
    }
    return norm_typed<T, O, 1, false>(a, p);
}

// A backward launch: its shape, and whether it takes windows and meets edges.
struct BackwardShape : Shape {
    bool windows = false, edge = false, wide = false;
};

template <typename T>
BackwardShape backward_shape(const NormBackwardArgs &a) {
    constexpr int V = 16 / sizeof(T);
    constexpr size_t es = sizeof(T);
    BackwardShape s;
    s.windows = in_step<V>(a.total, a.ldt, es, a.dy, a.lddy, es) &&
                in_step<V>(a.dtotal, a.lddt, es, a.dy, a.lddy, es) &&
                in_step<V>(a.dx, a.lddx, es, a.dy, a.lddy, es);
    s.edge = s.windows && !(reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 && a.lddy % V == 0 &&
                            a.hidden % V == 0 && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0);
    const auto threads = [](int) { return kBackwardThreads; };
    Shape &base = s;
    if (s.windows) base = staged_shape<V>(a.rows, a.hidden, s.edge, a.dtotal ? 3 : 2, a.sms, true);
    if (s.items != 4)   // eight windows a thread are too many here: dweight's sums and the weight
        base = s.windows
                   ? register_shape<V>(a.rows, a.hidden, s.edge, 4, a.sms, kBackwardShortRows,
                                       kBackwardThreadsSm, threads)
                   : register_shape<1>(a.rows, a.hidden, false, 4, a.sms, kBackwardShortRows,
                                       kBackwardThreadsSm, threads);
    const unsigned most = s.windows ? warps_of(windows_of<V>(a.hidden, s.edge), 4) : 2048;
    if (s.items == 0 && V == 4 && most <= 1024) {
        // rows of 8192 to 16384 f32: a block an SM (3000 x 16384 140 us, read again from
        // the L2 cache 263; with dtotal 184 and 313; 3000 x 8200 98 and 121)
        s.wide = true;
        s.items = 4;
        s.tx = most;
        s.grid = (unsigned)std::min<size_t>(a.rows, std::max<size_t>(a.sms / V * V, V));
    } else if (s.items == 0) {
        s.grid = (unsigned)std::max<size_t>(1, std::min<size_t>(a.rows, (size_t)a.sms * 2));
    }
    return s;
}

template <typename T, int V, bool EDGE>
cudaError_t norm_backward_typed(const NormBackwardArgs &a, const NormBackwardParams &p,
                                const BackwardShape &s) {
    if constexpr (V == 4) {
        if (s.wide) {
            norm_backward_kernel<T, V, 4, EDGE, true><<<s.grid, s.tx, 0, a.stream>>>(p);
            return cudaGetLastError();
        }
    }
    if constexpr (V > 1) {
        if (s.stages > 0) {
            static SharedMemoryLimit limit;
            const cudaError_t ready =
                limit.raise(norm_backward_staged_kernel<T, V, 4, EDGE>, kStagedSmem);
            if (ready != cudaSuccess) return ready;
            norm_backward_staged_kernel<T, V, 4, EDGE><<<s.grid, s.tx, s.smem, a.stream>>>(p);
            return cudaGetLastError();
        }
    }
    const dim3 block(s.tx, s.ty);
    if (s.items == 1) norm_backward_kernel<T, V, 1, EDGE><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == 2) norm_backward_kernel<T, V, 2, EDGE><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == 4) norm_backward_kernel<T, V, 4, EDGE><<<s.grid, block, 0, a.stream>>>(p);
    else norm_backward_long_kernel<T><<<s.grid, 1024, 0, a.stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t norm_backward_any(const NormBackwardArgs &a) {
    constexpr int V = 16 / sizeof(T);
    const BackwardShape s = backward_shape<T>(a);
    NormBackwardParams p{a.dy, a.total, a.weight, a.dtotal, a.dx, a.partial, a.lddy, a.ldt, a.lddt,
                         a.lddx, a.rows, (uint32_t)a.hidden,
                         (uint32_t)(reinterpret_cast<uintptr_t>(a.dy) / sizeof(T) % V), a.eps,
                         s.stages, a.err};
    const cudaError_t e = !s.windows ? norm_backward_typed<T, 1, false>(a, p, s)
                          : s.edge   ? norm_backward_typed<T, V, true>(a, p, s)
                                     : norm_backward_typed<T, V, false>(a, p, s);
    if (e != cudaSuccess) return e;
    // the join's launch overlaps the rows' kernel (509 x 1021 f32 7.5 us, launched after it 9.1)
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)((a.hidden + 31) / 32));
    c.blockDim = dim3(32, kJoinRows);
    c.stream = a.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, norm_join_kernel, (const float *)a.partial, a.dweight,
                              (uint32_t)a.hidden, (int)s.grid);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a) {
    if (a.dtype == PURLIN_F32)
        return a.out_dtype == PURLIN_E4M3 ? norm_any<float, __nv_fp8_e4m3>(a)
                                          : norm_any<float, float>(a);
    return a.out_dtype == PURLIN_E4M3 ? norm_any<__nv_bfloat16, __nv_fp8_e4m3>(a)
                                      : norm_any<__nv_bfloat16, __nv_bfloat16>(a);
}

size_t norm_backward_workspace(const NormBackwardArgs &a) {
    const Shape s = a.dtype == PURLIN_F32 ? backward_shape<float>(a)
                                          : backward_shape<__nv_bfloat16>(a);
    return (size_t)s.grid * a.hidden * sizeof(float);
}

cudaError_t launch_norm_backward(const NormBackwardArgs &a) {
    return a.dtype == PURLIN_F32 ? norm_backward_any<float>(a)
                                 : norm_backward_any<__nv_bfloat16>(a);
}

}  // namespace purlin

#endif  // PURLIN_ROWS_ONLY
