// rms_norm.cu -- root-mean-square norm with the residual's addition, output
// in the input's type or in e4m3 with one scale a row, and its backward pass.
//
// Forward, a row at a time, in binary32:
//   t = x + residual,  r = 1 / sqrt(mean(t^2) + eps),  y = t r w.
// One pass over memory: a row's t stays in the registers of the threads that
// loaded it (a block, or one warp for short rows), so x and the residual are
// read once and total and y written once; two block sums (t^2, then max |y|
// for e4m3) separate the load from the store.  Bound by bytes.
//
// Backward, with g = dy w:
//   dx = r (g - t r^2 mean(g t)) + dtotal,  dweight = sum over rows of dy t r.
// A block owns whole rows and walks them with the grid's stride; a thread owns
// the same columns in every row, so its share of dweight is a register sum,
// written once a block and added up over the blocks in block order by a second
// kernel: no atomics, the same bits every time.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "layers.h"

namespace purlin {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 1.17549435e-38f;   // 2^-126: its reciprocal is finite

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

// V elements as one aligned memory access.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ void load(const T *p, float (&out)[V]) {
    const Pack<T, V> k = *reinterpret_cast<const Pack<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = to_f32<T>(k.v[i]);
}

template <typename T, int V>
__device__ __forceinline__ void store(T *p, const float (&in)[V]) {
    Pack<T, V> k;
#pragma unroll
    for (int i = 0; i < V; ++i) k.v[i] = from_f32<T>(in[i]);
    *reinterpret_cast<Pack<T, V> *>(p) = k;
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

struct NormParams {
    const void *x, *residual, *weight;
    void *y, *total;
    float *scales;
    size_t ldx, ldr, ldy, ldt, rows;
    uint32_t hidden;
    float eps;
};

// A thread holds ITEMS chunks of V elements of its row.  blockDim.y rows a
// block; more than one only where blockDim.x is one warp.
template <typename T, typename O, int V, int ITEMS>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float sums[32], maxes[32];
    const bool warp_only = blockDim.x == 32;
    const size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.rows) return;   // whole warps; blockDim.y > 1 has no block barrier
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *res = p.residual ? static_cast<const T *>(p.residual) + row * p.ldr : nullptr;
    float t[ITEMS][V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const uint32_t e = (threadIdx.x + i * blockDim.x) * V;
        if (e < p.hidden) {
            load<T, V>(x + e, t[i]);
            if (res) {
                float u[V];
                load<T, V>(res + e, u);
#pragma unroll
                for (int j = 0; j < V; ++j) t[i][j] += u[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) t[i][j] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(t[i][j], t[i][j], ss);
    if (p.total) {
        T *total = static_cast<T *>(p.total) + row * p.ldt;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t e = (threadIdx.x + i * blockDim.x) * V;
            if (e < p.hidden) store<T, V>(total + e, t[i]);
        }
    }
    const float r = rsqrtf(reduce_row<Sum>(ss, warp_only, sums) / (float)p.hidden + p.eps);
    const T *w = static_cast<const T *>(p.weight);
    O *y = static_cast<O *>(p.y) + row * p.ldy;
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const uint32_t e = (threadIdx.x + i * blockDim.x) * V;
        if (e < p.hidden) {
            float u[V];
            load<T, V>(w + e, u);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                t[i][j] = t[i][j] * r * u[j];
                most = fmaxf(most, fabsf(t[i][j]));
            }
            if constexpr (sizeof(O) != 1) store<O, V>(y + e, t[i]);
        }
    }
    if constexpr (sizeof(O) == 1) {
        // fmaxf passes over NaN: the scale stays a number, the elements are NaN
        const float scale = fmaxf(reduce_row<Max>(most, warp_only, maxes) / kE4m3Max, kScaleMin);
        const float inv = 1.f / scale;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t e = (threadIdx.x + i * blockDim.x) * V;
            if (e < p.hidden) {
#pragma unroll
                for (int j = 0; j < V; ++j) t[i][j] *= inv;
                store<O, V>(y + e, t[i]);
            }
        }
        if (threadIdx.x == 0) p.scales[row] = scale;
    }
}

// Rows too long for the registers: x and the residual are read again (from
// the L2 cache mostly) for the output, and a third time for an e4m3 output.
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
    float inv = 1.f;
    if constexpr (sizeof(O) == 1) {
        float most = 0.f;
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x)
            most = fmaxf(most, fabsf(at(e) * r * to_f32<T>(w[e])));
        const float scale = fmaxf(reduce_row<Max>(most, false, maxes) / kE4m3Max, kScaleMin);
        inv = 1.f / scale;
        if (threadIdx.x == 0) p.scales[row] = scale;
    }
    for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
        // total may be x or the residual itself: each element is read before it is written
        const float t = at(e);
        if (p.total) static_cast<T *>(p.total)[row * p.ldt + e] = from_f32<T>(t);
        y[e] = from_f32<O>(t * r * to_f32<T>(w[e]) * inv);
    }
}

// ---------------------------------------------------------------- backward --

struct NormBackwardParams {
    const void *dy, *total, *weight, *dtotal;
    void *dx;
    float *partial;   // gridDim.x x hidden
    size_t lddy, ldt, lddt, lddx, rows;
    uint32_t hidden;
    float eps;
};

template <typename T, int V, int ITEMS>
__global__ void __launch_bounds__(1024)
norm_backward_kernel(const __grid_constant__ NormBackwardParams p) {
    __shared__ float sums[2][2][32];   // two rows in turn: one barrier a row
    float acc[ITEMS][V] = {};
    float w[ITEMS][V] = {};
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const uint32_t e = (threadIdx.x + i * blockDim.x) * V;
        if (e < p.hidden) load<T, V>(static_cast<const T *>(p.weight) + e, w[i]);
    }
    const int warps = blockDim.x >> 5;
    int turn = 0;
    for (size_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
        const T *dyp = static_cast<const T *>(p.dy) + row * p.lddy;
        const T *tp = static_cast<const T *>(p.total) + row * p.ldt;
        float dy[ITEMS][V], t[ITEMS][V];
        float tt = 0.f, gt = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t e = (threadIdx.x + i * blockDim.x) * V;
            if (e < p.hidden) {
                load<T, V>(dyp + e, dy[i]);
                load<T, V>(tp + e, t[i]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) dy[i][j] = t[i][j] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                tt = fmaf(t[i][j], t[i][j], tt);
                gt = fmaf(dy[i][j] * w[i][j], t[i][j], gt);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            tt += __shfl_xor_sync(0xffffffffu, tt, o);
            gt += __shfl_xor_sync(0xffffffffu, gt, o);
        }
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
        const float inv_n = 1.f / (float)p.hidden;
        const float r = rsqrtf(tt / (float)p.hidden + p.eps);
        const float c = r * r * (gt * inv_n);
        T *dxp = static_cast<T *>(p.dx) + row * p.lddx;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t e = (threadIdx.x + i * blockDim.x) * V;
            if (e >= p.hidden) continue;
            float d[V];
            if (p.dtotal) {
                load<T, V>(static_cast<const T *>(p.dtotal) + row * p.lddt + e, d);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) d[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                acc[i][j] = fmaf(dy[i][j], t[i][j] * r, acc[i][j]);
                d[j] += r * (dy[i][j] * w[i][j] - t[i][j] * c);
            }
            store<T, V>(dxp + e, d);
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const uint32_t e = (threadIdx.x + i * blockDim.x) * V;
        if (e >= p.hidden) continue;
#pragma unroll
        for (int j = 0; j < V; ++j)
            p.partial[(size_t)blockIdx.x * p.hidden + e + j] = acc[i][j];
    }
}

// dx of rows too long for the registers.
template <typename T>
__global__ void __launch_bounds__(1024)
norm_backward_long_kernel(const __grid_constant__ NormBackwardParams p) {
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
            float o = r * (d * to_f32<T>(w[e]) - u * c);
            if (p.dtotal) o += to_f32<T>(static_cast<const T *>(p.dtotal)[row * p.lddt + e]);
            static_cast<T *>(p.dx)[row * p.lddx + e] = from_f32<T>(o);
            partial[e] = fmaf(d, u * r, partial[e]);
        }
    }
}

// dweight[e] = the blocks' partial sums, in block order.
__global__ void norm_join_kernel(const float *partial, float *dweight, uint32_t hidden, int parts) {
    const uint32_t e = blockIdx.x * blockDim.x + threadIdx.x;
    if (e >= hidden) return;
    float v = 0.f;
    for (int b = 0; b < parts; ++b) v += partial[(size_t)b * hidden + e];
    dweight[e] = v;
}

constexpr int kMaxItems = 8;

bool aligned16(const void *p, size_t ld, size_t es) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (ld * es)) & 15u) == 0;
}

// Chunks a thread holds: as few as a block of `most` threads allows.
int items_for(size_t chunks, size_t most) {
    int items = 1;
    while (items < kMaxItems && (chunks + items - 1) / items > most) items *= 2;
    return items;
}

template <typename T, typename O, int V>
cudaError_t norm_typed(const NormArgs &a, const NormParams &p) {
    const size_t chunks = (a.hidden + V - 1) / V;
    int items = items_for(chunks, 512);
    if (chunks > (size_t)items * 1024) {
        norm_long_kernel<T, O><<<(unsigned)a.rows, 1024, 0, a.stream>>>(p);
        return cudaGetLastError();
    }
    unsigned tx = (unsigned)(((chunks + items - 1) / items + 31) / 32 * 32);
    dim3 block(tx, tx == 32 ? 4 : 1);
    const unsigned grid = (unsigned)((a.rows + block.y - 1) / block.y);
    switch (items) {
        case 1: norm_kernel<T, O, V, 1><<<grid, block, 0, a.stream>>>(p); break;
        case 2: norm_kernel<T, O, V, 2><<<grid, block, 0, a.stream>>>(p); break;
        case 4: norm_kernel<T, O, V, 4><<<grid, block, 0, a.stream>>>(p); break;
        default: norm_kernel<T, O, V, 8><<<grid, block, 0, a.stream>>>(p); break;
    }
    return cudaGetLastError();
}

template <typename T, typename O>
cudaError_t norm_any(const NormArgs &a) {
    NormParams p{a.x, a.residual, a.weight, a.y, a.total, a.scales, a.ldx, a.ldr, a.ldy, a.ldt,
                 a.rows, (uint32_t)a.hidden, a.eps};
    constexpr int V = 16 / sizeof(T);
    // e4m3 chunks are V bytes: their alignment is V
    const bool y_ok = ((reinterpret_cast<uintptr_t>(a.y) | (a.ldy * sizeof(O))) &
                       (V * sizeof(O) - 1)) == 0;
    if (a.hidden % V == 0 && y_ok && aligned16(a.x, a.ldx, sizeof(T)) &&
        aligned16(a.residual, a.ldr, sizeof(T)) && aligned16(a.total, a.ldt, sizeof(T)) &&
        aligned16(a.weight, 0, sizeof(T)))
        return norm_typed<T, O, V>(a, p);
    return norm_typed<T, O, 1>(a, p);
}

template <typename T, int V>
cudaError_t norm_backward_typed(const NormBackwardArgs &a, const NormBackwardParams &p) {
    const size_t chunks = (a.hidden + V - 1) / V;
    int items = items_for(chunks, 512);
    if (chunks > (size_t)items * 1024) {
        norm_backward_long_kernel<T><<<a.ctas, 1024, 0, a.stream>>>(p);
    } else {
        const unsigned tx = (unsigned)(((chunks + items - 1) / items + 31) / 32 * 32);
        switch (items) {
            case 1: norm_backward_kernel<T, V, 1><<<a.ctas, tx, 0, a.stream>>>(p); break;
            case 2: norm_backward_kernel<T, V, 2><<<a.ctas, tx, 0, a.stream>>>(p); break;
            case 4: norm_backward_kernel<T, V, 4><<<a.ctas, tx, 0, a.stream>>>(p); break;
            default: norm_backward_kernel<T, V, 8><<<a.ctas, tx, 0, a.stream>>>(p); break;
        }
    }
    norm_join_kernel<<<(unsigned)((a.hidden + 127) / 128), 128, 0, a.stream>>>(
        a.partial, a.dweight, (uint32_t)a.hidden, a.ctas);
    return cudaGetLastError();
}

template <typename T>
cudaError_t norm_backward_any(const NormBackwardArgs &a) {
    NormBackwardParams p{a.dy, a.total, a.weight, a.dtotal, a.dx, a.partial, a.lddy, a.ldt, a.lddt,
                         a.lddx, a.rows, (uint32_t)a.hidden, a.eps};
    constexpr int V = 16 / sizeof(T);
    if (a.hidden % V == 0 && aligned16(a.dy, a.lddy, sizeof(T)) &&
        aligned16(a.total, a.ldt, sizeof(T)) && aligned16(a.dtotal, a.lddt, sizeof(T)) &&
        aligned16(a.dx, a.lddx, sizeof(T)) && aligned16(a.weight, 0, sizeof(T)))
        return norm_backward_typed<T, V>(a, p);
    return norm_backward_typed<T, 1>(a, p);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a) {
    if (a.dtype == PURLIN_F32)
        return a.out_dtype == PURLIN_E4M3 ? norm_any<float, __nv_fp8_e4m3>(a)
                                          : norm_any<float, float>(a);
    return a.out_dtype == PURLIN_E4M3 ? norm_any<__nv_bfloat16, __nv_fp8_e4m3>(a)
                                      : norm_any<__nv_bfloat16, __nv_bfloat16>(a);
}

int norm_backward_ctas(size_t rows, size_t hidden, int dtype, int sms) {
    (void)hidden;
    (void)dtype;
    return (int)std::max<size_t>(1, std::min<size_t>(rows, (size_t)sms * 2));
}

cudaError_t launch_norm_backward(const NormBackwardArgs &a) {
    return a.dtype == PURLIN_F32 ? norm_backward_any<float>(a)
                                 : norm_backward_any<__nv_bfloat16>(a);
}

}  // namespace purlin
