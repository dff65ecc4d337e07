// block_norm.cu -- the norms after and before a block, with the block's gate and the
// residual's addition between them, and their backward pass.
//
// Forward, a row at a time, in binary32, with c = block_scale * post_weight * gate:
//   q = 1 / sqrt(mean(x^2) + eps),  t = residual_scale * residual + c x q,
//   r = 1 / sqrt(mean(t^2) + eps),  y = t r weight.
// Backward, with n = dy weight:
//   dt = r (n - t r^2 mean(n t)) + dtotal,  h = c dt,  dx = q (h - x q^2 mean(h x)),
// and the sums over rows  dweight = sum dy t r,  S = sum dt x q (gate):  of a column
// gate and the weight after the block, dgate = block_scale post_weight S and
// dpost_weight = block_scale gate S.
#define PURLIN_ROWS_ONLY
#include "rms_norm.cu"

namespace purlin {
namespace {

struct BlockParams {
    const void *x, *post, *gate, *residual, *weight;
    void *y, *total;
    float *scales;
    size_t ldx, ldg, ldr, ldy, ldt, rows;
    uint32_t hidden, phase;   // phase of row 0's first element in its window
    float block_scale, residual_scale, eps;
    bool gate_rows;
    int stages;               // of a staged launch
    unsigned long long *err;
};

constexpr int kStagedThreads = 512;
constexpr int kStagedSmem = 224 * 1024;       // most dynamic shared memory of a staged launch
constexpr size_t kBlockThreadsSm = 448;       // threads an SM that a staged launch aims at
constexpr size_t kBackwardThreadsSmDirect = 512;
constexpr size_t kBlockFlight = 96 * 1024;    // bytes of rows on their way, an SM

// Rows too long for the registers, element by element: x, the residual and the gate
// are read again, from the L2 cache mostly, for every sum.
template <typename T, typename O>
__global__ void __launch_bounds__(1024) block_norm_long_kernel(const __grid_constant__ BlockParams p) {
    __shared__ float sums[3][32];
    const size_t row = blockIdx.x;
    const T *x = static_cast<const T *>(p.x) + row * p.ldx;
    const T *res = p.residual ? static_cast<const T *>(p.residual) + row * p.ldr : nullptr;
    const T *gate = static_cast<const T *>(p.gate);
    if (p.gate_rows) gate += row * p.ldg;
    const T *post = static_cast<const T *>(p.post), *w = static_cast<const T *>(p.weight);
    float q = 1.f;
    if (post) {
        float xx = 0.f;
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
            const float v = to_f32<T>(x[e]);
            xx = fmaf(v, v, xx);
        }
        q = rsqrtf(reduce_row<Sum>(xx, false, sums[0]) / (float)p.hidden + p.eps);
    }
    auto at = [&](uint32_t e) {
        float u = to_f32<T>(x[e]) * q * p.block_scale;
        if (post) u *= to_f32<T>(post[e]);
        if (gate) u *= to_f32<T>(gate[e]);
        return res ? fmaf(p.residual_scale, to_f32<T>(res[e]), u) : u;
    };
    float r = 0.f, scale = 1.f;
    if (p.y) {
        float tt = 0.f;
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
            const float t = at(e);
            tt = fmaf(t, t, tt);
        }
        r = rsqrtf(reduce_row<Sum>(tt, false, sums[1]) / (float)p.hidden + p.eps);
    }
    if constexpr (sizeof(O) == 1) {
        float most = 0.f;
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x)
            most = fmaxf(most, fabsf(at(e) * r * to_f32<T>(w[e])));
        scale = fmaxf(reduce_row<Max>(most, false, sums[2]) / kE4m3Max, kScaleMin);
        if (threadIdx.x == 0) p.scales[row] = scale;
    }
    for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
        // total and y may be x or the residual: each element is read before it is written
        const float t = at(e);
        if (p.total) static_cast<T *>(p.total)[row * p.ldt + e] = from_f32<T>(t);
        if (!p.y) continue;
        const float v = t * r * to_f32<T>(w[e]);
        static_cast<O *>(p.y)[row * p.ldy + e] = from_f32<O>(sizeof(O) == 1 ? v / scale : v);
    }
}

// The factor of x q in t for a thread's windows, block_scale * post_weight * column
// gate, in binary32: staged rows keep it in shared memory, each thread its own.
template <typename T, int V, bool EDGE>
__device__ __forceinline__ void read_factor(const void *post, const void *gate, float scale, int e,
                                            int hidden, float (&c)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) c[j] = scale;
    if (post) {
        const Window<T, V> k = read_weight<T, V, EDGE>(static_cast<const T *>(post), e, hidden);
#pragma unroll
        for (int j = 0; j < V; ++j) c[j] *= k.at(j);
    }
    if (gate) {
        const Window<T, V> k = read_weight<T, V, EDGE>(static_cast<const T *>(gate), e, hidden);
#pragma unroll
        for (int j = 0; j < V; ++j) c[j] *= k.at(j);
    }
}

template <int V>
struct FactorStage {
    unsigned char *base;
    __device__ float4 *at(int i, int q) const {
        return reinterpret_cast<float4 *>(base) + (size_t)(i * (V / 4) + q) * blockDim.x + threadIdx.x;
    }
    __device__ void put(int i, const float (&c)[V]) const {
#pragma unroll
        for (int q = 0; q < V / 4; ++q)
            *at(i, q) = make_float4(c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]);
    }
    __device__ void get(int i, float (&c)[V]) const {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
            const float4 f = *at(i, q);
            c[4 * q] = f.x;
            c[4 * q + 1] = f.y;
            c[4 * q + 2] = f.z;
            c[4 * q + 3] = f.w;
        }
    }
};

// A thread holds ITEMS windows of V elements of its row's t.  STAGED: a block a row,
// rows through shared memory.  Else a block a row, or a warp (then blockDim.y rows a
// block), and every operand straight from global memory, x twice.
template <typename T, typename O, int V, int ITEMS, bool EDGE, bool STAGED, int THREADS>
__global__ void __launch_bounds__(THREADS)
block_norm_kernel(const __grid_constant__ BlockParams p) {
    using Ring = RowRing<T, V, 3>;
    extern __shared__ __align__(128) unsigned char stage[];
    __shared__ typename Ring::Shared shared;
    __shared__ float sums[3][2][32];   // rows take turns: a barrier a sum
    const bool warp_only = !STAGED && blockDim.x == 32;
    const size_t step = (size_t)gridDim.x * blockDim.y;
    size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.rows) return;   // whole warps; blockDim.y > 1 has no block barrier
    const int hidden = (int)p.hidden, estep = (int)blockDim.x * V;
    const T *x = static_cast<const T *>(p.x), *residual = static_cast<const T *>(p.residual);
    const T *gates = p.gate_rows ? static_cast<const T *>(p.gate) : nullptr;
    const void *columns = p.gate_rows ? nullptr : p.gate;
    int phase = EDGE ? phase_of<V>(p.phase, p.ldx, row) : 0;

    // the weight's windows, the factors', then the stages
    const WeightStage<T, V> weight{stage};
    const FactorStage<V> factor{stage + (p.y ? ITEMS * blockDim.x * 16 : 0)};
    const bool factors = p.post != nullptr || columns != nullptr;
    unsigned char *rows_at = factor.base + (factors ? ITEMS * blockDim.x * V * 4 : 0);
    const int second = residual ? 1 : 0, third = second + (gates ? 1 : 0);   // arrays of a stage
    Ring ring(shared, rows_at, p.stages, third + 1, hidden, phase, blockIdx.x, gridDim.x, p.rows);
    if constexpr (STAGED) {
        ring.src[0] = x;
        ring.ld[0] = p.ldx;
        ring.src[1] = residual ? residual : gates;
        ring.ld[1] = residual ? p.ldr : p.ldg;
        ring.src[2] = gates;
        ring.ld[2] = p.ldg;
        if (threadIdx.x == 0) ring.init();
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 0; i < p.stages; ++i) ring.issue();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {   // a thread reads back what it wrote
            const int e = (int)threadIdx.x * V - phase + i * estep;
            if (p.y) weight.put(i, read_weight<T, V, EDGE>(static_cast<const T *>(p.weight), e, hidden));
            if (factors) {
                float c[V];
                read_factor<T, V, EDGE>(p.post, columns, p.block_scale, e, hidden, c);
                factor.put(i, c);
            }
        }
    }
    const float inv_hidden = 1.f / (float)hidden;
    for (int turn = 0; row < p.rows; row += step, turn ^= 1) {
        if constexpr (EDGE && !STAGED) phase = phase_of<V>(p.phase, p.ldx, row);
        const int e0 = (int)threadIdx.x * V - phase;
        // window i of an operand of this row, which is array `a` of a stage
        auto read = [&](const T *base, size_t ld, int a, int i) {
            if constexpr (STAGED) {
                const int w = (int)threadIdx.x + i * (int)blockDim.x;
                if ((!EDGE || w >= ring.first) && w < ring.first + ring.count) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(ring.at + a * ring.array_bytes + w * 16);
                    Window<T, V> k;
                    k.w[0] = u.x;
                    k.w[1] = u.y;
                    k.w[2] = u.z;
                    k.w[3] = u.w;
                    return k;
                }
            }
            if constexpr (STAGED && !EDGE) {
                Window<T, V> k;
                k.w[0] = k.w[1] = k.w[2] = k.w[3] = 0;
                return k;
            } else {
                return read_window<T, V, EDGE>(base + row * ld, e0 + i * estep, hidden);
            }
        };
        if constexpr (STAGED) ring.wait(p.err);
        float q = 1.f;
        if (p.post) {
            float xx = 0.f;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const Window<T, V> xk = read(x, p.ldx, 0, i);
#pragma unroll
                for (int j = 0; j < V; ++j) xx = fmaf(xk.at(j), xk.at(j), xx);
            }
            q = rsqrtf(mean_of(reduce_row<Sum>(xx, warp_only, sums[0][turn]), (float)hidden, inv_hidden) + p.eps);
        }
        float t[ITEMS][V], tt = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const Window<T, V> xk = read(x, p.ldx, 0, i);
            float c[V];
            if constexpr (!STAGED) {
                read_factor<T, V, EDGE>(p.post, columns, p.block_scale, e0 + i * estep, hidden, c);
            } else if (factors) {
                factor.get(i, c);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) c[j] = p.block_scale;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) t[i][j] = xk.at(j) * q * c[j];
            if (gates) {
                const Window<T, V> gk = read(gates, p.ldg, third, i);
#pragma unroll
                for (int j = 0; j < V; ++j) t[i][j] *= gk.at(j);
            }
            if (residual) {
                const Window<T, V> rk = read(residual, p.ldr, 1, i);
#pragma unroll
                for (int j = 0; j < V; ++j) t[i][j] = fmaf(p.residual_scale, rk.at(j), t[i][j]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) tt = fmaf(t[i][j], t[i][j], tt);
        }
        if (p.total) {
            T *total = static_cast<T *>(p.total) + row * p.ldt;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) write_window<T, V, EDGE>(total, e0 + i * estep, hidden, t[i]);
        }
        if (!p.y) {
            if constexpr (STAGED) {
                __syncthreads();   // every thread has read its share
                if (threadIdx.x == 0) ring.issue();
                ring.next();
            }
            continue;
        }
        const float r =
            rsqrtf(mean_of(reduce_row<Sum>(tt, warp_only, sums[1][turn]), (float)hidden, inv_hidden) + p.eps);
        if constexpr (STAGED)
            if (threadIdx.x == 0) ring.issue();   // the sum's barrier: every thread has read its share
        O *y = static_cast<O *>(p.y) + row * p.ldy;
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            Window<T, V> wk;
            if constexpr (STAGED) wk = weight.get(i);
            else wk = read_weight<T, V, EDGE>(static_cast<const T *>(p.weight), e0 + i * estep, hidden);
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
                fmaxf(reduce_row<Max>(most, warp_only, sums[2][turn]) / kE4m3Max, kScaleMin);
            divide_row(t, scale);
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) write_window<O, V, EDGE>(y, e0 + i * estep, hidden, t[i]);
            if (threadIdx.x == 0) p.scales[row] = scale;
        }
        if constexpr (STAGED) ring.next();
    }
    if constexpr (STAGED)
        if (threadIdx.x == 0) ring.drain(p.err);
}

// ---------------------------------------------------------------- backward --

struct BlockBackwardParams {
    const void *dy, *dtotal, *x, *total, *post, *gate, *weight;
    void *dx, *dresidual, *dgate;   // dgate: rows, or null
    float *partial;                 // gridDim.x rows for dweight, then as many for S
    size_t lddy, lddt, ldx, ldt, ldg, lddx, lddr, lddg, rows;
    uint32_t hidden, phase;
    float block_scale, residual_scale, eps;
    bool gate_rows, sums;           // sums: S is wanted
    int stages;
    unsigned long long *err;
};

template <typename T>
__global__ void __launch_bounds__(1024)
block_norm_backward_long_kernel(const __grid_constant__ BlockBackwardParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be launched
    __shared__ float sums[4][32];
    float *pw = p.partial + (size_t)blockIdx.x * p.hidden;
    float *ps = p.partial + ((size_t)gridDim.x + blockIdx.x) * p.hidden;
    for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
        if (p.weight) pw[e] = 0.f;
        if (p.sums) ps[e] = 0.f;
    }
    const T *post = static_cast<const T *>(p.post), *w = static_cast<const T *>(p.weight);
    for (size_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T *dy = static_cast<const T *>(p.dy) + row * p.lddy;
        const T *total = static_cast<const T *>(p.total) + row * p.ldt;
        const T *x = static_cast<const T *>(p.x) + row * p.ldx;
        const T *dtotal = p.dtotal ? static_cast<const T *>(p.dtotal) + row * p.lddt : nullptr;
        const T *gate = static_cast<const T *>(p.gate);
        if (p.gate_rows) gate += row * p.ldg;
        float xx = 0.f, tt = 0.f, nt = 0.f;
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
            if (post) {
                const float v = to_f32<T>(x[e]);
                xx = fmaf(v, v, xx);
            }
            if (w) {
                const float t = to_f32<T>(total[e]);
                tt = fmaf(t, t, tt);
                nt = fmaf(to_f32<T>(dy[e]) * to_f32<T>(w[e]), t, nt);
            }
        }
        xx = reduce_row<Sum>(xx, false, sums[0]);
        tt = reduce_row<Sum>(tt, false, sums[1]);
        nt = reduce_row<Sum>(nt, false, sums[2]);
        const float q = post ? rsqrtf(xx / (float)p.hidden + p.eps) : 1.f;
        const float r = w ? rsqrtf(tt / (float)p.hidden + p.eps) : 0.f;
        const float c = r * r * (nt / (float)p.hidden);
        auto dt_at = [&](uint32_t e) {
            float d = dtotal ? to_f32<T>(dtotal[e]) : 0.f;
            if (w) d += r * fmaf(to_f32<T>(dy[e]), to_f32<T>(w[e]), -(to_f32<T>(total[e]) * c));
            return d;
        };
        auto factor = [&](uint32_t e) {   // of dt in h
            float f = p.block_scale;
            if (post) f *= to_f32<T>(post[e]);
            if (gate) f *= to_f32<T>(gate[e]);
            return f;
        };
        float k = 0.f;
        if (post) {
            float hx = 0.f;
            for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x)
                hx = fmaf(dt_at(e) * factor(e), to_f32<T>(x[e]), hx);
            k = q * q * (reduce_row<Sum>(hx, false, sums[3]) / (float)p.hidden);
        }
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
            // every input of an element is read before an output, which may be one, is written
            const float dt = dt_at(e), f = factor(e), v = to_f32<T>(x[e]);
            const float g = p.gate_rows ? to_f32<T>(gate[e]) : 1.f;
            const float pe = post ? to_f32<T>(post[e]) : 1.f;
            if (w) pw[e] = fmaf(to_f32<T>(dy[e]), to_f32<T>(total[e]) * r, pw[e]);
            if (p.sums) ps[e] = fmaf(dt * g, v * q, ps[e]);
            const float h = dt * f;
            if (p.dresidual)
                static_cast<T *>(p.dresidual)[row * p.lddr + e] = from_f32<T>(p.residual_scale * dt);
            if (p.dgate)
                static_cast<T *>(p.dgate)[row * p.lddg + e] =
                    from_f32<T>(p.block_scale * dt * (v * q * pe));
            static_cast<T *>(p.dx)[row * p.lddx + e] = from_f32<T>(post ? q * fmaf(-v, k, h) : h);
        }
        __syncthreads();   // before the next row's sums
    }
}

// A thread holds ITEMS windows of V elements of a row's h and x, and the sums over rows
// of its columns.  STAGED and the rest as in the forward kernel: every operand is read
// once for the first sums, and again for dt and h.
template <typename T, int V, int ITEMS, bool EDGE, bool STAGED, int THREADS>
__global__ void __launch_bounds__(THREADS)
block_norm_backward_kernel(const __grid_constant__ BlockBackwardParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be launched
    using Ring = RowRing<T, V, 5>;
    extern __shared__ __align__(128) unsigned char stage[];
    __shared__ typename Ring::Shared shared;
    __shared__ float sums[4][2][32];   // rows take turns
    const bool warp_only = !STAGED && blockDim.x == 32;
    const size_t step = (size_t)gridDim.x * blockDim.y;
    size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int hidden = (int)p.hidden, estep = (int)blockDim.x * V;
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    const T *total = static_cast<const T *>(p.total), *dtotal = static_cast<const T *>(p.dtotal);
    const T *gates = p.gate_rows ? static_cast<const T *>(p.gate) : nullptr;
    const void *columns = p.gate_rows ? nullptr : p.gate;
    const bool normed = p.weight != nullptr, factors = p.post != nullptr || columns != nullptr;
    const int phase = EDGE ? phase_of<V>(p.phase, p.ldx, row) : 0;   // (the grid keeps it)

    const WeightStage<T, V> weight{stage};
    const FactorStage<V> factor{stage + (normed ? ITEMS * blockDim.x * 16 : 0)};
    unsigned char *rows_at = factor.base + (factors ? ITEMS * blockDim.x * V * 4 : 0);
    // arrays of a stage: x, dy, total, then dtotal and gates where there are any
    const int a_dtotal = normed ? 3 : 1, a_gates = a_dtotal + (dtotal ? 1 : 0);
    Ring ring(shared, rows_at, p.stages, a_gates + (gates ? 1 : 0), hidden, phase, blockIdx.x, gridDim.x, p.rows);
    if constexpr (STAGED) {
        const T *from[5] = {x, dy, total, dtotal, gates};
        const size_t pitch[5] = {p.ldx, p.lddy, p.ldt, p.lddt, p.ldg};
        const bool there[5] = {true, normed, normed, dtotal != nullptr, gates != nullptr};
        int n = 0;
#pragma unroll
        for (int a = 0; a < 5; ++a) {
            ring.src[a] = nullptr;
            ring.ld[a] = 0;
        }
#pragma unroll
        for (int a = 0; a < 5; ++a) {
            if (!there[a]) continue;
#pragma unroll
            for (int k = 0; k < 5; ++k)
                if (k == n) {
                    ring.src[k] = from[a];
                    ring.ld[k] = pitch[a];
                }
            ++n;
        }
        if (threadIdx.x == 0) ring.init();
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 0; i < p.stages; ++i) ring.issue();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {   // a thread reads back what it wrote
            const int e = (int)threadIdx.x * V - phase + i * estep;
            if (normed) weight.put(i, read_weight<T, V, EDGE>(static_cast<const T *>(p.weight), e, hidden));
            if (factors) {
                float c[V];
                read_factor<T, V, EDGE>(p.post, columns, p.block_scale, e, hidden, c);
                factor.put(i, c);
            }
        }
    }
    const float inv_hidden = 1.f / (float)hidden;
    const int e0 = (int)threadIdx.x * V - phase;
    float acc_w[ITEMS][V] = {}, acc_s[ITEMS][V] = {};
    for (int turn = 0; row < p.rows; row += step, turn ^= 1) {
        auto read = [&](const T *base, size_t ld, int a, int i) {
            if constexpr (STAGED) {
                const int w = (int)threadIdx.x + i * (int)blockDim.x;
                if ((!EDGE || w >= ring.first) && w < ring.first + ring.count) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(ring.at + a * ring.array_bytes + w * 16);
                    Window<T, V> k;
                    k.w[0] = u.x;
                    k.w[1] = u.y;
                    k.w[2] = u.z;
                    k.w[3] = u.w;
                    return k;
                }
            }
            if constexpr (STAGED && !EDGE) {
                Window<T, V> k;
                k.w[0] = k.w[1] = k.w[2] = k.w[3] = 0;
                return k;
            } else {
                return read_window<T, V, EDGE>(base + row * ld, e0 + i * estep, hidden);
            }
        };
        auto weight_at = [&](int i) {
            if constexpr (STAGED) return weight.get(i);
            else return read_weight<T, V, EDGE>(static_cast<const T *>(p.weight), e0 + i * estep, hidden);
        };
        if constexpr (STAGED) ring.wait(p.err);
        float xx = 0.f, tt = 0.f, nt = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (p.post) {
                const Window<T, V> xk = read(x, p.ldx, 0, i);
#pragma unroll
                for (int j = 0; j < V; ++j) xx = fmaf(xk.at(j), xk.at(j), xx);
            }
            if (normed) {
                const Window<T, V> tk = read(total, p.ldt, 2, i), gk = read(dy, p.lddy, 1, i), wk = weight_at(i);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    tt = fmaf(tk.at(j), tk.at(j), tt);
                    nt = fmaf(gk.at(j) * wk.at(j), tk.at(j), nt);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            xx += __shfl_xor_sync(0xffffffffu, xx, o);
            tt += __shfl_xor_sync(0xffffffffu, tt, o);
            nt += __shfl_xor_sync(0xffffffffu, nt, o);
        }
        if (!warp_only) {
            const int warps = (int)blockDim.x >> 5;
            if ((threadIdx.x & 31) == 0) {
                sums[0][turn][threadIdx.x >> 5] = xx;
                sums[1][turn][threadIdx.x >> 5] = tt;
                sums[2][turn][threadIdx.x >> 5] = nt;
            }
            __syncthreads();
            xx = tt = nt = 0.f;
            for (int k = 0; k < warps; ++k) {
                xx += sums[0][turn][k];
                tt += sums[1][turn][k];
                nt += sums[2][turn][k];
            }
        }
        const float q = p.post ? rsqrtf(mean_of(xx, (float)hidden, inv_hidden) + p.eps) : 1.f;
        const float r = normed ? rsqrtf(mean_of(tt, (float)hidden, inv_hidden) + p.eps) : 0.f;
        const float c = r * r * mean_of(nt, (float)hidden, inv_hidden);
        float h[ITEMS][V], hx = 0.f;
        Window<T, V> xs[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int e = e0 + i * estep;
            float dt[V];
#pragma unroll
            for (int j = 0; j < V; ++j) dt[j] = 0.f;
            if (dtotal) {
                const Window<T, V> dk = read(dtotal, p.lddt, a_dtotal, i);
#pragma unroll
                for (int j = 0; j < V; ++j) dt[j] = dk.at(j);
            }
            xs[i] = read(x, p.ldx, 0, i);
            Window<T, V> kk;
            if (gates) kk = read(gates, p.ldg, a_gates, i);
            if (normed) {
                const Window<T, V> tk = read(total, p.ldt, 2, i), gk = read(dy, p.lddy, 1, i), wk = weight_at(i);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float u = tk.at(j), d = gk.at(j);
                    acc_w[i][j] = fmaf(d, u * r, acc_w[i][j]);
                    dt[j] = fmaf(r, fmaf(d, wk.at(j), -(u * c)), dt[j]);
                }
            }
            // outputs may be inputs: an element's were all read above
            if (p.dresidual) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = p.residual_scale * dt[j];
                write_window<T, V, EDGE>(static_cast<T *>(p.dresidual) + row * p.lddr, e, hidden, o);
            }
            float f[V];
            if constexpr (!STAGED) {
                read_factor<T, V, EDGE>(p.post, columns, p.block_scale, e, hidden, f);
            } else if (factors) {
                factor.get(i, f);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) f[j] = p.block_scale;
            }
            if (p.dgate) {
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = dt[j] * (f[j] * (xs[i].at(j) * q));
                write_window<T, V, EDGE>(static_cast<T *>(p.dgate) + row * p.lddg, e, hidden, o);
            }
            if (gates) {
#pragma unroll
                for (int j = 0; j < V; ++j) dt[j] *= kk.at(j);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                acc_s[i][j] = fmaf(dt[j], xs[i].at(j) * q, acc_s[i][j]);
                h[i][j] = dt[j] * f[j];
                hx = fmaf(h[i][j], xs[i].at(j), hx);
            }
        }
        float k = 0.f;
        if (p.post)
            k = q * q * mean_of(reduce_row<Sum>(hx, warp_only, sums[3][turn]), (float)hidden, inv_hidden);
        else if constexpr (STAGED)
            __syncthreads();
        if constexpr (STAGED) {   // behind the barrier: every thread has read its share
            if (threadIdx.x == 0) ring.issue();
            ring.next();
        }
        T *dx = static_cast<T *>(p.dx) + row * p.lddx;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (p.post) {
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] = q * fmaf(-xs[i].at(j), k, h[i][j]);
            }
            write_window<T, V, EDGE>(dx, e0 + i * estep, hidden, h[i]);
        }
    }
    if constexpr (STAGED)
        if (threadIdx.x == 0) ring.drain(p.err);
    float *pw = p.partial + (size_t)blockIdx.x * hidden;
    float *ps = p.partial + ((size_t)gridDim.x + blockIdx.x) * hidden;
    if (!STAGED && blockDim.y > 1) {   // the warps' sums, warp by warp
        __shared__ float joined[2][STAGED ? 1 : 32 * ITEMS * V];
        for (unsigned y = 0; y < blockDim.y; ++y) {
            if (threadIdx.y == y) {
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const int e = e0 + i * estep + j;
                        if (e >= 0 && e < hidden) {
                            joined[0][e] = y == 0 ? acc_w[i][j] : joined[0][e] + acc_w[i][j];
                            joined[1][e] = y == 0 ? acc_s[i][j] : joined[1][e] + acc_s[i][j];
                        }
                    }
            }
            __syncthreads();
        }
        for (int e = (int)(threadIdx.y * blockDim.x + threadIdx.x); e < hidden; e += (int)(blockDim.x * blockDim.y)) {
            if (normed) pw[e] = joined[0][e];
            if (p.sums) ps[e] = joined[1][e];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = e0 + i * estep + j;
            if (e < 0 || e >= hidden) continue;
            if (normed) pw[e] = acc_w[i][j];
            if (p.sums) ps[e] = acc_s[i][j];
        }
}

constexpr int kJoinRows = 32;

// The blocks' sums, added up in a fixed order: dweight, and from S the gradients of
// the weight after the block and of a column gate.
template <typename T>
__global__ void __launch_bounds__(32 * kJoinRows)
block_join_kernel(const float *partial, const T *post, const T *gate, float block_scale,
                  float *dweight, float *dpost, float *dgate, uint32_t hidden, int parts) {
    __shared__ float sums[kJoinRows][33];
    const uint32_t e = blockIdx.x * 32 + threadIdx.x;
    const bool second = blockIdx.y == (dweight ? 1 : 0);
    if (second) partial += (size_t)parts * hidden;
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
    if (!second) {
        dweight[e] = v;
        return;
    }
    v *= block_scale;
    if (dpost) dpost[e] = gate ? v * to_f32<T>(gate[e]) : v;
    if (dgate) dgate[e] = post ? v * to_f32<T>(post[e]) : v;
}

// Rows on the registers: a warp a row where it holds one, else a block; `most` values
// a thread.  items 0: the row does not fit `threads`.
template <int V>
Shape direct_shape(size_t rows, size_t hidden, int most, unsigned threads, int sms) {
    Shape s;
    const size_t windows = windows_of<V>(hidden, V > 1);
    const int items = std::max(1, most / V);
    // the fewest windows a thread: the quickest for a block's first row, unless there
    // are rows enough to keep every SM busy with warps
    const int least = rows >= 8 * (size_t)sms && windows <= (size_t)32 * items ? items : 1;
    for (int n = least; n <= items; n *= V == 1 ? 4 : 2) {
        const unsigned tx = warps_of(windows, n);
        if (tx > threads) continue;
        s.items = n;
        s.tx = tx;
        break;
    }
    if (s.items == 0) return s;
    s.ty = s.tx == 32 ? 8 : 1;
    s.grid = (unsigned)((rows + s.ty - 1) / s.ty);
    return s;
}

// Rows through shared memory, `arrays` operands a stage and `vector_bytes` a column for
// the vectors beside them.
template <int V>
Shape block_staged_shape(size_t rows, size_t hidden, bool edge, int arrays, size_t vector_bytes, int items,
                         int sms) {
    Shape s;
    constexpr size_t kSmemSm = 227 * 1024, kReserved = 3 * 1024;   // an SM's; a block's own
    const size_t windows = windows_of<V>(hidden, edge);
    const size_t stage = (hidden + 2 * (V - 1)) / V * 16 * (size_t)arrays;   // as RowRing has it
    const unsigned tx = warps_of(windows, items);
    if (V == 1 || windows <= 64 || tx > (unsigned)kStagedThreads || rows < (size_t)sms) return s;
    const size_t vectors = (size_t)items * tx * V * vector_bytes;
    for (size_t b = std::max<size_t>(2, kBlockThreadsSm / tx); b >= 1; --b) {
        if (kSmemSm / b < kReserved + vectors) continue;
        const size_t fit = std::min<size_t>((kSmemSm / b - kReserved - vectors) / stage, kMaxStages);
        if (fit < 2) continue;
        s.items = items;
        s.tx = tx;
        s.stages = (int)std::min(fit, std::max<size_t>(2, kBlockFlight / (b * stage)));
        s.smem = vectors + (size_t)s.stages * stage;
        s.grid = (unsigned)std::min<size_t>(rows, std::max<size_t>((size_t)sms * b / V * V, V));
        break;
    }
    return s;
}

template <typename T, typename O, int V, int ITEMS, bool EDGE>
cudaError_t run_staged(const BlockNormArgs &a, const BlockParams &p, const Shape &s) {
    static SharedMemoryLimit limit;
    const cudaError_t ready = limit.raise(block_norm_kernel<T, O, V, ITEMS, EDGE, true, kStagedThreads>, kStagedSmem);
    if (ready != cudaSuccess) return ready;
    block_norm_kernel<T, O, V, ITEMS, EDGE, true, kStagedThreads><<<s.grid, s.tx, s.smem, a.stream>>>(p);
    return cudaGetLastError();
}

template <typename T, typename O, int V, bool EDGE>
cudaError_t try_staged(const BlockNormArgs &a, BlockParams &p, bool *done) {
    const int arrays = 1 + (a.residual ? 1 : 0) + (a.gate_rows ? 1 : 0);
    const bool factors = a.post_weight || (a.gate && !a.gate_rows);
    const size_t vector_bytes = (a.y ? sizeof(T) : 0) + (factors ? 4 : 0);
    Shape s = block_staged_shape<V>(a.rows, a.hidden, EDGE, arrays, vector_bytes, 4, a.sms);
    *done = s.items != 0;
    p.stages = s.stages;
    if (*done) return run_staged<T, O, V, 4, EDGE>(a, p, s);
    if constexpr (V == 4) {
        s = block_staged_shape<V>(a.rows, a.hidden, EDGE, arrays, vector_bytes, 8, a.sms);
        *done = s.items != 0;
        p.stages = s.stages;
        if (*done) return run_staged<T, O, V, 8, EDGE>(a, p, s);
    }
    return cudaSuccess;
}

template <typename T, typename O, int V>
cudaError_t run_direct(const BlockNormArgs &a, const BlockParams &p) {
    Shape s = direct_shape<V>(a.rows, a.hidden, 16, 512, a.sms);
    const dim3 block(s.tx, s.ty);
    constexpr bool EDGE = V > 1;
    if (s.items == 1) block_norm_kernel<T, O, V, 1, EDGE, false, 512><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == 2) {
        if constexpr (V > 1) block_norm_kernel<T, O, V, 2, EDGE, false, 512><<<s.grid, block, 0, a.stream>>>(p);
    } else if (s.items == 4) {
        if constexpr (V <= 4) block_norm_kernel<T, O, V, 4, EDGE, false, 512><<<s.grid, block, 0, a.stream>>>(p);
    } else if (s.items == 16) {
        if constexpr (V == 1) block_norm_kernel<T, O, V, 16, EDGE, false, 512><<<s.grid, block, 0, a.stream>>>(p);
    } else {
        s = direct_shape<V>(a.rows, a.hidden, 16, 1024, a.sms);
        if (s.items == 16 / V)
            block_norm_kernel<T, O, V, 16 / V, EDGE, false, 1024><<<s.grid, s.tx, 0, a.stream>>>(p);
        else
            block_norm_long_kernel<T, O><<<(unsigned)a.rows, 1024, 0, a.stream>>>(p);
    }
    return cudaGetLastError();
}

template <typename T, typename O>
cudaError_t block_norm_any(const BlockNormArgs &a) {
    constexpr int V = 16 / sizeof(T);
    constexpr size_t es = sizeof(T);
    BlockParams p{a.x, a.post_weight, a.gate, a.residual, a.weight, a.y, a.total, a.scales,
                  a.ldx, a.ldg, a.ldr, a.ldy, a.ldt, a.rows, (uint32_t)a.hidden,
                  (uint32_t)(reinterpret_cast<uintptr_t>(a.x) / es % V),
                  a.block_scale, a.residual_scale, a.eps, a.gate_rows, 0, a.err};
    const bool windows = in_step<V>(a.residual, a.ldr, es, a.x, a.ldx, es) &&
                         in_step<V>(a.gate_rows ? a.gate : nullptr, a.ldg, es, a.x, a.ldx, es) &&
                         in_step<V>(a.total, a.ldt, es, a.x, a.ldx, es) &&
                         in_step<V>(a.y, a.ldy, sizeof(O), a.x, a.ldx, es);
    if (!windows) return run_direct<T, O, 1>(a, p);
    bool done = false;
    bool whole = p.phase == 0 && a.ldx % V == 0 && a.hidden % V == 0;
    for (const void *v : {a.post_weight, a.gate_rows ? nullptr : a.gate, a.weight})
        whole = whole && reinterpret_cast<uintptr_t>(v) % 16 == 0;
    const cudaError_t e = whole ? try_staged<T, O, V, false>(a, p, &done) : try_staged<T, O, V, true>(a, p, &done);
    return done || e != cudaSuccess ? e : run_direct<T, O, V>(a, p);
}

// Whether the sum S over rows is wanted.
bool wants_sums(const BlockNormBackwardArgs &a) {
    return a.post_weight != nullptr || (a.gate != nullptr && !a.gate_rows);
}

// A backward launch: its shape, and whether it takes windows and meets edges.
struct BlockBackwardShape : Shape {
    bool windows = false, edge = false, wide = false;
};

constexpr int kBackwardHeld = 16;   // values of a thread

template <typename T>
BlockBackwardShape block_backward_shape(const BlockNormBackwardArgs &a) {
    constexpr int V = 16 / sizeof(T);
    constexpr size_t es = sizeof(T);
    BlockBackwardShape s;
    const void *gates = a.gate_rows ? a.gate : nullptr, *dgates = a.gate_rows ? a.dgate : nullptr;
    s.windows = in_step<V>(a.dy, a.lddy, es, a.x, a.ldx, es) &&
                in_step<V>(a.total, a.ldt, es, a.x, a.ldx, es) &&
                in_step<V>(a.dtotal, a.lddt, es, a.x, a.ldx, es) &&
                in_step<V>(gates, a.ldg, es, a.x, a.ldx, es) &&
                in_step<V>(a.dx, a.lddx, es, a.x, a.ldx, es) &&
                in_step<V>(a.dresidual, a.lddr, es, a.x, a.ldx, es) &&
                in_step<V>(dgates, a.lddg, es, a.x, a.ldx, es);
    s.edge = !(reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx % V == 0 && a.hidden % V == 0);
    for (const void *v : {a.post_weight, a.gate_rows ? nullptr : a.gate, a.weight})
        s.edge = s.edge || reinterpret_cast<uintptr_t>(v) % 16 != 0;
    Shape &base = s;
    if (s.windows) {
        const int arrays = 1 + (a.weight ? 2 : 0) + (a.dtotal ? 1 : 0) + (gates ? 1 : 0);
        const bool factors = a.post_weight || (a.gate && !a.gate_rows);
        base = block_staged_shape<V>(a.rows, a.hidden, s.edge, arrays, (a.weight ? es : 0) + (factors ? 4 : 0),
                                     kBackwardHeld / V, a.sms);
        if (s.items != 0) return s;
    }
    for (unsigned threads : {512u, 1024u}) {
        base = s.windows ? direct_shape<V>(a.rows, a.hidden, kBackwardHeld, threads, a.sms)
                         : direct_shape<1>(a.rows, a.hidden, kBackwardHeld, threads, a.sms);
        s.wide = threads > 512;
        if (s.items != 0) break;
    }
    if (s.items == 0) {   // the long kernel
        s.grid = (unsigned)std::min<size_t>(a.rows, (size_t)a.sms * 2);
        return s;
    }
    // blocks that fit at once, a multiple of the windows' elements so that a block's rows
    // share their phase, or a row a block
    if (s.ty > 1) s.ty = 4;
    const size_t fit = std::max<size_t>(1, kBackwardThreadsSmDirect / (s.tx * s.ty));
    const size_t grid = std::max<size_t>((size_t)a.sms * fit / V * V, V);
    s.grid = (unsigned)std::min<size_t>((a.rows + s.ty - 1) / s.ty, grid);
    return s;
}

template <typename T, int V, bool EDGE>
cudaError_t backward_staged(const BlockNormBackwardArgs &a, const BlockBackwardParams &p, const Shape &s) {
    static SharedMemoryLimit limit;
    constexpr int ITEMS = kBackwardHeld / V;
    const cudaError_t ready =
        limit.raise(block_norm_backward_kernel<T, V, ITEMS, EDGE, true, kStagedThreads>, kStagedSmem);
    if (ready != cudaSuccess) return ready;
    block_norm_backward_kernel<T, V, ITEMS, EDGE, true, kStagedThreads><<<s.grid, s.tx, s.smem, a.stream>>>(p);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t backward_direct(const BlockNormBackwardArgs &a, const BlockBackwardParams &p,
                            const BlockBackwardShape &s) {
    constexpr bool EDGE = V > 1;
    constexpr int MOST = kBackwardHeld / V;
    const dim3 block(s.tx, s.ty);
    if (s.items == 0) block_norm_backward_long_kernel<T><<<s.grid, 1024, 0, a.stream>>>(p);
    else if (s.wide) block_norm_backward_kernel<T, V, MOST, EDGE, false, 1024><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == 1) block_norm_backward_kernel<T, V, 1, EDGE, false, 512><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == MOST) block_norm_backward_kernel<T, V, MOST, EDGE, false, 512><<<s.grid, block, 0, a.stream>>>(p);
    else if constexpr (V == 4) block_norm_backward_kernel<T, V, 2, EDGE, false, 512><<<s.grid, block, 0, a.stream>>>(p);
    else if constexpr (V == 1) block_norm_backward_kernel<T, V, 4, EDGE, false, 512><<<s.grid, block, 0, a.stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t block_norm_backward_any(const BlockNormBackwardArgs &a) {
    constexpr int V = 16 / sizeof(T);
    const bool sums = wants_sums(a);
    const BlockBackwardShape s = block_backward_shape<T>(a);
    const BlockBackwardParams p{a.dy, a.dtotal, a.x, a.total, a.post_weight, a.gate, a.weight,
                                a.dx, a.dresidual, a.gate_rows ? a.dgate : nullptr, a.partial,
                                a.lddy, a.lddt, a.ldx, a.ldt, a.ldg, a.lddx, a.lddr, a.lddg, a.rows,
                                (uint32_t)a.hidden,
                                (uint32_t)(reinterpret_cast<uintptr_t>(a.x) / sizeof(T) % V),
                                a.block_scale, a.residual_scale, a.eps, a.gate_rows, sums, s.stages,
                                a.err};
    const cudaError_t e = s.stages > 0 ? s.edge ? backward_staged<T, V, true>(a, p, s)
                                                : backward_staged<T, V, false>(a, p, s)
                          : s.windows ? backward_direct<T, V>(a, p, s)
                                      : backward_direct<T, 1>(a, p, s);
    const unsigned vectors = (a.weight ? 1 : 0) + (sums ? 1 : 0);
    if (e != cudaSuccess || vectors == 0) return e;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)((a.hidden + 31) / 32), vectors);
    c.blockDim = dim3(32, kJoinRows);
    c.stream = a.stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, block_join_kernel<T>, (const float *)a.partial,
                              static_cast<const T *>(a.post_weight),
                              a.gate_rows ? (const T *)nullptr : static_cast<const T *>(a.gate),
                              a.block_scale, a.dweight, a.dpost_weight,
                              a.gate_rows ? (float *)nullptr : static_cast<float *>(a.dgate),
                              (uint32_t)a.hidden, (int)s.grid);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs &a) {
    if (a.dtype == PURLIN_F32)
        return a.out_dtype == PURLIN_E4M3 ? block_norm_any<float, __nv_fp8_e4m3>(a)
                                          : block_norm_any<float, float>(a);
    return a.out_dtype == PURLIN_E4M3 ? block_norm_any<__nv_bfloat16, __nv_fp8_e4m3>(a)
                                      : block_norm_any<__nv_bfloat16, __nv_bfloat16>(a);
}

size_t block_norm_backward_workspace(const BlockNormBackwardArgs &a) {
    if (a.weight == nullptr && !wants_sums(a)) return 0;
    const Shape s = a.dtype == PURLIN_F32 ? block_backward_shape<float>(a)
                                          : block_backward_shape<__nv_bfloat16>(a);
    return 2 * (size_t)s.grid * a.hidden * sizeof(float);
}

cudaError_t launch_block_norm_backward(const BlockNormBackwardArgs &a) {
    return a.dtype == PURLIN_F32 ? block_norm_backward_any<float>(a)
                                 : block_norm_backward_any<__nv_bfloat16>(a);
}

}  // namespace purlin
