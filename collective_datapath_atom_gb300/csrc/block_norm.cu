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

template <typename T, typename O>
cudaError_t block_norm_any(const BlockNormArgs &a) {
    BlockParams p{a.x, a.post_weight, a.gate, a.residual, a.weight, a.y, a.total, a.scales,
                  a.ldx, a.ldg, a.ldr, a.ldy, a.ldt, a.rows, (uint32_t)a.hidden, 0,
                  a.block_scale, a.residual_scale, a.eps, a.gate_rows, 0, a.err};
    block_norm_long_kernel<T, O><<<(unsigned)a.rows, 1024, 0, a.stream>>>(p);
    return cudaGetLastError();
}

unsigned backward_grid(const BlockNormBackwardArgs &a) {
    return (unsigned)std::min<size_t>(a.rows, (size_t)a.sms * 2);
}

// Whether the sum S over rows is wanted.
bool wants_sums(const BlockNormBackwardArgs &a) {
    return a.post_weight != nullptr || (a.gate != nullptr && !a.gate_rows);
}

template <typename T>
cudaError_t block_norm_backward_any(const BlockNormBackwardArgs &a) {
    const bool sums = wants_sums(a);
    const unsigned grid = backward_grid(a);
    BlockBackwardParams p{a.dy, a.dtotal, a.x, a.total, a.post_weight, a.gate, a.weight,
                          a.dx, a.dresidual, a.gate_rows ? a.dgate : nullptr, a.partial,
                          a.lddy, a.lddt, a.ldx, a.ldt, a.ldg, a.lddx, a.lddr, a.lddg, a.rows,
                          (uint32_t)a.hidden, 0, a.block_scale, a.residual_scale, a.eps,
                          a.gate_rows, sums, 0, a.err};
    block_norm_backward_long_kernel<T><<<grid, 1024, 0, a.stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    const unsigned vectors = (a.weight ? 1 : 0) + (sums ? 1 : 0);
    if (e != cudaSuccess || vectors == 0) return e;
    block_join_kernel<T><<<dim3((unsigned)((a.hidden + 31) / 32), vectors), dim3(32, kJoinRows), 0, a.stream>>>(
        a.partial, static_cast<const T *>(a.post_weight),
        a.gate_rows ? nullptr : static_cast<const T *>(a.gate), a.block_scale, a.dweight,
        a.dpost_weight, a.gate_rows ? nullptr : static_cast<float *>(a.dgate), (uint32_t)a.hidden,
        (int)grid);
    return cudaGetLastError();
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
    return a.weight != nullptr || wants_sums(a) ? 2 * (size_t)backward_grid(a) * a.hidden * sizeof(float) : 0;
}

cudaError_t launch_block_norm_backward(const BlockNormBackwardArgs &a) {
    return a.dtype == PURLIN_F32 ? block_norm_backward_any<float>(a)
                                 : block_norm_backward_any<__nv_bfloat16>(a);
}

}  // namespace purlin
