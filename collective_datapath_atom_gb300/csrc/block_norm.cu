// block_norm.cu -- the norms after and before a block, with the block's gate and the
// residual's addition between them.  A row at a time, in binary32, with
// c = block_scale * post_weight * gate:
//   q = 1 / sqrt(mean(x^2) + eps),  t = residual_scale * residual + c x q,
//   r = 1 / sqrt(mean(t^2) + eps),  y = t r weight.
// t is rounded where it is stored alone; y is of the unrounded t.  Means are quotients
// by the hidden size (mean_of), and the products above are taken in that order, in every
// kernel: a row is the same among few rows and many but for the order of its sums.
//
// Bound by bytes: every operand is read once and every result written once.  Two sums over
// the row stand between the loads and the last store, so rows are many at a time on an SM:
// persistent blocks of teams of warps, a team a row, with rings of rows that bulk copies
// fill (16384 x 7168 bf16 with the residual to e4m3 133 us, 6.2 TB/s; 16384 x 4096 bf16 99
// us, 5.4 TB/s; two blocks an SM with a ring each 170).  Few rows, and rows whose operands
// are out of step, have a block each, and registers (1 x 4096: the launch); rows that fit
// neither are read again, element by element.
#include "block_rows.cuh"

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
    const float n = (float)p.hidden, inv = 1.f / n;
    float q = 1.f;
    if (post) {
        float xx = 0.f;
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
            const float v = to_f32<T>(x[e]);
            xx = fmaf(v, v, xx);
        }
        q = rsqrtf(mean_of(reduce_row<Sum>(xx, false, sums[0]), n, inv) + p.eps);
    }
    auto at = [&](uint32_t e) {
        float c = p.block_scale;
        if (post) c *= to_f32<T>(post[e]);
        if (gate) c *= to_f32<T>(gate[e]);
        const float u = c * (to_f32<T>(x[e]) * q);
        return res ? fmaf(p.residual_scale, to_f32<T>(res[e]), u) : u;
    };
    float r = 0.f, scale = 1.f;
    if (p.y) {
        float tt = 0.f;
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
            const float t = at(e);
            tt = fmaf(t, t, tt);
        }
        r = rsqrtf(mean_of(reduce_row<Sum>(tt, false, sums[1]), n, inv) + p.eps);
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

// Rows on the registers, for few of them: a thread holds ITEMS windows of V elements of
// its row's t; a block a row, or a warp (then blockDim.y rows a block).
template <typename T, typename O, int V, int ITEMS, bool EDGE, int THREADS>
__global__ void __launch_bounds__(THREADS)
block_norm_kernel(const __grid_constant__ BlockParams p) {
    __shared__ float sums[3][32];
    const bool warp_only = blockDim.x == 32;
    const size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= p.rows) return;   // whole warps; blockDim.y > 1 has no block barrier
    const int hidden = (int)p.hidden, estep = (int)blockDim.x * V;
    const int e0 = (int)threadIdx.x * V - (EDGE ? phase_of<V>(p.phase, p.ldx, row) : 0);
    const float n = (float)hidden, inv = 1.f / n;
    Window<T, V> xk[ITEMS];
    float t[ITEMS][V];
    float xx = 0.f, tt = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        xk[i] = read_window<T, V, EDGE>(static_cast<const T *>(p.x) + row * p.ldx, e0 + i * estep, hidden);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {   // the factors, while x is on its way
        read_factor<T, V, EDGE>(p.post, p.gate_rows ? nullptr : p.gate, p.block_scale, e0 + i * estep, hidden, t[i]);
        if (p.gate_rows) {
            const Window<T, V> gk = read_window<T, V, EDGE>(static_cast<const T *>(p.gate) + row * p.ldg,
                                                            e0 + i * estep, hidden);
#pragma unroll
            for (int j = 0; j < V; ++j) t[i][j] *= gk.at(j);
        }
    }
    float q = 1.f;
    if (p.post) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) xx = fmaf(xk[i].at(j), xk[i].at(j), xx);
        q = rsqrtf(mean_of(reduce_row<Sum>(xx, warp_only, sums[0]), n, inv) + p.eps);
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) t[i][j] *= xk[i].at(j) * q;
        if (p.residual) {
            const Window<T, V> rk = read_window<T, V, EDGE>(static_cast<const T *>(p.residual) + row * p.ldr,
                                                            e0 + i * estep, hidden);
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
    if (!p.y) return;
    const float r = rsqrtf(mean_of(reduce_row<Sum>(tt, warp_only, sums[1]), n, inv) + p.eps);
    O *y = static_cast<O *>(p.y) + row * p.ldy;
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const Window<T, V> wk = read_weight<T, V, EDGE>(static_cast<const T *>(p.weight), e0 + i * estep, hidden);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            t[i][j] = t[i][j] * r * wk.at(j);
            most = fmaxf(most, fabsf(t[i][j]));
        }
        if constexpr (sizeof(O) != 1) write_window<O, V, EDGE>(y, e0 + i * estep, hidden, t[i]);
    }
    if constexpr (sizeof(O) == 1) {
        // fmaxf passes over NaN: the scale stays a number, the elements are NaN
        const float scale = fmaxf(reduce_row<Max>(most, warp_only, sums[2]) / kE4m3Max, kScaleMin);
        divide_row(t, scale);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) write_window<O, V, EDGE>(y, e0 + i * estep, hidden, t[i]);
        if (threadIdx.x == 0) p.scales[row] = scale;
    }
}

// A thread holds ITEMS windows of its row's t, made behind the first sum's barrier from
// operands that it reads from the stage again.  Holding those, which frees the stage a
// barrier earlier, needs 128 registers, and three teams of seven warps are worth more
// than early loads (16384 x 7168 bf16 to e4m3 140 us, two teams that hold them 153).
// With 16 / 21 / 24 warps of a block at most (us, 8192 rows, 16384 of 7168 columns; of 24 a
// thread has fewer registers):
//   bf16 to e4m3: 4096 50 / 49 / 50, 5120 58 / 58 / 62, 6144 74 / 66 / 70, 7168 138 / 133 / 139,
//   8192 86 / 90 / 96;  bf16: 4096 54 / 53 / 52, 6144 76 / 74 / 73;  f32: 4096 89 / 100 / 89,
//   5120 119 / 125 / 122;  f32 to e4m3: 5120 122 / 98 / 93, 6144 130 / 121 / 128.
constexpr int kForwardWarps = 21;

// Operands of the rows, in the order of their arrays in a stage: x, the gates where
// there are any, and the residual.
struct TeamParams : BlockParams {
    const void *src[3];
    size_t ld[3];
};

template <typename T, typename O, int V, int ITEMS, bool EDGE, bool GATES>
__global__ void __launch_bounds__(32 * kForwardWarps)
block_norm_team_kernel(const __grid_constant__ TeamParams p, const __grid_constant__ TeamPlan plan) {
    __shared__ uint64_t full[kForwardWarps][kMaxStages];
    __shared__ __align__(16) float sums[3][2][kTeams][kTeamWarps];   // rows take turns; single warps have none
    const Team team(plan.warps);
    const int hidden = (int)p.hidden, phase = EDGE ? phase_of<V>(p.phase, p.ldx, blockIdx.x) : 0;
    const Vectors<T, V, ITEMS, EDGE> vectors(plan, p.weight, p.post, GATES ? nullptr : p.gate, p.block_scale,
                                             hidden, phase, team);
    const size_t row0 = blockIdx.x + (size_t)team.index * gridDim.x;
    const size_t step = (size_t)(blockDim.x / team.threads()) * gridDim.x;
    TeamRing<T, V, 3, ITEMS, EDGE, TeamParams> ring(p, plan, team, full[team.index], vectors.end, phase, hidden, row0, step);
    constexpr int kResidual = GATES ? 2 : 1;
    const int slot = team.warps == 1 ? 0 : team.index;
    for (int i = threadIdx.x; i < (int)(sizeof(sums) / sizeof(float)); i += (int)blockDim.x) (&sums[0][0][0][0])[i] = 0.f;
    ring.clear();
    team.sync();
    ring.start();
    vectors.start();
    __syncthreads();
    const float n = (float)hidden, inv_hidden = 1.f / n;
    int turn = 0;
    for (size_t row = row0; row < p.rows; row += step, turn ^= 1) {
        ring.wait();
        F2 xx = 0, tt = 0;
        float q = 1.f;
        if (p.post) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const Window<T, V> xk = ring.window(0, i);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) xx = fma2(pair_of(xk, j), pair_of(xk, j), xx);
            }
            const float sum = team.template total<Sum>(low(xx) + high(xx), sums[0][turn][slot]);
            q = rsqrtf(mean_of(sum, n, inv_hidden) + p.eps);
        }
        F2 t[ITEMS][V / 2];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            F2 c[V / 2];
            vectors.factor(i, c);
            if constexpr (GATES) {
                const Window<T, V> gk = ring.window(1, i);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) c[j] = mul2(c[j], pair_of(gk, j));
            }
            const Window<T, V> xk = ring.window(0, i);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) t[i][j] = mul2(mul2(pair_of(xk, j), both(q)), c[j]);
            if (p.residual) {
                const Window<T, V> rk = ring.window(kResidual, i);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) t[i][j] = fma2(both(p.residual_scale), pair_of(rk, j), t[i][j]);
            }
#pragma unroll
            for (int j = 0; j < V / 2; ++j) tt = fma2(t[i][j], t[i][j], tt);
        }
        if (p.total) {
            T *total = static_cast<T *>(p.total) + row * p.ldt;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) write_pairs<T, V, EDGE>(total, vectors.column(i), hidden, t[i]);
        }
        ring.settle();   // the row before's refill, before a barrier
        // behind one, the stage is free for another row
        if (!p.y) {
            team.sync();
            ring.refill();
        } else {
            const float sum = team.template total<Sum>(low(tt) + high(tt), sums[1][turn][slot]);
            const float r = rsqrtf(mean_of(sum, n, inv_hidden) + p.eps);
            if (team.warps == 1) __syncwarp();
            ring.refill();
            O *y = static_cast<O *>(p.y) + row * p.ldy;
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const Window<T, V> wk = vectors.weights(i);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    t[i][j] = mul2(mul2(t[i][j], both(r)), pair_of(wk, j));
                    if constexpr (sizeof(O) == 1) most = fmaxf(fmaxf(most, fabsf(low(t[i][j]))), fabsf(high(t[i][j])));
                }
                if constexpr (sizeof(O) != 1) write_pairs<O, V, EDGE>(y, vectors.column(i), hidden, t[i]);
            }
            if constexpr (sizeof(O) == 1) {
                // fmaxf passes over NaN: the scale stays a number, the elements are NaN
                float scale = fmaxf(team.template total<Max>(most, sums[2][turn][slot]) / kE4m3Max, kScaleMin);
                if (team.thread == 0) p.scales[row] = scale;
                // the binary32 quotients, as divide_row has them
                if (scale < 0x1p-80f) {   // remainders would fall below the smallest value
                    scale *= 0x1p64f;
#pragma unroll
                    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
                        for (int j = 0; j < V / 2; ++j) t[i][j] = mul2(t[i][j], both(0x1p64f));
                }
                const float inv = 1.f / scale, d = scale <= kF32Max ? scale : 0.f;
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) {
                        const F2 first = mul2(t[i][j], both(inv));
                        t[i][j] = fma2(fma2(first, both(-d), t[i][j]), both(inv), first);
                    }
                    write_pairs<O, V, EDGE>(y, vectors.column(i), hidden, t[i]);
                }
            }
        }
        if (EDGE && plan.stages == 1) {   // the next row's ends are read at once
            ring.settle();
            team.sync();
        }
        ring.next();
    }
    if (team.thread == 0) ring.drain();
}

template <typename T, typename O, int V, int ITEMS, bool EDGE, bool GATES>
cudaError_t run_teams(const BlockNormArgs &a, const TeamParams &p, const TeamShape &s) {
    static SharedMemoryLimit limit;
    const cudaError_t ready = limit.raise(block_norm_team_kernel<T, O, V, ITEMS, EDGE, GATES>, kTeamSmem);
    if (ready != cudaSuccess) return ready;
    block_norm_team_kernel<T, O, V, ITEMS, EDGE, GATES><<<s.grid, s.threads, s.smem, a.stream>>>(p, s.plan);
    return cudaGetLastError();
}

// `done`: whether the rows took the teams' kernel.
template <typename T, typename O, int V, bool EDGE, bool GATES>
cudaError_t try_teams(const BlockNormArgs &a, const BlockParams &b, bool *done) {
    TeamParams p{b, {a.x, GATES ? a.gate : a.residual, a.residual}, {a.ldx, GATES ? a.ldg : a.ldr, a.ldr}};
    const int arrays = 1 + (a.residual ? 1 : 0) + (GATES ? 1 : 0);
    const bool factors = a.post_weight || (a.gate && !GATES);
    // Warps that the arithmetic wants: the maximum and the quotients of e4m3 all of them
    // (8192 x 4096 bf16 to e4m3 49 us, with 12 55; 6144 66 and 78), rows of f32, of which
    // fewer are as many bytes, the fewest (4096 100 us with 8, 12 or 21); bf16 4096 53 with 12
    // or 8, 57 with 21, 6144 74 and 80, 8192 104, 107 with 8, 5120 68, 64 with 8.
    const auto shape = [&](int items) {
        const TeamShape s =
            team_shape<V>(a.rows, a.hidden, EDGE, arrays, a.y != nullptr, factors, items, false, false,
                          kForwardWarps, sizeof(O) == 1 ? kForwardWarps : sizeof(T) == 2 ? 12 : 8, a.sms);
        *done = s.plan.warps != 0;
        return s;
    };
    // one warp of half the windows for short rows, then 32 values a thread, held as f32
    constexpr int kLeast = V == 8 ? 2 : 4;
    TeamShape s;
    if (windows_of<V>(a.hidden, EDGE) <= 32 * kLeast) {
        s = shape(kLeast);
        if (*done) return run_teams<T, O, V, kLeast, EDGE, GATES>(a, p, s);
    }
    s = shape(4);
    if (*done) return run_teams<T, O, V, 4, EDGE, GATES>(a, p, s);
    if constexpr (V == 4) {
        s = shape(8);
        if (*done) return run_teams<T, O, V, 8, EDGE, GATES>(a, p, s);
    }
    return cudaSuccess;
}

template <typename T, typename O, int V>
cudaError_t run_direct(const BlockNormArgs &a, const BlockParams &p, bool edge) {
    Shape s = direct_shape<V>(a.rows, a.hidden, edge, 16, 512, a.sms);
    const dim3 block(s.tx, s.ty);
    constexpr bool EDGE = V > 1;
    if (s.items == 1) block_norm_kernel<T, O, V, 1, EDGE, 512><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == 2) {
        if constexpr (V > 1) block_norm_kernel<T, O, V, 2, EDGE, 512><<<s.grid, block, 0, a.stream>>>(p);
    } else if (s.items == 4) {
        if constexpr (V <= 4) block_norm_kernel<T, O, V, 4, EDGE, 512><<<s.grid, block, 0, a.stream>>>(p);
    } else if (s.items == 16) {
        if constexpr (V == 1) block_norm_kernel<T, O, V, 16, EDGE, 512><<<s.grid, block, 0, a.stream>>>(p);
    } else {
        s = direct_shape<V>(a.rows, a.hidden, edge, 16, 1024, a.sms);
        if (s.items == 16 / V)
            block_norm_kernel<T, O, V, 16 / V, EDGE, 1024><<<s.grid, s.tx, 0, a.stream>>>(p);
        else
            block_norm_long_kernel<T, O><<<(unsigned)a.rows, 1024, 0, a.stream>>>(p);
    }
    return cudaGetLastError();
}

template <typename T, typename O>
cudaError_t block_norm_any(const BlockNormArgs &a) {
    constexpr int V = 16 / sizeof(T);
    constexpr size_t es = sizeof(T);
    const BlockParams p{a.x, a.post_weight, a.gate, a.residual, a.weight, a.y, a.total, a.scales,
                        a.ldx, a.ldg, a.ldr, a.ldy, a.ldt, a.rows, (uint32_t)a.hidden,
                        (uint32_t)(reinterpret_cast<uintptr_t>(a.x) / es % V),
                        a.block_scale, a.residual_scale, a.eps, a.gate_rows, a.err};
    const bool windows = in_step<V>(a.residual, a.ldr, es, a.x, a.ldx, es) &&
                         in_step<V>(a.gate_rows ? a.gate : nullptr, a.ldg, es, a.x, a.ldx, es) &&
                         in_step<V>(a.total, a.ldt, es, a.x, a.ldx, es) &&
                         in_step<V>(a.y, a.ldy, sizeof(O), a.x, a.ldx, es);
    if (!windows) return run_direct<T, O, 1>(a, p, false);
    const bool edge = p.phase != 0 || a.ldx % V != 0 || a.hidden % V != 0;
    bool vectors = true;   // on 16-byte boundaries
    for (const void *v : {a.post_weight, a.gate_rows ? nullptr : a.gate, a.weight})
        vectors = vectors && reinterpret_cast<uintptr_t>(v) % 16 == 0;
    bool done = false;
    const cudaError_t e = a.gate_rows
                              ? !edge && vectors ? try_teams<T, O, V, false, true>(a, p, &done)
                                                 : try_teams<T, O, V, true, true>(a, p, &done)
                              : !edge && vectors ? try_teams<T, O, V, false, false>(a, p, &done)
                                                 : try_teams<T, O, V, true, false>(a, p, &done);
    return done || e != cudaSuccess ? e : run_direct<T, O, V>(a, p, edge);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs &a) {
    if (a.dtype == PURLIN_F32)
        return a.out_dtype == PURLIN_E4M3 ? block_norm_any<float, __nv_fp8_e4m3>(a)
                                          : block_norm_any<float, float>(a);
    return a.out_dtype == PURLIN_E4M3 ? block_norm_any<__nv_bfloat16, __nv_fp8_e4m3>(a)
                                      : block_norm_any<__nv_bfloat16, __nv_bfloat16>(a);
}

}  // namespace purlin
