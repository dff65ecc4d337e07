// block_norm_backward.cu -- gradients of the norms around a block (block_norm.cu), with
// n = dy weight and c = block_scale * post_weight * gate:
//   dt = r (n - t r^2 mean(n t)) + dtotal,  h = c dt,  dx = q (h - x q^2 mean(h x)).
// The powers of r are taken one at a time: t r and r mean(n t), of the sizes of 1 and of
// n.  r^2 or r^3 by themselves leave binary32 where dt does not (r^3 for rows of 1e13 on,
// or of 1e-13 without an eps).
// The sums over rows are  dweight = sum dy t r,  S = sum dt x q (gate):  of a column
// gate and the weight after the block, dgate = block_scale post_weight S and
// dpost_weight = block_scale gate S.  A thread owns the same columns in every row, so its
// shares of the two sums stay in registers, are written once a block, 16 bytes at a time
// (1 x 16384 bf16 21 us; element by element, eight apart in a warp, 35), and added up over
// the blocks in a fixed order by a second kernel: no atomics, the same bits every time.
//
// Bound by bytes where rows are many (32768 x 4096 bf16 with dtotal 260 us, 6.2 TB/s), by
// the two chains of sums of a row where they are few.  Of rows above 8192 bf16 or 4096 f32
// columns an SM has one at a time: two windows a thread would take more than sixteen warps,
// so nine do the row with four, which hold none of its operands (1000 x 4099 f32 with a gate
// a row 50 us, 4096 columns, sixteen warps that hold them, 33; 4000 x 8200 bf16 142), and of
// the widest the columns' sums take most of the registers (4000 x 16384 306, 2.6 TB/s).
#include "block_rows.cuh"

namespace purlin {
namespace {

// Warps of a block of teams, with two windows a thread; or fewer, with four and with all
// the registers there are, so that what is done once a row and thread is half as much (as
// compared: 32768 x 4096 bf16 261 us, else 274; 16384 x 7168 257 and 295; 8000 x 4096 f32 128 and
// 134). That needs rows of four warps or more (20000 x 2048, two of them, 114 and 109),
// teams that leave one warp idle at most (8000 x 2560 f32, three idle, 115 and 97) and
// rows enough for its slower first and last ones (2000 x 4096 35 and 33, 500 rows 19 and 17).
constexpr int kBackwardWarps = 16, kFewWarps = 8;
// Rows on the registers, threads an SM: more of them share out what is one row after
// another, and leave more sums to join (512, 256 and 1024: 8000 x 4096 bf16 out of step 547,
// 965 and 559 us; without the second norm 8000 x 512 27, 31 and 35, 2000 x 2048 25, 36 and 29;
// 2000 x 1024 out of step 37, 57 and 29).
constexpr size_t kDirectThreadsSm = 512;

struct BlockBackwardParams {
    const void *dy, *dtotal, *x, *total, *post, *gate, *weight;
    void *dx, *dresidual, *dgate;   // dgate: rows, or null
    float *partial;                 // gridDim.x rows for dweight, then as many for S
    uint32_t pitch;                 // of those rows, which start a block's phase early
    size_t lddy, lddt, ldx, ldt, ldg, lddx, lddr, lddg, rows;
    uint32_t hidden, phase;
    float block_scale, residual_scale, eps;
    bool gate_rows, sums;           // sums: S is wanted
    unsigned long long *err;
};

// A window's sums over rows to their place, on 16-byte boundaries where V is above 1.
template <int V>
__device__ __forceinline__ void write_sums(float *to, const float (&v)[V]) {
    if constexpr (V == 1) {
        *to = v[0];
    } else {
#pragma unroll
        for (int n = 0; n < V / 4; ++n)
            reinterpret_cast<float4 *>(to)[n] = make_float4(v[4 * n], v[4 * n + 1], v[4 * n + 2], v[4 * n + 3]);
    }
}

template <typename T>
__global__ void __launch_bounds__(1024)
block_norm_backward_long_kernel(const __grid_constant__ BlockBackwardParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be launched
    __shared__ float sums[4][32];
    float *pw = p.partial + (size_t)blockIdx.x * p.pitch;
    float *ps = pw + (size_t)gridDim.x * p.pitch;
    for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
        if (p.weight) pw[e] = 0.f;
        if (p.sums) ps[e] = 0.f;
    }
    const T *post = static_cast<const T *>(p.post), *w = static_cast<const T *>(p.weight);
    const float columns = (float)p.hidden, inv_hidden = 1.f / columns;
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
        const float q = post ? rsqrtf(mean_of(xx, columns, inv_hidden) + p.eps) : 1.f;
        const float r = w ? rsqrtf(mean_of(tt, columns, inv_hidden) + p.eps) : 0.f;
        const float m = r * mean_of(nt, columns, inv_hidden);
        auto dt_at = [&](uint32_t e) {
            float d = dtotal ? to_f32<T>(dtotal[e]) : 0.f;
            if (w) d = fmaf(r, fmaf(-(to_f32<T>(total[e]) * r), m, to_f32<T>(dy[e]) * to_f32<T>(w[e])), d);
            return d;
        };
        auto gate_at = [&](uint32_t e) { return p.gate_rows ? to_f32<T>(gate[e]) : 1.f; };
        auto factor = [&](uint32_t e) {   // of dt and a row's gate in h
            float f = p.block_scale;
            if (post) f *= to_f32<T>(post[e]);
            if (gate && !p.gate_rows) f *= to_f32<T>(gate[e]);
            return f;
        };
        float k = 0.f;
        if (post) {
            float hx = 0.f;
            for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x)
                hx = fmaf(dt_at(e) * gate_at(e) * factor(e), to_f32<T>(x[e]), hx);
            k = q * (q * mean_of(reduce_row<Sum>(hx, false, sums[3]), columns, inv_hidden));
        }
        for (uint32_t e = threadIdx.x; e < p.hidden; e += blockDim.x) {
            // every input of an element is read before an output, which may be one, is written
            const float dt = dt_at(e), f = factor(e), g = gate_at(e), v = to_f32<T>(x[e]);
            if (w) pw[e] = fmaf(to_f32<T>(dy[e]), to_f32<T>(total[e]) * r, pw[e]);
            if (p.sums) ps[e] = fmaf(dt * g, v * q, ps[e]);
            const float h = dt * g * f;
            if (p.dresidual)
                static_cast<T *>(p.dresidual)[row * p.lddr + e] = from_f32<T>(p.residual_scale * dt);
            if (p.dgate)
                static_cast<T *>(p.dgate)[row * p.lddg + e] = from_f32<T>(dt * (f * (v * q)));
            static_cast<T *>(p.dx)[row * p.lddx + e] = from_f32<T>(post ? q * fmaf(-v, k, h) : h);
        }
        __syncthreads();   // before the next row's sums
    }
}

// Rows on the registers, for few of them: a thread holds ITEMS windows of V elements of
// a row's h and x, and the sums over rows of its columns.  The operands are read for the
// first sums, and again, from the caches, for dt and h.
template <typename T, int V, int ITEMS, bool EDGE, int THREADS>
__global__ void __launch_bounds__(THREADS)
block_norm_backward_kernel(const __grid_constant__ BlockBackwardParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be launched
    __shared__ float sums[4][2][32];   // rows take turns
    __shared__ float joined[2][32 * ITEMS * V];
    const bool warp_only = blockDim.x == 32;
    const size_t step = (size_t)gridDim.x * blockDim.y;
    size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
    const int hidden = (int)p.hidden, estep = (int)blockDim.x * V;
    const T *gates = p.gate_rows ? static_cast<const T *>(p.gate) : nullptr;
    const bool normed = p.weight != nullptr;
    const int e0 = (int)threadIdx.x * V - (EDGE ? phase_of<V>(p.phase, p.ldx, row) : 0);   // (the grid keeps the phase)
    const float inv_hidden = 1.f / (float)hidden;
    float acc_w[ITEMS][V] = {}, acc_s[ITEMS][V] = {};
    for (int turn = 0; row < p.rows; row += step, turn ^= 1) {
        auto read = [&](const void *base, size_t ld, int i) {
            return read_window<T, V, EDGE>(static_cast<const T *>(base) + row * ld, e0 + i * estep, hidden);
        };
        auto weight = [&](int i) {
            return read_weight<T, V, EDGE>(static_cast<const T *>(p.weight), e0 + i * estep, hidden);
        };
        float xx = 0.f, tt = 0.f, nt = 0.f;
        Window<T, V> xs[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) xs[i] = read(p.x, p.ldx, i);
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (normed) {
                const Window<T, V> tk = read(p.total, p.ldt, i), gk = read(p.dy, p.lddy, i), wk = weight(i);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    tt = fmaf(tk.at(j), tk.at(j), tt);
                    nt = fmaf(gk.at(j) * wk.at(j), tk.at(j), nt);
                }
            }
#pragma unroll
            for (int j = 0; j < V; ++j) xx = fmaf(xs[i].at(j), xs[i].at(j), xx);
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
        const float m = r * mean_of(nt, (float)hidden, inv_hidden);
        float h[ITEMS][V], hx = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int e = e0 + i * estep;
            float dt[V], f[V];
#pragma unroll
            for (int j = 0; j < V; ++j) dt[j] = 0.f;
            if (p.dtotal) {
                const Window<T, V> dk = read(p.dtotal, p.lddt, i);
#pragma unroll
                for (int j = 0; j < V; ++j) dt[j] = dk.at(j);
            }
            Window<T, V> kk;
            if (gates) kk = read(gates, p.ldg, i);
            if (normed) {
                const Window<T, V> tk = read(p.total, p.ldt, i), gk = read(p.dy, p.lddy, i), wk = weight(i);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float v = tk.at(j) * r, d = gk.at(j);
                    acc_w[i][j] = fmaf(d, v, acc_w[i][j]);
                    dt[j] = fmaf(r, fmaf(-v, m, d * wk.at(j)), dt[j]);
                }
            }
            // outputs may be inputs: an element's were all read above
            if (p.dresidual) {
#pragma unroll
                for (int j = 0; j < V; ++j) f[j] = p.residual_scale * dt[j];
                write_window<T, V, EDGE>(static_cast<T *>(p.dresidual) + row * p.lddr, e, hidden, f);
            }
            read_factor<T, V, EDGE>(p.post, p.gate_rows ? nullptr : p.gate, p.block_scale, e, hidden, f);
            if (p.dgate) {
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] = dt[j] * (f[j] * (xs[i].at(j) * q));
                write_window<T, V, EDGE>(static_cast<T *>(p.dgate) + row * p.lddg, e, hidden, h[i]);
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
            k = q * (q * mean_of(reduce_row<Sum>(hx, warp_only, sums[3][turn]), (float)hidden, inv_hidden));
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
    float *pw = p.partial + (size_t)blockIdx.x * p.pitch;
    float *ps = pw + (size_t)gridDim.x * p.pitch;
    if (blockDim.y > 1) {   // the warps' sums, warp by warp
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
    for (int i = 0; i < ITEMS; ++i) {
        if (e0 + i * estep >= hidden) continue;
        const int at = (int)threadIdx.x * V + i * estep;
        if (normed) write_sums(pw + at, acc_w[i]);
        if (p.sums) write_sums(ps + at, acc_s[i]);
    }
}

// A thread holds ITEMS windows of its row, and the sums over rows of its columns.  HOLD:
// all of the operands' windows, so that the stage is free behind the first sums'
// barrier; else (wide rows, more windows a thread) they are read from the stage again,
// and x's and h's alone are held behind the second one.  AGAIN: not those either, the
// widest rows' sums leave no registers for them; dt is made again for dx, from the stage
// and from vectors in shared memory, and with them there a second stage is not worth its
// room (4000 x 10000 bf16 188 us; held, and spilled, 198; that and two stages, the vectors
// in global memory, 236; 4000 x 8200 152 and 192).
// The rows are normed (dy, total and the weight are there).  Arrays of a stage: x, dy,
// total, the gates where there are any, and dtotal.
struct TeamParams : BlockBackwardParams {
    const void *src[5];
    size_t ld[5];
};

template <typename T, int V, int ITEMS, bool EDGE, bool GATES, bool HOLD, bool AGAIN, int WARPS>
__global__ void __launch_bounds__(32 * WARPS)
block_norm_backward_team_kernel(const __grid_constant__ TeamParams p, const __grid_constant__ TeamPlan plan) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be launched
    __shared__ uint64_t full[WARPS][kMaxStages];
    // rows take turns
    __shared__ __align__(16) float sums[2][kTeams][3][kTeamWarps], last[2][kTeams][kTeamWarps];
    const Team team(plan.warps);
    const int teams = (int)blockDim.x / team.threads(), hidden = (int)p.hidden;
    const int phase = EDGE ? phase_of<V>(p.phase, p.ldx, blockIdx.x) : 0;
    const Vectors<T, V, ITEMS, EDGE> vectors(plan, p.weight, p.post, GATES ? nullptr : p.gate, p.block_scale,
                                             hidden, phase, team);
    constexpr int kDtotal = GATES ? 4 : 3;
    const int slot = team.warps == 1 ? 0 : team.index;   // of what the warps add up
    const size_t row0 = blockIdx.x + (size_t)team.index * gridDim.x, step = (size_t)teams * gridDim.x;
    TeamRing<T, V, 5, ITEMS, EDGE, TeamParams> ring(p, plan, team, full[team.index], vectors.end, phase, hidden, row0, step);
    for (int i = threadIdx.x; i < (int)(sizeof(sums) / sizeof(float)); i += (int)blockDim.x) {
        (&sums[0][0][0][0])[i] = 0.f;
        if (i < (int)(sizeof(last) / sizeof(float))) (&last[0][0][0])[i] = 0.f;
    }
    ring.clear();
    team.sync();
    ring.start();
    vectors.start();
    __syncthreads();
    const float columns = (float)hidden, inv_hidden = 1.f / columns;
    F2 acc_w[ITEMS][V / 2] = {}, acc_s[ITEMS][V / 2] = {};
    int turn = 0;
    for (size_t row = row0; row < p.rows; row += step, turn ^= 1) {
        ring.wait();
        constexpr int kHeld = HOLD ? ITEMS : 1, kKept = AGAIN ? 1 : ITEMS;
        Window<T, V> xs[kKept], gk[kHeld], tk[kHeld], dk[kHeld], kk[kHeld];
        F2 xx = 0, tt = 0, nt = 0;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int h = HOLD ? i : 0, x = AGAIN ? 0 : i;
            xs[x] = ring.window(0, i);
            gk[h] = ring.window(1, i);
            tk[h] = ring.window(2, i);
            if constexpr (HOLD) {
                if constexpr (GATES) kk[h] = ring.window(3, i);
                if (p.dtotal) dk[h] = ring.window(kDtotal, i);
            }
            const Window<T, V> wk = vectors.weights(i);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const F2 u = pair_of(tk[h], j);
                xx = fma2(pair_of(xs[x], j), pair_of(xs[x], j), xx);
                tt = fma2(u, u, tt);
                nt = fma2(mul2(pair_of(gk[h], j), pair_of(wk, j)), u, nt);
            }
        }
        ring.settle();   // the row before's refill, before a barrier
        float sx = low(xx) + high(xx), st = low(tt) + high(tt), sn = low(nt) + high(nt);
        team.sums(sx, st, sn, sums[turn][slot]);
        auto refill = [&] {   // behind a barrier: every thread has its share of the row
            if (team.warps == 1) __syncwarp();
            ring.refill();
        };
        if constexpr (HOLD) refill();
        const float q = p.post ? rsqrtf(mean_of(sx, columns, inv_hidden) + p.eps) : 1.f;
        const float r = rsqrtf(mean_of(st, columns, inv_hidden) + p.eps);
        const float m = r * mean_of(sn, columns, inv_hidden);
        F2 h[kKept][V / 2], hx = 0;
        // dt of a window, r (dy weight - t r m) + dtotal; and dy t r for dweight
        auto gradient = [&](int i, F2 (&dt)[V / 2], bool sum) {
            const int n = HOLD ? i : 0;
            if constexpr (!HOLD) {
                gk[n] = ring.window(1, i);
                tk[n] = ring.window(2, i);
                if constexpr (GATES) kk[n] = ring.window(3, i);
                if (p.dtotal) dk[n] = ring.window(kDtotal, i);
            }
            const Window<T, V> wk = vectors.weights(i);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const F2 v = mul2(pair_of(tk[n], j), both(r)), d = pair_of(gk[n], j);
                if (sum) acc_w[i][j] = fma2(d, v, acc_w[i][j]);
                dt[j] = fma2(v, both(-m), mul2(d, pair_of(wk, j)));
            }
#pragma unroll
            for (int j = 0; j < V / 2; ++j) dt[j] = fma2(dt[j], both(r), p.dtotal ? pair_of(dk[n], j) : 0);
        };
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int n = HOLD ? i : 0, x = AGAIN ? 0 : i, e = vectors.column(i);
            F2 dt[V / 2], f[V / 2];
            gradient(i, dt, true);
            if constexpr (AGAIN) xs[x] = ring.window(0, i);
            if (p.dresidual) {
#pragma unroll
                for (int j = 0; j < V / 2; ++j) f[j] = mul2(dt[j], both(p.residual_scale));
                write_pairs<T, V, EDGE>(static_cast<T *>(p.dresidual) + row * p.lddr, e, hidden, f);
            }
            vectors.factor(i, f);
            if constexpr (GATES) {
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    h[x][j] = mul2(dt[j], mul2(f[j], mul2(pair_of(xs[x], j), both(q))));
                    dt[j] = mul2(dt[j], pair_of(kk[n], j));
                }
                write_pairs<T, V, EDGE>(static_cast<T *>(p.dgate) + row * p.lddg, e, hidden, h[x]);
            }
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const F2 u = pair_of(xs[x], j);
                acc_s[i][j] = fma2(dt[j], mul2(u, both(q)), acc_s[i][j]);
                h[x][j] = mul2(dt[j], f[j]);
                hx = fma2(h[x][j], u, hx);
            }
        }
        float k = 0.f;
        if (p.post) {
            const float sum = team.template total<Sum>(low(hx) + high(hx), last[turn][slot]);
            k = q * (q * mean_of(sum, columns, inv_hidden));
        } else if constexpr (!HOLD && !AGAIN) {
            team.sync();
        }
        if constexpr (!HOLD && !AGAIN) refill();
        T *dx = static_cast<T *>(p.dx) + row * p.lddx;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int x = AGAIN ? 0 : i;
            if constexpr (AGAIN) {
                F2 dt[V / 2], f[V / 2];
                gradient(i, dt, false);
                xs[x] = ring.window(0, i);
                vectors.factor(i, f);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    if constexpr (GATES) dt[j] = mul2(dt[j], pair_of(kk[0], j));
                    h[x][j] = mul2(dt[j], f[j]);
                }
            }
            if (p.post) {
#pragma unroll
                for (int j = 0; j < V / 2; ++j)
                    h[x][j] = mul2(fma2(pair_of(xs[x], j), both(-k), h[x][j]), both(q));
            }
            write_pairs<T, V, EDGE>(dx, vectors.column(i), hidden, h[x]);
        }
        if constexpr (AGAIN) {
            team.sync();
            refill();
        }
        if (EDGE && plan.stages == 1) {   // the next row's ends are read at once
            ring.settle();
            team.sync();
        }
        ring.next();
    }
    if (team.thread == 0) ring.drain();
    float *pw = p.partial + (size_t)blockIdx.x * p.pitch;
    float *ps = pw + (size_t)gridDim.x * p.pitch;
    auto put = [&](float *w, float *s) {   // the thread's sums, from its columns' phase on
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (vectors.column(i) >= hidden) continue;
            const int at = vectors.column(i) + phase;
#pragma unroll
            for (int n = 0; n < V / 4; ++n) {
                const F2 *a = &acc_w[i][2 * n], *b = &acc_s[i][2 * n];
                reinterpret_cast<float4 *>(w + at)[n] = make_float4(low(a[0]), high(a[0]), low(a[1]), high(a[1]));
                if (p.sums)
                    reinterpret_cast<float4 *>(s + at)[n] = make_float4(low(b[0]), high(b[0]), low(b[1]), high(b[1]));
            }
        }
    };
    if (teams == 1) {
        put(pw, ps);
        return;
    }
    // the teams' sums, where the vectors and rows lay, added up in the teams' order (all at
    // once: 3000 x 512 bf16 17 us, team by team 29; the loop over teams keeps the compiler
    // from holding what follows through the rows: 20000 x 2048 with row gates 114, else 138)
    float *joined = reinterpret_cast<float *>(smem());
    const int pitch = (int)p.pitch;
    __syncthreads();
    for (int g = 0; g < teams; ++g)
        if (team.index == g) put(joined + 2 * g * pitch, joined + (2 * g + 1) * pitch);
    __syncthreads();
    for (int at = 4 * (int)threadIdx.x; at < pitch; at += 4 * (int)blockDim.x) {
        for (int n = 0; n < (p.sums ? 2 : 1); ++n) {
            const float *from = joined + n * pitch + at;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int g = 0; g < teams; ++g, from += 2 * pitch) {
                const float4 u = *reinterpret_cast<const float4 *>(from);
                v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
            *reinterpret_cast<float4 *>((n == 0 ? pw : ps) + at) = v;
        }
    }
}

// The blocks' sums, added up in a fixed order: dweight, and from S the gradients of
// the weight after the block and of a column gate.  A block's sums start its rows' phase
// into its row of them, where `phases` (V - 1, or 0) says so.
constexpr int kJoinRows = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kJoinRows)
block_join_kernel(const float *partial, const T *post, const T *gate, float block_scale,
                  float *dweight, float *dpost, float *dgate, uint32_t hidden, uint32_t pitch,
                  uint32_t phase, uint32_t ld, uint32_t phases, int parts) {
    __shared__ float sums[kJoinRows][33];
    const uint32_t e = blockIdx.x * 32 + threadIdx.x;
    const bool second = blockIdx.y == (dweight ? 1 : 0);
    if (second) partial += (size_t)parts * pitch;
    // launched while the rows are still being worked on: wait for all of them
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float v = 0.f;
    if (e < hidden) {
#pragma unroll 8
        for (uint32_t b = threadIdx.y; b < (uint32_t)parts; b += blockDim.y)
            v += partial[(size_t)b * pitch + ((phase + ld * b) & phases) + e];
    }
    sums[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y != 0 || e >= hidden) return;
    v = sums[0][threadIdx.x];
    for (unsigned k = 1; k < blockDim.y; ++k) v += sums[k][threadIdx.x];
    if (!second) {
        dweight[e] = v;
        return;
    }
    v *= block_scale;
    if (dpost) dpost[e] = gate ? v * to_f32<T>(gate[e]) : v;
    if (dgate) dgate[e] = post ? v * to_f32<T>(post[e]) : v;
}

// Whether the sum S over rows is wanted.
bool wants_sums(const BlockNormBackwardArgs &a) {
    return a.post_weight != nullptr || (a.gate != nullptr && !a.gate_rows);
}

// A block's row of sums over rows: whole windows, whatever the phase.
uint32_t sums_pitch(const BlockNormBackwardArgs &a) {
    const size_t V = a.dtype == PURLIN_F32 ? 4 : 8;
    return (uint32_t)((a.hidden + 2 * V - 2) / V * V);
}

// A backward launch: its shape, and whether it takes windows and meets edges.
struct BlockBackwardShape : Shape {
    TeamShape team;   // plan.warps 0: none
    int team_items = 0;
    bool few_warps = false;
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
    const bool edge = reinterpret_cast<uintptr_t>(a.x) % 16 != 0 || a.ldx % V != 0 || a.hidden % V != 0;
    s.edge = edge;
    for (const void *v : {a.post_weight, a.gate_rows ? nullptr : a.gate, a.weight})
        s.edge = s.edge || reinterpret_cast<uintptr_t>(v) % 16 != 0;
    Shape &base = s;
    if (s.windows && a.weight) {
        const int arrays = 3 + (a.dtotal ? 1 : 0) + (gates ? 1 : 0);
        const bool factors = a.post_weight || (a.gate && !a.gate_rows);
        const int warps = (int)(warps_of(windows_of<V>(a.hidden, s.edge), 4) / 32);
        s.few_warps = warps >= 4 && warps <= kFewWarps && kFewWarps % warps <= 1 && a.rows / a.sms >= 32;
        if (s.few_warps) {
            s.team = team_shape<V>(a.rows, a.hidden, s.edge, arrays, true, factors, 4, true, false, kFewWarps,
                                   kFewWarps, a.sms);
            s.grid = s.team.grid;
            if (s.team.plan.warps != 0) return s;
        }
        s.few_warps = false;
        for (s.team_items = 2; s.team_items <= 32 / V; s.team_items *= 2) {
            s.team = team_shape<V>(a.rows, a.hidden, s.edge, arrays, true, factors, s.team_items, true,
                                   s.team_items == 32 / V, kBackwardWarps, kBackwardWarps, a.sms);
            s.grid = s.team.grid;
            if (s.team.plan.warps != 0) return s;
        }
    }
    for (unsigned threads : {512u, 1024u}) {
        base = s.windows ? direct_shape<V>(a.rows, a.hidden, edge, kBackwardHeld, threads, a.sms)
                         : direct_shape<1>(a.rows, a.hidden, false, kBackwardHeld, threads, a.sms);
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
    const size_t fit = std::max<size_t>(1, kDirectThreadsSm / (s.tx * s.ty));
    const size_t grid = std::max<size_t>((size_t)a.sms * fit / V * V, V);
    s.grid = (unsigned)std::min<size_t>((a.rows + s.ty - 1) / s.ty, grid);
    return s;
}

template <typename T, int V, int ITEMS, bool EDGE, bool GATES, int WARPS = kBackwardWarps>
cudaError_t backward_teams(const BlockNormBackwardArgs &a, const TeamParams &p, const TeamShape &s) {
    constexpr bool HOLD = ITEMS == 2 || WARPS != kBackwardWarps, AGAIN = !HOLD && ITEMS * V == 32;
    static SharedMemoryLimit limit;
    const auto kernel = block_norm_backward_team_kernel<T, V, ITEMS, EDGE, GATES, HOLD, AGAIN, WARPS>;
    const cudaError_t ready = limit.raise(kernel, kTeamSmem);
    if (ready != cudaSuccess) return ready;
    kernel<<<s.grid, s.threads, s.smem, a.stream>>>(p, s.plan);
    return cudaGetLastError();
}

template <typename T, int V, bool EDGE, bool GATES>
cudaError_t backward_teams(const BlockNormBackwardArgs &a, const BlockBackwardParams &b,
                           const BlockBackwardShape &s) {
    const TeamParams p{b, {a.x, a.dy, a.total, GATES ? a.gate : a.dtotal, a.dtotal},
                       {a.ldx, a.lddy, a.ldt, GATES ? a.ldg : a.lddt, a.lddt}};
    if (s.few_warps) return backward_teams<T, V, 4, EDGE, GATES, kFewWarps>(a, p, s.team);
    if (s.team_items == 2) return backward_teams<T, V, 2, EDGE, GATES>(a, p, s.team);
    if (s.team_items == 4) return backward_teams<T, V, 4, EDGE, GATES>(a, p, s.team);
    if constexpr (V == 4) return backward_teams<T, V, 8, EDGE, GATES>(a, p, s.team);
    return cudaErrorInvalidConfiguration;
}

template <typename T, int V>
cudaError_t backward_direct(const BlockNormBackwardArgs &a, const BlockBackwardParams &p,
                            const BlockBackwardShape &s) {
    constexpr bool EDGE = V > 1;
    constexpr int MOST = kBackwardHeld / V;
    const dim3 block(s.tx, s.ty);
    if (s.items == 0) block_norm_backward_long_kernel<T><<<s.grid, 1024, 0, a.stream>>>(p);
    else if (s.wide) block_norm_backward_kernel<T, V, MOST, EDGE, 1024><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == 1) block_norm_backward_kernel<T, V, 1, EDGE, 512><<<s.grid, block, 0, a.stream>>>(p);
    else if (s.items == MOST) block_norm_backward_kernel<T, V, MOST, EDGE, 512><<<s.grid, block, 0, a.stream>>>(p);
    else if constexpr (V == 4) block_norm_backward_kernel<T, V, 2, EDGE, 512><<<s.grid, block, 0, a.stream>>>(p);
    else if constexpr (V == 1) block_norm_backward_kernel<T, V, 4, EDGE, 512><<<s.grid, block, 0, a.stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t block_norm_backward_any(const BlockNormBackwardArgs &a) {
    constexpr int V = 16 / sizeof(T);
    const bool sums = wants_sums(a);
    const BlockBackwardShape s = block_backward_shape<T>(a);
    const BlockBackwardParams p{a.dy, a.dtotal, a.x, a.total, a.post_weight, a.gate, a.weight,
                                a.dx, a.dresidual, a.gate_rows ? a.dgate : nullptr, a.partial, sums_pitch(a),
                                a.lddy, a.lddt, a.ldx, a.ldt, a.ldg, a.lddx, a.lddr, a.lddg, a.rows,
                                (uint32_t)a.hidden,
                                (uint32_t)(reinterpret_cast<uintptr_t>(a.x) / sizeof(T) % V),
                                a.block_scale, a.residual_scale, a.eps, a.gate_rows, sums, a.err};
    const cudaError_t e = s.team.plan.warps != 0
                              ? a.gate_rows ? s.edge ? backward_teams<T, V, true, true>(a, p, s)
                                                     : backward_teams<T, V, false, true>(a, p, s)
                                : s.edge    ? backward_teams<T, V, true, false>(a, p, s)
                                            : backward_teams<T, V, false, false>(a, p, s)
                          : s.windows ? backward_direct<T, V>(a, p, s)
                                      : backward_direct<T, 1>(a, p, s);
    const unsigned vectors = (a.weight ? 1 : 0) + (sums ? 1 : 0);
    // the sums of rows in windows, unless a block adds up those of several phases itself
    const bool phased = s.team.plan.warps != 0 || (s.windows && s.items != 0 && s.ty == 1);
    if (e != cudaSuccess || vectors == 0) return e;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)((a.hidden + 31) / 32), vectors);
    // more blocks than fit at once, or few sums to add: smaller ones (400 x 12288 bf16 51
    // us, else 56; 2000 x 1024 18 and 17)
    const bool small = (size_t)c.gridDim.x * vectors > 2 * (size_t)a.sms || s.grid <= kJoinRows / 4;
    c.blockDim = dim3(32, small ? kJoinRows / 4 : kJoinRows);
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
                              (uint32_t)a.hidden, p.pitch, p.phase, (uint32_t)(a.ldx % V),
                              phased ? (uint32_t)(V - 1) : 0u, (int)s.grid);
}

}  // namespace

size_t block_norm_backward_workspace(const BlockNormBackwardArgs &a) {
    if (a.weight == nullptr && !wants_sums(a)) return 0;
    const unsigned grid = a.dtype == PURLIN_F32 ? block_backward_shape<float>(a).grid
                                                : block_backward_shape<__nv_bfloat16>(a).grid;
    return 2 * (size_t)grid * sums_pitch(a) * sizeof(float);
}

cudaError_t launch_block_norm_backward(const BlockNormBackwardArgs &a) {
    return a.dtype == PURLIN_F32 ? block_norm_backward_any<float>(a)
                                 : block_norm_backward_any<__nv_bfloat16>(a);
}

}  // namespace purlin
