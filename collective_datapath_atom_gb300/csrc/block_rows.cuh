// block_rows.cuh -- what the norms around a block (block_norm.cu) and their backward
// pass (block_norm_backward.cu) share: the factor of the block's output, teams of warps
// with rings of rows in shared memory, and the launches' shapes.  Internal to the library.
#pragma once

#include <iterator>

#define PURLIN_ROWS_ONLY
#include "rms_norm.cu"

namespace purlin {
namespace {

constexpr int kTeamWarps = 16;                // most warps of a team
constexpr int kTeams = 15;                    // most teams of more than a warp: their barriers
constexpr int kTeamSmem = 216 * 1024;         // most dynamic shared memory of one: 11 KiB are its own

// The factor of x q in t for a window, block_scale * post_weight * column gate, in
// binary32.
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

// ------------------------------------------------------------------- pairs --

// Two binary32 values in one register pair: a multiplication, a sum or both of two
// columns in one instruction, each rounded as it would be alone.  The rows' arithmetic
// would fill the issue slots otherwise (backward of 32768 x 4096 bf16: 53 instructions an
// element, 293 us).
using F2 = unsigned long long;

__device__ __forceinline__ F2 pair(float lo, float hi) {
    F2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ F2 both(float v) { return pair(v, v); }
__device__ __forceinline__ float low(F2 a) {
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
    return lo;
}
__device__ __forceinline__ float high(F2 a) {
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a));
    return hi;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// The j-th pair of a window.
template <typename T, int V>
__device__ __forceinline__ F2 pair_of(const Window<T, V> &k, int j) {
    return pair(k.at(2 * j), k.at(2 * j + 1));
}
template <typename O, int V, bool EDGE>
__device__ __forceinline__ void write_pairs(O *row, int e, int hidden, const F2 (&in)[V / 2]) {
    float f[V];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
        f[2 * j] = low(in[j]);
        f[2 * j + 1] = high(in[j]);
    }
    write_window<O, V, EDGE>(row, e, hidden, f);
}

// ------------------------------------------------------------ teams of warps --

// Many rows: a block an SM for good, its warps in teams of `warps`, a row a team at a
// time.  A team has a ring of its own rows in shared memory and a barrier of its own;
// the vectors (weights, column gates) lie there once for all of them.  Rows of a block
// are a multiple of the windows' elements apart, so they have one phase, and a thread's
// columns are the same in all of them.
struct TeamPlan {
    int warps;                           // of a team
    int stages;                          // of its ring
    int arrays;                          // operands of a stage
    bool weight_staged, factor_staged;   // vectors that lie in shared memory
};

// Dynamic shared memory, by its name: addresses of 32 bits.
__device__ __forceinline__ unsigned char *smem() {
    extern __shared__ __align__(128) unsigned char stage[];
    return stage;
}

template <typename T, int V>
__device__ __forceinline__ Window<T, V> staged_window(uint32_t at) {
    const uint4 u = *reinterpret_cast<const uint4 *>(smem() + at);
    Window<T, V> k;
    k.w[0] = u.x;
    k.w[1] = u.y;
    k.w[2] = u.z;
    k.w[3] = u.w;
    return k;
}

// What the warps of a team add up: a float a warp, and zeros behind them.
// Eight floats at once, as a tree.
template <typename Op>
__device__ __forceinline__ float join_eight(const float *shared) {
    const float4 a = reinterpret_cast<const float4 *>(shared)[0], b = reinterpret_cast<const float4 *>(shared)[1];
    return Op::f(Op::f(Op::f(a.x, a.y), Op::f(a.z, a.w)), Op::f(Op::f(b.x, b.y), Op::f(b.z, b.w)));
}
template <typename Op>
__device__ __forceinline__ float join_warps(const float *shared, int warps) {
    const float v = join_eight<Op>(shared);
    return warps <= 8 ? v : Op::f(v, join_eight<Op>(shared + 8));
}

struct Team {
    // thread: within the team.  A thread's windows are every 32nd from window(ITEMS) on:
    // a warp's lie together, and the distances are known to the compiler
    int index, warps, thread;
    __device__ explicit Team(int warps)
        : index((int)(threadIdx.x >> 5) / warps), warps(warps),
          thread((int)threadIdx.x - index * warps * 32) {}
    __device__ int threads() const { return warps * 32; }
    __device__ int window(int items) const { return (thread & ~31) * items + (thread & 31); }
    __device__ __forceinline__ void sync() const {
        if (warps == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(warps * 32) : "memory");
    }
    // Reduction over the team's threads; `shared`: kTeamWarps floats, which the next
    // but one reduction may use again.
    template <typename Op>
    __device__ __forceinline__ float total(float v, float *shared) const {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = Op::f(v, __shfl_xor_sync(0xffffffffu, v, o));
        if (warps == 1) return v;
        if ((thread & 31) == 0) shared[thread >> 5] = v;
        sync();
        return join_warps<Op>(shared, warps);
    }
    // Three sums at once; lanes hand over what they do not keep: six exchanges for fifteen.
    __device__ __forceinline__ void sums(float &a, float &b, float &c, float (*shared)[kTeamWarps]) const {
        const int lane = thread & 31;
        const bool upper = lane & 16, odd = lane & 8;
        float u = (upper ? c : a) + __shfl_xor_sync(0xffffffffu, upper ? a : c, 16);
        float v = (upper ? 0.f : b) + __shfl_xor_sync(0xffffffffu, upper ? b : 0.f, 16);
        u = (odd ? v : u) + __shfl_xor_sync(0xffffffffu, odd ? u : v, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
        if (warps == 1) {   // a in lane 0, b in 8, c in 16
            a = __shfl_sync(0xffffffffu, u, 0);
            b = __shfl_sync(0xffffffffu, u, 8);
            c = __shfl_sync(0xffffffffu, u, 16);
            return;
        }
        if (lane % 8 == 0 && lane < 24) shared[lane / 8][thread >> 5] = u;
        sync();
        a = join_warps<Sum>(shared[0], warps);
        b = join_warps<Sum>(shared[1], warps);
        c = join_warps<Sum>(shared[2], warps);
    }
};

// A team's ring of rows: `arrays` operands of a row a stage, the windows that lie wholly
// in the row brought by bulk copies, each at its place, and the elements at the row's
// ends one by one, loads of a few threads that are under way while the row before is
// worked on.  Whatever else a stage has up to the last thread's last window is zero and
// stays so: a thread reads its windows without asking.  One thread issues; a stage is
// refilled behind a barrier after which every thread has its share of it.
template <typename T, int V, int ARRAYS, int ITEMS, bool EDGE, typename P>
struct TeamRing {
    static constexpr int kEnds = (ARRAYS * 2 * V + 31) / 32;   // of a thread, at most
    const P &p;             // src[], ld[], rows, err: read where they are needed
    const Team &team;
    uint64_t *full;         // a barrier a stage
    uint32_t base, array_bytes, stage_bytes;   // base: of the ring, from the start of shared memory
    int stages, arrays, phase, hidden;
    uint32_t at;            // this thread's first window in the stage of the row at hand
    int st = 0;
    uint32_t parity = 0;
    int fill = 0;           // the stage for the next row
    size_t next_row, step;
    uint32_t issued = 0;
    bool dead = false;      // a wait expired: no more of them
    bool pending = false;   // a refill whose ends are still to be put in place
    T end[EDGE ? kEnds : 1];
    int place[EDGE ? kEnds : 1];   // of this thread's ends: elements from the row's start, or -1

    __device__ TeamRing(const P &p, const TeamPlan &plan, const Team &team, uint64_t *full, uint32_t rings,
                        int phase, int hidden, size_t row0, size_t step)
        : p(p), team(team), full(full), array_bytes(ITEMS * team.threads() * 16),
          stage_bytes(plan.arrays * array_bytes), stages(plan.stages), arrays(plan.arrays), phase(phase),
          hidden(hidden), next_row(row0), step(step) {
        base = rings + team.index * stages * stage_bytes;
        at = base + team.window(ITEMS) * 16;
    }
    // Team thread 0: fill the stage at `fill` with the next row, if one is left.
    __device__ __forceinline__ void issue() {
        const int first = EDGE && phase > 0 ? 1 : 0, count = max(0, (phase + hidden) / V - first);
        atom::mbar_arrive_expect_tx(&full[fill], (uint32_t)(count * 16 * arrays));
        if (count == 0) return;
        unsigned char *to = smem() + base + fill * stage_bytes + first * 16;
#pragma unroll
        for (int a = 0; a < ARRAYS; ++a)
            if (a < arrays)
                atom::bulk_load(to + a * array_bytes,
                                static_cast<const T *>(p.src[a]) + next_row * p.ld[a] + first * V - phase,
                                (uint32_t)count * 16, &full[fill]);
    }
    __device__ __forceinline__ int end_array(int k) const { return (team.thread + k * team.threads()) / (2 * V); }
    // Where this thread's k-th end lies in its row; -1: it has none.
    __device__ int end_place(int k) const {
        const int n = team.thread + k * team.threads(), whole = (phase + hidden) / V;
        const bool last = n / V % 2 == 1;
        // the first window is partial where the row starts within it; a window that is
        // both first and last is the first
        if (n / (2 * V) >= arrays || (last ? whole == 0 && phase > 0 : phase == 0)) return -1;
        const int e = (last ? whole * V : 0) + n % V - phase;
        return e < hidden ? e : -1;
    }
    // Every thread, behind a barrier after which the row at hand is no longer read from
    // its stage: the next row is on its way there.
    __device__ __forceinline__ void refill() {
        pending = next_row < p.rows && !dead;
        if (pending && team.thread == 0) issue();
        if constexpr (EDGE) {
            // every thread loads, some element of its block's first row where it has none to:
            // behind a branch the compiler waits for the load (8000 x 4000 f32 of pitch 4099,
            // backward, 171 us, so 164; aligned 128)
            const size_t row = pending ? next_row : blockIdx.x;
#pragma unroll
            for (int k = 0; k < kEnds; ++k) {
                const int a = min(end_array(k), arrays - 1);
                end[k] = static_cast<const T *>(p.src[a])[row * p.ld[a] + max(place[k], 0)];
            }
        }
    }
    // Every thread, later: and its ends are in place, for reads behind the team's next
    // barrier.  Nothing where no refill is pending.
    __device__ __forceinline__ void settle() {
        if (!pending) return;
        pending = false;
        if constexpr (EDGE) {
#pragma unroll
            for (int k = 0; k < kEnds; ++k)
                if (place[k] >= 0)
                    reinterpret_cast<T *>(smem() + base + fill * stage_bytes +
                                          end_array(k) * array_bytes)[phase + place[k]] = end[k];
        }
        ++issued;
        fill = fill + 1 == stages ? 0 : fill + 1;
        next_row += step;
    }
    // Every thread, once: zeros and barriers.  A barrier of the team follows.
    __device__ void clear() {
        if constexpr (EDGE) {
#pragma unroll
            for (int k = 0; k < kEnds; ++k) place[k] = end_place(k);
        }
        const int first = EDGE && phase > 0 ? 1 : 0, behind = (phase + hidden) / V;   // windows of no bulk copy
        for (int n = 0; n < stages * arrays; ++n)
            for (int w = team.thread; w < ITEMS * team.threads(); w += team.threads())
                if (w < first || w >= behind)
                    *reinterpret_cast<uint4 *>(smem() + base + n * array_bytes + w * 16) = make_uint4(0, 0, 0, 0);
        if (team.thread == 0) {
            for (int i = 0; i < stages; ++i) atom::mbar_init(&full[i], 1);
            atom::mbar_init_fence();
        }
    }
    // Every thread, behind it: the first rows.  A block barrier follows.
    __device__ void start() {
        for (int i = 0; i < stages; ++i) {
            refill();
            settle();
        }
    }
    // Every thread: the row at hand is in its stage.  Two seconds at most.
    __device__ __forceinline__ void wait() {
        if (!dead && !bounded_row_wait(&full[st], parity, p.err)) dead = true;
    }
    // Every thread: on to the next row.
    __device__ __forceinline__ void next() {
        at += stage_bytes;
        if (++st == stages) {
            st = 0;
            parity ^= 1;
            at = base + team.window(ITEMS) * 16;
        }
    }
    __device__ __forceinline__ Window<T, V> window(int a, int i) const {
        return staged_window<T, V>(at + a * array_bytes + i * 512);
    }
    // Team thread 0, at the end: copies that a wait gave up on land before the exit.
    __device__ void drain() {
        if (!dead) return;
        for (uint32_t n = issued > (uint32_t)stages ? issued - stages : 0; n < issued; ++n)
            bounded_row_wait(&full[n % (uint32_t)stages], (n / (uint32_t)stages) & 1, p.err);
    }
};

// The vectors of a block, in windows; thread by thread of a team, which all agree.
template <typename T, int V, int ITEMS, bool EDGE>
struct Vectors {
    const void *weight, *post, *gate;
    float scale;
    int hidden, e0;
    uint32_t weight_at, factor_at, end;   // this thread's, from the start of shared memory; behind them
    bool weight_staged, factor_staged, factors;

    __device__ Vectors(const TeamPlan &plan, const void *weight, const void *post, const void *gate, float scale,
                       int hidden, int phase, const Team &team)
        : weight(weight), post(post), gate(gate), scale(scale), hidden(hidden),
          e0(team.window(ITEMS) * V - phase), weight_staged(plan.weight_staged),
          factor_staged(plan.factor_staged), factors(post != nullptr || gate != nullptr) {
        const uint32_t weight_bytes = weight_staged ? ITEMS * team.threads() * 16 : 0;
        weight_at = team.window(ITEMS) * 16;
        factor_at = weight_bytes + team.window(ITEMS * (V / 4)) * 16;
        end = weight_bytes + (factor_staged ? ITEMS * team.threads() * V * 4 : 0);
    }
    __device__ __forceinline__ int column(int i) const { return e0 + i * 32 * V; }
    __device__ __forceinline__ float4 *factor_quad(int i, int n) const {
        return reinterpret_cast<float4 *>(smem() + factor_at + (i * (V / 4) + n) * 512);
    }
    // Every team writes the same; a block barrier follows.
    __device__ void start() const {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (weight_staged) {
                const Window<T, V> k = read_weight<T, V, EDGE>(static_cast<const T *>(weight), column(i), hidden);
                *reinterpret_cast<uint4 *>(smem() + weight_at + i * 512) = make_uint4(k.w[0], k.w[1], k.w[2], k.w[3]);
            }
            if (factor_staged) {
                float c[V];
                read_factor<T, V, EDGE>(post, gate, scale, column(i), hidden, c);
#pragma unroll
                for (int n = 0; n < V / 4; ++n)
                    *factor_quad(i, n) = make_float4(c[4 * n], c[4 * n + 1], c[4 * n + 2], c[4 * n + 3]);
            }
        }
    }
    __device__ __forceinline__ Window<T, V> weights(int i) const {
        if (!weight_staged) return read_weight<T, V, EDGE>(static_cast<const T *>(weight), column(i), hidden);
        return staged_window<T, V>(weight_at + i * 512);
    }
    __device__ __forceinline__ void factor(int i, F2 (&c)[V / 2]) const {
        if (factor_staged) {
#pragma unroll
            for (int n = 0; n < V / 4; ++n) {
                const float4 f = *factor_quad(i, n);
                c[2 * n] = pair(f.x, f.y);
                c[2 * n + 1] = pair(f.z, f.w);
            }
        } else if (factors) {
            float f[V];
            read_factor<T, V, EDGE>(post, gate, scale, column(i), hidden, f);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) c[j] = pair(f[2 * j], f[2 * j + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < V / 2; ++j) c[j] = both(scale);
        }
    }
};

// Rows on the registers: a warp a row where it holds one, else a block; `most` values
// a thread.  items 0: the row does not fit `threads`.
template <int V>
Shape direct_shape(size_t rows, size_t hidden, bool edge, int most, unsigned threads, int sms) {
    Shape s;
    const size_t windows = windows_of<V>(hidden, edge);
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

// A launch of teams; plan.warps 0 where the rows are too few or too long for it.
struct TeamShape {
    TeamPlan plan = {};
    unsigned threads = 0, grid = 0;
    size_t smem = 0;
};

// Teams with `items` windows a thread, `arrays` operands a stage, and two stages at
// least; vectors that the rows leave no room for are read from global memory, and last a
// ring has one stage.  vectors_first: that comes before, where the vectors are read again
// and again in a row.  Teams: `least_warps` an SM, which the arithmetic wants, and rows
// for about 100 KB on their way; reads that run further ahead of the writes slow both
// down (forward 16384 x 4096 bf16: three teams of two stages, 98 KB, 91 us, four 104).
// joins: the teams' sums over rows are added up in shared memory, two floats a column
// and team.
// block_warps: of a block at most, 32 at most.
constexpr size_t kTeamFlight = 100 * 1024, kRingFlight = 128 * 1024;

template <int V>
TeamShape team_shape(size_t rows, size_t hidden, bool edge, int arrays, bool weight, bool factors, int items,
                     bool joins, bool vectors_first, int block_warps, int least_warps, int sms) {
    TeamShape s;
    if (rows < (size_t)sms) return s;
    const int warps = (int)(warps_of(windows_of<V>(hidden, edge), items) / 32);
    if (warps > std::min(kTeamWarps, block_warps)) return s;
    const size_t windows = (size_t)items * warps * 32;
    const size_t stage = windows * 16 * (size_t)arrays, room = kTeamSmem;
    // stages at least, and vectors that are left in global memory
    constexpr int kRowsFirst[][2] = {{2, 0}, {2, 1}, {2, 2}, {1, 2}};
    constexpr int kVectorsFirst[][2] = {{2, 0}, {1, 0}, {2, 1}, {1, 1}, {1, 2}};
    const auto *tries = vectors_first ? kVectorsFirst : kRowsFirst;
    const int most = vectors_first ? (int)std::size(kVectorsFirst) : (int)std::size(kRowsFirst);
    for (int n = 0; n < most; ++n) {
        const int want = tries[n][0], drop = tries[n][1];
        const bool ws = weight && drop < 2, fs = factors && drop < 1;
        const size_t vectors = windows * ((ws ? 16 : 0) + (fs ? 4 * V : 0));
        const size_t some = std::max<size_t>((least_warps + warps - 1) / warps, kTeamFlight / (2 * stage));
        for (size_t teams = std::min({some, (size_t)(block_warps / warps), (rows + sms - 1) / sms}); teams >= 1; --teams) {
            if (vectors + teams * want * stage > room) continue;
            if (joins && teams > 1 && vectors + teams * want * stage < 8 * (hidden + 2 * V) * teams) continue;
            const size_t stages = std::min({(size_t)kMaxStages, (room - vectors) / (teams * stage),
                                            std::max<size_t>(want, kRingFlight / (teams * stage))});
            s.plan = TeamPlan{warps, (int)stages, arrays, ws, fs};
            s.threads = (unsigned)(teams * warps * 32);
            s.smem = vectors + teams * stages * stage;
            s.grid = (unsigned)std::max<size_t>((size_t)sms / V * V, V);
            return s;
        }
    }
    return s;
}

}  // namespace
}  // namespace purlin
