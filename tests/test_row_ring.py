"""The norm's ring of rows in shared memory (RowRing in csrc/rms_norm.cu), compiled
here on the host from the library's own source, over barriers and bulk copies that
land in any order.

Rows of every phase and length have to come out as they lie in memory, and a stage may
not be filled while its row is still to be read.  A copy that never lands (dropped here
on the host) makes a wait run out: the ring then waits for nothing more, fetches
nothing more, records the error, and sees its other copies in flight land before the
block's exit, all of it in bounded time.
"""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(os.path.dirname(HERE), "collective_datapath_atom_gb300", "csrc", "rms_norm.cu")

PRELUDE = r"""
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <random>
#include <vector>
using std::max;
using std::min;
struct __nv_bfloat16 { unsigned short bits; };
struct uint4 { uint32_t x, y, z, w; };
static float __uint_as_float(uint32_t u) { float f; std::memcpy(&f, &u, 4); return f; }
static uint32_t __float_as_uint(float f) { uint32_t u; std::memcpy(&u, &f, 4); return u; }
static struct { unsigned x = 0; } blockIdx;
enum { PURLIN_ERR_TIMEOUT = 7 };
static int errors = 0;
namespace snac {
constexpr uint64_t kRingWaitNs = 2000000000ull;
enum { kSiteRowWait = 11 };
static void record_error(unsigned long long *, int, int, unsigned) { ++errors; }
}
/* ---- barriers of one arrival, and copies that land when chance lets them */
struct Bar { int phase = 0, pending = 1; long tx = 0; };
struct Copy { void *to; const void *from; uint32_t bytes; uint64_t *bar; bool dropped; uint64_t due; };
static std::map<uint64_t *, Bar> bars;
static std::vector<Copy> flying;
static std::mt19937 rng;
static uint64_t now = 0;
static int copies = 0, drop = -1, fault = 0;
static bool slow = false;   /* copies take up to 3.9 s, longer than a wait */
static void settle(Bar &b) {
    if (b.pending == 0 && b.tx == 0) { ++b.phase; b.pending = 1; }
}
static void land(size_t i) {
    Copy c = flying[i];
    flying.erase(flying.begin() + i);
    std::memcpy(c.to, c.from, c.bytes);
    Bar &b = bars[c.bar];
    b.tx -= c.bytes;
    settle(b);
}
static void time_passes() {
    now += 10000000;   /* 10 ms a look */
    if (!flying.empty()) {
        const size_t i = rng() % flying.size();
        if (!flying[i].dropped && now >= flying[i].due && rng() % 3 == 0) land(i);
    }
}
namespace atom {
static void mbar_init(uint64_t *b, int n) { bars[b] = Bar{0, n, 0}; }
static void mbar_init_fence() {}
static void mbar_arrive_expect_tx(uint64_t *b, uint32_t bytes) {
    Bar &s = bars[b];
    if (s.pending == 0) fault |= 1;          /* the stage is still being filled */
    s.tx += bytes;
    --s.pending;
    settle(s);
}
static bool mbar_try_wait(uint64_t *b, uint32_t parity) {
    time_passes();
    return (bars[b].phase & 1) != (int)parity;
}
static uint64_t globaltimer_ns() { return now; }
static void bulk_load(void *to, const void *from, uint32_t bytes, uint64_t *bar) {
    if ((uintptr_t)to % 16 || (uintptr_t)from % 16 || bytes % 16 || bytes == 0) fault |= 2;
    const uint64_t due = slow ? now + rng() % 3800000000u : 0;
    flying.push_back({to, from, bytes, bar, copies++ == drop, due});
}
}
"""

MAIN = r"""
/* the block's walk, as the staged kernels have it: thread 0 issues, `late` only a row
   after (backward, which reads a row twice) */
template <typename T, int V, bool EDGE>
static int block(int rows, int hidden, int ld, int off, int arrays, int stages, int grid, int b,
                 bool late, int lost) {
    using Ring = RowRing<T, V, 3>;
    bars.clear(); flying.clear();
    errors = fault = copies = 0; now = 1; drop = lost;
    const int phase0 = off % V;
    std::vector<std::vector<T>> src(arrays);
    unsigned value = 1;
    std::vector<T *> p(arrays);
    for (int a = 0; a < arrays; ++a) {
        src[a].resize((size_t)rows * ld + off + 16 / sizeof(T));
        T *base = src[a].data();
        while ((uintptr_t)base % 16) ++base;
        p[a] = base + off;
        for (size_t i = 0; i + (base - src[a].data()) < src[a].size(); ++i) {
            const unsigned v = value++;
            std::memcpy(&base[i], &v, sizeof(T));
        }
    }
    const int phase = EDGE ? (phase0 + b * (ld % V)) % V : 0;
    typename Ring::Shared shared;
    const size_t windows = (size_t)(hidden + 2 * (V - 1)) / V;
    std::vector<unsigned char> mem((size_t)stages * arrays * windows * 16 + 16);
    unsigned char *base = mem.data();
    while ((uintptr_t)base % 16) ++base;
    Ring t0(shared, base, stages, arrays, hidden, phase, b, grid, rows);
    for (int a = 0; a < 3; ++a) { t0.src[a] = a < arrays ? p[a] : nullptr; t0.ld[a] = ld; }
    Ring t1 = t0;
    unsigned long long err = 0;
    t0.init();
    for (int i = 0; i < stages; ++i) t0.issue();
    uint32_t n = 0, issued_dead = 0;
    bool dead = false;
    uint64_t died = 0;
    for (size_t row = b; row < (size_t)rows; row += grid, ++n, t0.next(), t1.next()) {
        t0.wait(&err);
        /* (thread 1 waits at the same time, and sees the same) */
        if (t0.dead && !dead) { dead = true; issued_dead = t0.issued; died = now; }
        auto check = [&] {
            for (int a = 0; a < arrays && !t0.dead; ++a)
                for (int w = 0; w * V - phase < hidden; ++w) {
                    const Window<T, V> k = t1.template read<EDGE>(row, a, w, hidden);
                    for (int j = 0; j < V; ++j) {
                        const int e = w * V - phase + j;
                        uint32_t want = 0;
                        if (e >= 0 && e < hidden) want = bits_of(p[a] + row * ld + e);
                        const float f = k.at(j);
                        const uint32_t got = sizeof(T) == 4 ? __float_as_uint(f) : __float_as_uint(f) >> 16;
                        if (got != want) fault |= 4;
                    }
                }
        };
        check();
        if (late) {
            if (n > 0) t0.issue();
            check();
        } else {
            t0.issue();
        }
    }
    if (dead && t0.issued != issued_dead) fault |= 8;         /* fetched on */
    t0.drain(&err);
    for (const Copy &c : flying) if (!c.dropped) fault |= 16; /* a copy outlives the block */
    const bool short_of_one = lost >= 0 && lost < copies;
    if (slow ? short_of_one && errors == 0 : short_of_one != (errors > 0)) fault |= 32;
    if (dead && now - died > (uint64_t)stages * 2100000000ull) fault |= 64;   /* the drain's waits */
    return fault;
}

template <typename T, int V>
static int many() {
    int bad = 0;
    for (int turn = 0; turn < 3000 && !bad; ++turn) {
        rng.seed(turn);
        const int hidden = 1 + rng() % 70, arrays = 1 + rng() % 3, stages = 2 + rng() % 3;
        const bool edge = rng() % 3 != 0, late = rng() % 2;
        const int grid = V * (1 + rng() % 2), rows = 1 + rng() % 60, b = rng() % std::min(grid, rows);
        slow = rng() % 4 == 0;
        const int lost = rng() % 2 ? (int)(rng() % 20) : -1;
        if (edge) {
            const int ld = hidden + rng() % 5;
            bad = block<T, V, true>(rows, hidden, ld, rng() % V, arrays, stages, grid, b, late, lost);
        } else {
            const int h = (hidden + V - 1) / V * V;
            bad = block<T, V, false>(rows, h, h + V * (rng() % 2), 0, arrays, stages, grid, b, late, lost);
        }
        if (bad) std::printf("V=%d turn %d: %d\n", V, turn, bad);
    }
    return bad;
}

int main() {
    return many<__nv_bfloat16, 8>() | many<float, 4>();
}
"""


def cut_ring():
    text = open(SOURCE).read()
    a = text.index("// V elements as 32-bit words")
    b = text.index("template <typename O, int V, bool EDGE>\n__device__ __forceinline__ void write_window")
    c = text.index("constexpr int kMaxStages")
    d = text.index("// The weight's windows of a block")
    body = text[a:b] + text[c:d]
    body = body.replace("__device__ __forceinline__", "inline").replace("__device__ ", "")
    return re.sub(r"#pragma unroll.*", "", body)


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("row_ring")

    def go(body):
        src, exe = d / "ring.cpp", d / "ring"
        src.write_text(PRELUDE + body + MAIN)
        subprocess.run([gxx, "-std=c++17", "-O1", "-w", str(src), "-o", str(exe)], check=True)
        return subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)

    return go


def test_rows_come_as_they_lie_and_lost_copies_end_the_block(run):
    r = run(cut_ring())
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("right,wrong", [
    ("if (row >= rows || dead) return;", "if (row >= rows) return;"),
    ("if (!dead && !bounded_row_wait(&s.full[st], parity, err)) dead = true;",
     "bounded_row_wait(&s.full[st], parity, err);"),
    ("if (!dead) return;", "return;"),
    ("(n / (uint32_t)stages) & 1, err);", "(n / (uint32_t)stages + 1) & 1, err);"),
], ids=["fetches on", "waits on", "no drain", "drain of another turn"])
def test_planted_mistakes_are_reported(run, right, wrong):
    body = cut_ring()
    assert body.count(right) == 1
    assert run(body.replace(right, wrong)).returncode != 0
