"""The ring of rows of a team of warps (TeamRing in csrc/block_rows.cuh), compiled here
on the host from the library's own source, over barriers and bulk copies that land in
any order.

Every thread has to read its windows as they lie in memory, with zeros outside the row,
for rows of every phase and length, teams of one and of several warps, and rings of one
stage and more.  A copy that never lands makes the threads' waits run out, once each:
the ring then fetches nothing more, and sees its other copies in flight land before the
block's exit.
"""
import os
import re
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "collective_datapath_atom_gb300", "csrc")
if HERE not in sys.path:
    sys.path.insert(0, HERE)

from test_row_ring import PRELUDE  # noqa: E402

TEAM = r"""
static uint4 make_uint4(uint32_t x, uint32_t y, uint32_t z, uint32_t w) { return {x, y, z, w}; }
struct TeamPlan { int warps, stages, arrays; };
struct Team {
    int index, warps, thread;
    int threads() const { return warps * 32; }
    int window(int items) const { return (thread & ~31) * items + (thread & 31); }
    void sync() const {}
};
static std::vector<unsigned char> memory;
static unsigned char *smem() {
    unsigned char *p = memory.data();
    while ((uintptr_t)p % 16) ++p;
    return p;
}
"""

MAIN = r"""
template <typename T>
struct P {
    const void *src[5];
    size_t ld[5], rows;
    unsigned long long *err;
};

/* one team's walk, its threads one after another between the barriers */
template <typename T, int V, int ITEMS, bool EDGE>
static int team(int rows, int hidden, int ld, int off, int arrays, int stages, int grid, int b, int warps,
                int index, int teams, bool hold, int lost) {
    using Ring = TeamRing<T, V, 5, ITEMS, EDGE, P<T>>;
    bars.clear(); flying.clear();
    errors = fault = copies = 0; now = 1; drop = lost;
    blockIdx.x = b;
    std::vector<std::vector<T>> src(arrays);
    unsigned value = 1;
    std::vector<T *> from(arrays);
    P<T> p{};
    for (int a = 0; a < arrays; ++a) {
        src[a].resize((size_t)rows * ld + off + 16 / sizeof(T));
        T *base = src[a].data();
        while ((uintptr_t)base % 16) ++base;
        from[a] = base + off;
        for (size_t i = 0; i + (base - src[a].data()) < src[a].size(); ++i) {
            const unsigned v = value++;
            std::memcpy(&base[i], &v, sizeof(T));
        }
        p.src[a] = from[a];
        p.ld[a] = ld;
    }
    unsigned long long err = 0;
    p.rows = rows;
    p.err = &err;
    const int phase = EDGE ? (off % V + b * (ld % V)) % V : 0, threads = 32 * warps;
    const uint32_t before = 64;      /* the vectors, which no ring may touch */
    memory.assign((size_t)before + (size_t)teams * stages * arrays * ITEMS * threads * 16 + 64, 0xAB);
    uint64_t full[4];
    const size_t row0 = b + (size_t)index * grid, step = (size_t)teams * grid;
    std::vector<Team> who;
    for (int t = 0; t < threads; ++t) who.push_back(Team{index, warps, t});
    std::vector<Ring> ring;
    for (int t = 0; t < threads; ++t)
        ring.emplace_back(p, TeamPlan{warps, stages, arrays}, who[t], full, before, phase, hidden, row0, step);
    for (Ring &r : ring) r.clear();
    for (Ring &r : ring) r.start();
    uint32_t issued_dead = 0;
    bool dead = false;
    uint64_t died = 0;
    for (size_t row = row0; row < (size_t)rows; row += step) {
        ring[0].wait();   /* the others wait at the same time, and see the same */
        for (Ring &r : ring) r.dead = ring[0].dead;
        if (ring[0].dead && !dead) { dead = true; issued_dead = ring[0].issued; died = now; }
        auto check = [&] {
            for (int t = 0; t < threads && !dead; ++t)
                for (int a = 0; a < arrays; ++a)
                    for (int i = 0; i < ITEMS; ++i) {
                        const Window<T, V> k = ring[t].window(a, i);
                        for (int j = 0; j < V; ++j) {
                            const int e = (who[t].window(ITEMS) + 32 * i) * V - phase + j;
                            const uint32_t want = e >= 0 && e < hidden ? bits_of(from[a] + row * ld + e) : 0;
                            const float f = k.at(j);
                            const uint32_t got = sizeof(T) == 4 ? __float_as_uint(f) : __float_as_uint(f) >> 16;
                            if (got != want) fault |= 4;
                        }
                    }
        };
        check();
        for (Ring &r : ring) r.settle();         /* a barrier */
        if (!hold) check();                      /* (read again, and a second barrier) */
        for (Ring &r : ring) r.refill();
        if (EDGE && stages == 1)
            for (Ring &r : ring) r.settle();
        for (Ring &r : ring) r.next();
    }
    if (dead && ring[0].issued > issued_dead + 1) fault |= 8;   /* fetched on (one was pending) */
    ring[0].drain();
    for (const Copy &c : flying) if (!c.dropped) fault |= 16;   /* a copy outlives the block */
    const bool short_of_one = lost >= 0 && lost < copies;
    if (slow ? short_of_one && errors == 0 : short_of_one != (errors > 0)) fault |= 32;
    /* the drain waits: two seconds each, of a clock that is read every 64th look, 0.64 s here */
    if (dead && now - died > (uint64_t)stages * 3300000000ull) fault |= 64;
    for (uint32_t i = 0; i < before; ++i) if (smem()[i] != 0xAB) fault |= 128;
    return fault;
}

template <typename T, int V, int ITEMS>
static int many() {
    int bad = 0;
    for (int turn = 0; turn < 400 && !bad; ++turn) {
        rng.seed(turn);
        const int warps = 1 + rng() % 2, room = 32 * warps * ITEMS * V - 2 * V;
        const int hidden = rng() % 3 ? 1 + rng() % room : 1 + rng() % 20;
        const int arrays = 1 + rng() % 5, stages = 1 + rng() % 4, teams = 1 + rng() % 2;
        const bool edge = rng() % 3 != 0, hold = rng() % 2;
        const int grid = V * (1 + rng() % 2), rows = grid + rng() % 60, b = rng() % grid;
        slow = rng() % 4 == 0;
        const int lost = rng() % 2 ? (int)(rng() % 20) : -1;
        if (edge) {
            const int ld = hidden + rng() % 5;
            bad = team<T, V, ITEMS, true>(rows, hidden, ld, rng() % V, arrays, stages, grid, b, warps,
                                          rng() % teams, teams, hold, lost);
        } else {
            const int h = (hidden + V - 1) / V * V;
            bad = team<T, V, ITEMS, false>(rows, h, h + V * (rng() % 2), 0, arrays, stages, grid, b, warps,
                                           rng() % teams, teams, hold, lost);
        }
        if (bad) std::printf("V=%d ITEMS=%d turn %d: %d\n", V, ITEMS, turn, bad);
    }
    return bad;
}

int main() {
    return many<__nv_bfloat16, 8, 2>() | many<float, 4, 2>() | many<float, 4, 4>();
}
"""


def host(text):
    text = text.replace("__device__ __forceinline__", "inline").replace("__device__ ", "")
    return re.sub(r"#pragma unroll.*", "", text)


def cut():
    rows = open(os.path.join(CSRC, "rms_norm.cu")).read()
    a = rows.index("// V elements as 32-bit words")
    b = rows.index("template <typename O, int V, bool EDGE>\n__device__ __forceinline__ void write_window")
    c = rows.index("// Wait for a stage, two seconds at most.")
    d = rows.index("// A block's rows on their way through shared memory")
    team = open(os.path.join(CSRC, "block_rows.cuh")).read()
    e = team.index("template <typename T, int V>\n__device__ __forceinline__ Window<T, V> staged_window")
    f = team.index("// What the warps of a team add up")
    g = team.index("// A team's ring of rows")
    h = team.index("// The vectors of a block, in windows")
    return host(rows[a:b] + rows[c:d]) + TEAM + host(team[e:f] + team[g:h])


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("team_ring")

    def go(body):
        src, exe = d / "ring.cpp", d / "ring"
        src.write_text(PRELUDE + body + MAIN)
        subprocess.run([gxx, "-std=c++17", "-O1", "-w", str(src), "-o", str(exe)], check=True)
        return subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)

    return go


def test_rows_come_as_they_lie_and_lost_copies_end_the_block(run):
    r = run(cut())
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("right,wrong", [
    ("pending = next_row < p.rows && !dead;", "pending = next_row < p.rows;"),
    ("if (!dead && !bounded_row_wait(&full[st], parity, p.err)) dead = true;",
     "bounded_row_wait(&full[st], parity, p.err);"),
    ("if (!dead) return;", "return;"),
    ("(n / (uint32_t)stages) & 1, p.err);", "(n / (uint32_t)stages + 1) & 1, p.err);"),
    ("if (w < first || w >= behind)", "if (w < first)"),
    ("(last ? whole * V : 0) + n % V - phase", "(last ? whole * V : 0) + n % V"),
    ("[phase + place[k]] = end[k];", "[place[k]] = end[k];"),
], ids=["fetches on", "waits on", "no drain", "drain of another turn", "no zeros behind", "ends out of phase",
        "ends elsewhere"])
def test_planted_mistakes_are_reported(run, right, wrong):
    body = cut()
    assert body.count(right) == 1
    assert run(body.replace(right, wrong)).returncode != 0
