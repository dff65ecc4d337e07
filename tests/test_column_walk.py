"""The walk of a writer warp over an accumulator's columns (walk_columns in
csrc/tensor.cuh), compiled here on the host from the library's own source.

Loads of tensor memory are asynchronous: each that a warp issues has to be waited
for before the warp gives the accumulator back, or its registers are used for
something else.  The walk runs here with loads, waits and stores that record
themselves, for every tile width and either half of the warps.  The planted
mistake is the walk that fetches its first columns whether it has any or not.
"""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
SOURCE = os.path.join(os.path.dirname(HERE), "collective_datapath_atom_gb300", "csrc", "tensor.cuh")

MAIN = r"""
#include <cstdio>
int main() {
    int bad = 0;
    for (int half = 0; half < 2; ++half)
        for (int nj = 1; nj <= 256; ++nj) {
            int flying = -1, landed = -1, next = 16 * half;
            walk_columns(16 * half, 32, nj,
                [&](int c) {
                    if (flying >= 0 || c >= nj || c + 16 > (nj + 15) / 16 * 16) bad |= 1;
                    flying = c;
                },
                [&] {
                    if (flying < 0) bad |= 2;
                    landed = flying;
                    flying = -1;
                },
                [&](int c) {
                    if (c != landed || c != next) bad |= 4;
                    next += 32;
                });
            if (flying >= 0) bad |= 8;      /* a load that nothing waited for */
            if (next < nj) bad |= 16;       /* columns left out */
        }
    std::printf("%d\n", bad);
    return 0;
}
"""


def cut_walk():
    text = open(SOURCE).read()
    start = text.index("template <typename Fetch, typename Wait, typename Put>")
    body = text[start:text.index("\n}\n", start) + 3]
    body = body.replace("__device__ __forceinline__", "static inline")
    return re.sub(r"#pragma unroll.*", "", body)


@pytest.fixture(scope="module")
def faults(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("column_walk")

    def go(body):
        src, exe = d / "walk.cpp", d / "walk"
        src.write_text(body + MAIN)
        subprocess.run([gxx, "-std=c++17", "-O1", str(src), "-o", str(exe)], check=True)
        return int(subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout)

    return go


def test_every_load_is_waited_for(faults):
    assert faults(cut_walk()) == 0


def test_a_first_load_without_columns_is_reported(faults):
    planted = cut_walk().replace("if (first >= end) return;", "")
    assert planted != cut_walk()
    assert faults(planted) & 8
