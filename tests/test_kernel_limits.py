"""A kernel's shared-memory limit is raised once on every device (SharedMemoryLimit
in csrc/layers.h), on the host against a fake of the two runtime calls: the
attribute belongs to the current device, and a call that fails is made again."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "collective_datapath_atom_gb300", "csrc")

DRIVER = r"""
#include <cstdio>
#include <map>
#include "layers.h"
static int current = 0, asked = 0;
static cudaError_t answer = cudaSuccess;
static std::map<int, int> limit;   /* of the kernel, by device */
extern "C" cudaError_t cudaGetDevice(int *d) { *d = current; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, enum cudaFuncAttribute, int v) {
    ++asked;
    if (answer == cudaSuccess) limit[current] = v;
    return answer;
}
static void kernel(int) {}
static cudaError_t launch() {   /* as a launch does */
    static purlin::SharedMemoryLimit l;
    return l.raise(kernel, 200 * 1024);
}
int main() {
    answer = cudaErrorInvalidValue;
    if (launch() == cudaSuccess) return 1;          /* a failure is reported */
    answer = cudaSuccess;
    if (launch() != cudaSuccess || limit[0] != 200 * 1024) return 2;   /* and not for good */
    for (int d : {1, 0, 3, 70, 1, 0, 3, 70}) {
        current = d;
        if (launch() != cudaSuccess || limit[d] != 200 * 1024) return 3;
    }
    if (asked != 2 + 2 + 2) return 4;               /* once a device; a 71st every time */
    std::printf("ok\n");
    return 0;
}
"""


def test_limits_are_raised_on_every_device(tmp_path):
    gxx = shutil.which("g++")
    cuda = "/usr/local/cuda/include"
    if gxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime_api.h")):
        pytest.skip("no host C++ compiler or CUDA headers")
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, "-I", cuda, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert (r.returncode, r.stdout) == (0, "ok\n")


@pytest.mark.parametrize("unit", ["rms_norm.cu", "grouped.cu"])
def test_no_launch_keeps_an_attribute_s_result_for_the_process(unit):
    text = open(os.path.join(CSRC, unit)).read()
    assert "cudaFuncSetAttribute" not in text and "limit.raise(" in text
    assert not re.search(r"static\s+const\s+cudaError_t", text)
