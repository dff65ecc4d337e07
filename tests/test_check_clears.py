"""purlin_check's writes to the context's memory, on the host: api.cpp and
layers_api.cpp compiled against a fake of the CUDA runtime that records them.

After an error, purlin_check clears the error word and the counters of the grouped
products' joins.  On a GPU a plain memset runs on the default stream and returns
before it is done, so it can land in the middle of the next call on a context's own
non-blocking stream.  The fake carries out work on a stream only when something
waits for that stream, or when later work is put on it, as late as the real one may.
"""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "collective_datapath_atom_gb300", "csrc")

DRIVER = r"""
#include <cuda_runtime.h>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <map>
#include <vector>
#include "host.h"
#include "layers.h"

/* ---- the fake runtime: work waits on its stream */
static std::map<cudaStream_t, std::vector<std::function<void()>>> queued;
static void run(cudaStream_t s) {
    auto work = std::move(queued[s]);
    queued[s].clear();
    for (auto &f : work) f();
}
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, enum cudaDeviceAttr a, int) {
    *v = a == cudaDevAttrMultiProcessorCount ? 152 : 227 * 1024;
    return cudaSuccess;
}
cudaError_t cudaMalloc(void **p, size_t n) { *p = std::calloc(n, 1); return cudaSuccess; }
cudaError_t cudaFree(void *p) { std::free(p); return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void *p, int v, size_t n, cudaStream_t s) {
    queued[s].push_back([=] { std::memset(p, v, n); });
    return cudaSuccess;
}
cudaError_t cudaMemset(void *p, int v, size_t n) { return cudaMemsetAsync(p, v, n, nullptr); }
cudaError_t cudaMemcpyAsync(void *d, const void *s, size_t n, enum cudaMemcpyKind, cudaStream_t st) {
    queued[st].push_back([=] { std::memcpy(d, s, n); });
    return cudaSuccess;
}
cudaError_t cudaMemcpy(void *d, const void *s, size_t n, enum cudaMemcpyKind) {
    run(nullptr);
    std::memcpy(d, s, n);
    return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t s) { run(s); return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, enum cudaStreamCaptureStatus *st) {
    *st = cudaStreamCaptureStatusNone;
    return cudaSuccess;
}
}
namespace purlin {
cudaError_t configure_kernels(int) { return cudaSuccess; }
cudaError_t configure_vcounts(int) { return cudaSuccess; }
}

int main() {
    const cudaStream_t own = reinterpret_cast<cudaStream_t>(0x77);   /* non-blocking */
    purlin_ctx *ctx = nullptr;
    if (purlin_init(1, own, &ctx) != PURLIN_OK) return 2;
    for (int turn = 0; turn < 2; ++turn) {
        /* a call that gave up: its error, and counters part-way */
        ctx->err[0] = PURLIN_ERR_TIMEOUT;
        for (int i = 0; i < purlin::kJoinCounters; ++i) ctx->arrived[i] = 3;
        if (purlin_check(ctx) != PURLIN_ERR_TIMEOUT) return 3;
        /* the next call on the context's stream counts, and records an error of its own */
        queued[own].push_back([=] {
            for (int i = 0; i < purlin::kJoinCounters; ++i) {
                if (ctx->arrived[i] != 0) std::exit(4);    /* it found counters part-way */
                ctx->arrived[i] = 1;
            }
            if (ctx->err[0] != 0) std::exit(5);
            ctx->err[0] = PURLIN_ERR_INVALID_ARG;
        });
        run(own);
        run(nullptr);   /* whatever is still on the default stream lands now */
        for (int i = 0; i < purlin::kJoinCounters; ++i)
            if (ctx->arrived[i] != 1) return 6;            /* cleared in the middle of a call */
        if (purlin_check(ctx) != PURLIN_ERR_INVALID_ARG) return 7;   /* its error was lost */
        run(own);
        run(nullptr);
        if (purlin_check(ctx) != PURLIN_OK) return 8;
    }
    std::printf("ok\n");
    return purlin_finalize(ctx) == PURLIN_OK ? 0 : 9;
}
"""


def test_clears_stay_on_the_context_s_stream(tmp_path):
    gxx = shutil.which("g++")
    cuda = "/usr/local/cuda/include"
    if gxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("no host C++ compiler or CUDA headers")
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    # what the driver does not reach (kernels, launches) stays unresolved
    subprocess.run([gxx, "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                    "-I", cuda, str(src), os.path.join(CSRC, "api.cpp"),
                    os.path.join(CSRC, "layers_api.cpp"), os.path.join(CSRC, "plan.cpp"),
                    "-Wl,--unresolved-symbols=ignore-all", "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert (r.returncode, r.stdout) == (0, "ok\n")
