// layers.h -- host-side interface to the layer operators' kernels: the RMS
// norm (rms_norm.cu) and the products grouped by expert (grouped.cu).
// Internal to the library.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "../../include/purlin.h"

namespace purlin {

// Lets one kernel's dynamic shared memory grow, once on each device: the attribute
// belongs to the device that is current, and a call that failed is made again.
class SharedMemoryLimit {
public:
    template <typename K>
    cudaError_t raise(K *kernel, int bytes) {
        int device = 0;
        cudaError_t e = cudaGetDevice(&device);
        if (e != cudaSuccess) return e;
        const uint64_t bit = device < 64 ? 1ull << device : 0;   // past 64 devices: every time
        if (raised_.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) raised_.fetch_or(bit, std::memory_order_acq_rel);
        return e;
    }

private:
    std::atomic<uint64_t> raised_{0};
};

// ------------------------------------------------------------- RMS norm --

struct NormArgs {
    const void *x = nullptr;
    const void *residual = nullptr;   // or null
    const void *weight = nullptr;
    void *y = nullptr;
    void *total = nullptr;            // or null
    float *scales = nullptr;          // e4m3 output only
    size_t ldx = 0, ldr = 0, ldy = 0, ldt = 0;
    size_t rows = 0, hidden = 0;
    float eps = 0;
    int dtype = 0, out_dtype = 0;
    int sms = 0;
    unsigned long long *err = nullptr;
    cudaStream_t stream = nullptr;
};

struct NormBackwardArgs {
    const void *dy = nullptr;
    const void *total = nullptr;
    const void *weight = nullptr;
    const void *dtotal = nullptr;   // or null
    void *dx = nullptr;
    float *dweight = nullptr;
    float *partial = nullptr;       // norm_backward_workspace() bytes
    size_t lddy = 0, ldt = 0, lddt = 0, lddx = 0;
    size_t rows = 0, hidden = 0;
    float eps = 0;
    int dtype = 0;
    int sms = 0;
    unsigned long long *err = nullptr;
    cudaStream_t stream = nullptr;
};

cudaError_t launch_norm(const NormArgs &a);
size_t norm_backward_workspace(const NormBackwardArgs &a);
cudaError_t launch_norm_backward(const NormBackwardArgs &a);

// ------------------------------------------------------ grouped products --

// What a grouped product computes: out[j][i] = sum over k of A[i][k] B[j][k].
//   kGroupedNK    A = weights N x K, B = rows            (i: channel, j: row)
//   kGroupedKN    A = weights K x N, B = rows            (i: channel, j: row)
//   kGroupedGrad  A = x, B = dy, k over the group's rows (i: column of x, j: column of dy)
enum GroupedMode : int { kGroupedNK = 0, kGroupedKN = 1, kGroupedGrad = 2 };

struct GroupedArgs {
    int mode = 0;
    const void *x = nullptr;     // rows x k (kGroupedGrad: the forward pass's input)
    const void *w = nullptr;     // weights (kGroupedGrad: dy, rows x n)
    void *y = nullptr;           // rows x n (kGroupedGrad: groups x n x k)
    const float *x_scales = nullptr;   // e4m3 only
    const float *w_scales = nullptr;
    const int64_t *begin = nullptr;    // device
    const int64_t *count = nullptr;    // device
    size_t ldx = 0, ldw = 0, ldy = 0;
    int groups = 0;
    size_t rows = 0, n = 0, k = 0;
    int dtype = 0;
    int sms = 0;
    float *partial = nullptr;       // grouped_workspace(sms) bytes
    unsigned *arrived = nullptr;    // kJoinCounters, zero between launches
    unsigned long long *err = nullptr;
    cudaStream_t stream = nullptr;
};

constexpr int kMaxGroups = PURLIN_MAX_GROUPS;
constexpr int kJoinCounters = 16384;         // eight writers a CTA, 2048 CTAs
constexpr size_t kGroupedRowTile = 32;       // the narrowest tile's rows, and its channels
constexpr size_t kGroupedChannelTile = 128;

size_t grouped_workspace(int sms);

cudaError_t launch_grouped(const GroupedArgs &a);

}  // namespace purlin
