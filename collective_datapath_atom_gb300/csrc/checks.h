// checks.h -- argument checks that the layer operators' entry points share
// (layers_api.cpp, experts_api.cpp, block_api.cpp).  Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "../../include/purlin.h"

namespace purlin {
namespace host {

constexpr size_t kMaxExtent = 0x7FFFF000;         // rows, columns: 32-bit coordinates, a tile past the end too
constexpr size_t kMaxPitch = (size_t)1 << 35;     // elements

inline int size_of(int dtype) { return dtype == PURLIN_F32 ? 4 : dtype == PURLIN_BF16 ? 2 : 1; }

// A rows x cols matrix in memory, rows `pitch` bytes apart.
struct Matrix {
    const void *p = nullptr;
    size_t rows = 0, width = 0, pitch = 0;   // width and pitch in bytes
};

inline Matrix matrix(const void *p, size_t rows, size_t cols, size_t ld, int dtype) {
    return {p, p ? rows : 0, cols * (size_t)size_of(dtype), ld * (size_t)size_of(dtype)};
}

// Whether two matrices share a byte.  Two column ranges of one pitched buffer
// (equal pitches) share none although their extents interleave.
inline bool overlap(const Matrix &a, const Matrix &b) {
    if (a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t a1 = a0 + (a.rows - 1) * a.pitch + a.width;
    const uintptr_t b1 = b0 + (b.rows - 1) * b.pitch + b.width;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a.pitch != b.pitch) return true;
    const size_t d = b0 >= a0 ? (b0 - a0) % a.pitch : (a.pitch - (a0 - b0) % a.pitch) % a.pitch;
    return !(d >= a.width && d + b.width <= a.pitch);
}

inline bool any_overlap(const Matrix &out, std::initializer_list<Matrix> others) {
    for (const Matrix &m : others)
        if (overlap(out, m)) return true;
    return false;
}

// The same elements in the same places: allowed where a thread reads an
// element before it writes it.
inline bool same(const Matrix &a, const Matrix &b) {
    return a.p == b.p && a.pitch == b.pitch && a.width == b.width && a.rows == b.rows;
}

inline bool misaligned(const void *p, size_t to) {
    return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

inline purlin_status done(cudaError_t e) { return e == cudaSuccess ? PURLIN_OK : PURLIN_ERR_CUDA; }

inline bool bad_ld(size_t ld, size_t cols) { return ld < cols || ld > kMaxPitch; }

}  // namespace host
}  // namespace purlin
