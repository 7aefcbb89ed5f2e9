// Host-side checks that the C entry points share (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"

namespace w4a16 {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// [lo, hi) byte ranges overlap?
inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    if (!a || !b || an == 0 || bn == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bn && b0 < a0 + an;
}

// Bytes from the first element of a [rows][cols] array with rows ld apart to its last one.
inline size_t span_bytes(int64_t rows, int64_t cols, int64_t ld, size_t elem) {
    if (rows <= 0 || cols <= 0) return 0;
    return (size_t(rows - 1) * size_t(ld) + size_t(cols)) * elem;
}

inline w4a16_status_t from_hip(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_EHIP; }

// the dtypes of activations
inline bool act_dtype(w4a16_dtype_t t) { return t == W4A16_BF16 || t == W4A16_F16; }

}  // namespace w4a16
