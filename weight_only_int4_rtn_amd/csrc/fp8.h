// Linear layer on 8-bit floats: arguments and launch plans of its kernels
// (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"

namespace w4a16 {

// Codes are e4m3 bytes (OCP: 3 bits behind the point, largest value 448, no
// infinities, NaN 0x7F).  Rows of x: [m][k] codes, FP32 scales [m][k / 128].
// Weights: [n][k] codes, FP32 scales [ceil(n / 128)][k / 128], one per block of
// 128 rows and 128 columns.  Both stay row-major: a lane's 32 bytes of an MFMA
// operand are two 16-byte pieces of one row, so no packing is needed, and a
// checkpoint's codes are used as they are.
constexpr float kFp8Max = 448.0f;
constexpr uint32_t kFp8Nan = 0x7F;

struct Fp8QuantizeArgs {
    const void* x;
    int64_t m, k, ldx;  // ldx: elements between rows
    uint8_t* codes;     // [m][k]
    float* scales;      // [m][k / 128]
};
// dtype of x: 0 (FP32, without an activation), kActBf16, kActF16; act_fn: ActFn,
// SwiGLU rows hold [up | gate], 2k values
hipError_t launch_fp8_quantize(const Fp8QuantizeArgs& a, int dtype, int act_fn, hipStream_t stream);
// scales [ceil(m / 128)][k / 128]
hipError_t launch_fp8_quantize_blocks(const Fp8QuantizeArgs& a, int dtype, hipStream_t stream);

struct Fp8LinearArgs {
    const uint8_t* x;
    const float* xs;
    int64_t m, k, ldx;
    const uint8_t* w;
    const float* ws;
    int64_t n;
    const uint16_t* bias;  // may be null
    uint16_t* y;
    int64_t ldy;
    unsigned* counters;  // zero before and after; one per output tile of a K split
    float* slots;        // FP32 tiles of a K split
};

struct Fp8Plan {
    int kind;           // 0: the kernel for at most 16 rows; else an index of the tiled kernel's shapes
    int bm, bn, waves;  // rows of x and output columns of a workgroup
    int64_t mtiles, ntiles;
    int splits, gps;    // parts of K, groups of 128 in each
    size_t workspace;   // FP32 tiles of a K split
};
Fp8Plan plan_fp8_linear(int64_t m, int64_t n, int64_t k);
hipError_t launch_fp8_linear(const Fp8LinearArgs& a, const Fp8Plan& p, int act, hipStream_t stream);

}  // namespace w4a16
