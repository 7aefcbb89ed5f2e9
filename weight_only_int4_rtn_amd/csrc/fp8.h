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

// ---------------------------------------------------------------------------
// Quantization of a group (device): 16 lanes hold it, eight values each.
// ---------------------------------------------------------------------------
// A magnitude's bits order numbers, infinities and NaNs as integers do; from kFp8Inf on it is not a number.
constexpr uint32_t kFp8Inf = 0x7F800000u;

__device__ inline float fp8_scale(uint32_t top) { return top >= kFp8Inf ? __uint_as_float(0x7FC00000u) : __uint_as_float(top) / kFp8Max; }

// four values of a group with the largest magnitude `top` and scale s as codes
__device__ inline uint32_t fp8_codes(float a, float b, float c, float d, float s, uint32_t top) {
    if (top >= kFp8Inf) return kFp8Nan * 0x01010101u;
    if (s == 0.0f) return 0;
    auto q = [&](float v) { return fminf(fmaxf(v / s, -kFp8Max), kFp8Max); };
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q(a), q(b), 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(q(c), q(d), w, true));
}
__device__ inline uint2 fp8_codes8(const float (&v)[8], float s, uint32_t top) {
    return make_uint2(fp8_codes(v[0], v[1], v[2], v[3], s, top), fp8_codes(v[4], v[5], v[6], v[7], s, top));
}

// Eight consecutive values from element `at` on as FP32, of dtype DT (0: FP32), activated; SwiGLU's gates lie k further.
template <int DT, int AF>
__device__ inline void fp8_load8(const void* p, int64_t at, int64_t k, float (&v)[8]) {
    if constexpr (DT == 0) {
        const float4 a = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at)[0];
        const float4 b = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint16_t* x = static_cast<const uint16_t*>(p) + at;
        uint4 r = *reinterpret_cast<const uint4*>(x);
        if constexpr (AF == kActFnSwiglu) r = activate8<DT, AF>(r, *reinterpret_cast<const uint4*>(x + k));
        if constexpr (AF == kActFnGeluTanh) r = activate8<DT, AF>(r, uint4{});
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = to_f32<DT>(uint16_t(w[i]));
            v[2 * i + 1] = to_f32<DT>(uint16_t(w[i] >> 16));
        }
    }
}

__device__ inline uint32_t fp8_top8(const float (&v)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return top;
}

template <int M>
__device__ inline uint32_t fp8_max_xor(uint32_t v) {
    return max(v, uint32_t(__builtin_amdgcn_ds_swizzle(int(v), 0x1F | (M << 10))));
}
// the largest magnitude of the group
__device__ inline uint32_t fp8_group_top(const float (&v)[8]) {
    return fp8_max_xor<8>(fp8_max_xor<4>(fp8_max_xor<2>(fp8_max_xor<1>(fp8_top8(v)))));
}

struct Fp8QuantizeArgs {
    const void* x;
    int64_t m, k, ldx;  // ldx: elements between rows
    uint8_t* codes;     // [m][k]
    float* scales;      // [m][k / 128], or by group [k / 128][m]
    bool by_group;      // (16-bit x)
};
// dtype of x: 0 (FP32, without an activation), kActBf16, kActF16; act_fn: ActFn,
// SwiGLU rows hold [up | gate], 2k values
hipError_t launch_fp8_quantize(const Fp8QuantizeArgs& a, int dtype, int act_fn, hipStream_t stream);
// scales [ceil(m / 128)][k / 128]
hipError_t launch_fp8_quantize_blocks(const Fp8QuantizeArgs& a, int dtype, hipStream_t stream);

struct Fp8LinearArgs {
    const uint8_t* x;   // codes, or (few rows) 16-bit values that the kernel quantizes itself
    const float* xs;    // of row i, group g at i * rs + g * gs
    int64_t rs, gs;
    int64_t m, k, ldx;  // ldx: elements
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
    int bm, bn;         // rows of x and output columns of a workgroup
    int64_t mtiles, ntiles;
    int splits, gps;    // parts of K, groups of 128 in each
    size_t workspace;   // FP32 tiles of a K split
};
Fp8Plan plan_fp8_linear(int64_t m, int64_t n, int64_t k);
// Whether the kernel quantizes 16-bit x itself: act_fn is then the activation, else it is not looked at and x holds codes.
bool fp8_linear_quantizes(int64_t m, const Fp8Plan& p);
hipError_t launch_fp8_linear(const Fp8LinearArgs& a, const Fp8Plan& p, int act, bool quantize, int act_fn, hipStream_t stream);

}  // namespace w4a16
