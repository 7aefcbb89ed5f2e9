// Quantization to 8-bit floats (e4m3):
//
//   s = fl32(max|x| / 448),  code = e4m3(fl32(x / s)), nearest, ties to even
//
// per row and group of 128 columns (activations) or per block of 128 x 128
// (weights).  A group of zeros, or one whose scale underflows, has s = 0 and
// codes 0; a group with a NaN or an infinity has a NaN scale and NaN codes, so
// what is computed from it is NaN.  A subnormal scale is coarse enough for
// quotients beyond 448: they are clamped.
#include "fp8.h"
#include "kernels.h"

namespace w4a16 {

namespace {

constexpr uint32_t kAbs = 0x7FFFFFFFu, kInf = 0x7F800000u;

// The magnitude's bits order numbers, infinities and NaNs as integers do.
__device__ inline uint32_t magnitude(float v) { return __float_as_uint(v) & kAbs; }

__device__ inline float fp8_scale(uint32_t top) { return top >= kInf ? __uint_as_float(0x7FC00000u) : __uint_as_float(top) / kFp8Max; }

// four values of a group with the largest magnitude `top` and scale s as codes
__device__ inline uint32_t fp8_codes(float a, float b, float c, float d, float s, uint32_t top) {
    if (top >= kInf) return kFp8Nan * 0x01010101u;
    if (s == 0.0f) return 0;
    auto q = [&](float v) { return fminf(fmaxf(v / s, -kFp8Max), kFp8Max); };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q(a), q(b), 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(q(c), q(d), w, true));
}

// Eight consecutive values from p as FP32.
template <int DT>
__device__ inline void load8(const void* p, int64_t at, float (&v)[8]) {
    if constexpr (DT == 0) {
        const float4 a = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at)[0];
        const float4 b = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = to_f32<DT>(uint16_t(w[i]));
            v[2 * i + 1] = to_f32<DT>(uint16_t(w[i] >> 16));
        }
    }
}

__device__ inline uint32_t max8(const float (&v)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, magnitude(v[i]));
    return top;
}

template <int M>
__device__ inline uint32_t max_xor(uint32_t v) {
    return max(v, uint32_t(__builtin_amdgcn_ds_swizzle(int(v), 0x1F | (M << 10))));
}

// Rows: 16 lanes a group, 8 values a lane; GROUPS groups a lane, all loaded first.
constexpr int kRowGroups = 4;

template <int DT, int AF>
__global__ __launch_bounds__(256) void fp8_rows_kernel(Fp8QuantizeArgs a, uint32_t groups, uint32_t total) {
    const int sub = threadIdx.x % 16;
    const uint32_t first = blockIdx.x * uint32_t(16 * kRowGroups) + threadIdx.x / 16;
    float v[kRowGroups][8];
#pragma unroll
    for (int u = 0; u < kRowGroups; ++u) {
        const uint32_t at = min(first + 16 * u, total - 1);
        const uint32_t row = at / groups, g = at - row * groups;
        const int64_t in = int64_t(row) * a.ldx + int64_t(g) * kGroup + sub * 8;
        if constexpr (AF == kActFnNone) {
            load8<DT>(a.x, in, v[u]);
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(a.x) + in;
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            const uint4 gate = AF == kActFnSwiglu ? *reinterpret_cast<const uint4*>(p + a.k) : uint4{};
            const uint4 r = activate8<DT, AF>(x, gate);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[u][2 * i] = to_f32<DT>(uint16_t(w[i]));
                v[u][2 * i + 1] = to_f32<DT>(uint16_t(w[i] >> 16));
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kRowGroups; ++u) {
        const uint32_t at = first + 16 * u;
        const uint32_t top = max_xor<8>(max_xor<4>(max_xor<2>(max_xor<1>(max8(v[u])))));
        const float s = fp8_scale(top);
        const uint2 c = make_uint2(fp8_codes(v[u][0], v[u][1], v[u][2], v[u][3], s, top),
                                   fp8_codes(v[u][4], v[u][5], v[u][6], v[u][7], s, top));
        if (at < total) {
            *reinterpret_cast<uint2*>(a.codes + int64_t(at) * kGroup + sub * 8) = c;
            if (sub == 0) a.scales[at] = s;
        }
    }
}

// Blocks: one workgroup a block of 128 x 128, 16 rows at a time, everything in
// registers between the maximum and the codes.
template <int DT>
__global__ __launch_bounds__(256) void fp8_blocks_kernel(Fp8QuantizeArgs a, uint32_t groups) {
    __shared__ uint32_t tops[4];
    const int sub = threadIdx.x % 16, lane = threadIdx.x % 64;
    const int64_t block = blockIdx.x / groups, g = blockIdx.x % groups;
    float v[8][8];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int64_t row = min(block * 128 + u * 16 + int64_t(threadIdx.x / 16), a.m - 1);
        load8<DT>(a.x, row * a.ldx + g * kGroup + sub * 8, v[u]);
        top = max(top, max8(v[u]));
    }
    top = max_xor<16>(max_xor<8>(max_xor<4>(max_xor<2>(max_xor<1>(top)))));
    top = max(top, uint32_t(__shfl_xor(int(top), 32)));
    if (lane == 0) tops[threadIdx.x / 64] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    const float s = fp8_scale(top);
    if (threadIdx.x == 0) a.scales[blockIdx.x] = s;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int64_t row = block * 128 + u * 16 + threadIdx.x / 16;
        const uint2 c = make_uint2(fp8_codes(v[u][0], v[u][1], v[u][2], v[u][3], s, top),
                                   fp8_codes(v[u][4], v[u][5], v[u][6], v[u][7], s, top));
        if (row < a.m) *reinterpret_cast<uint2*>(a.codes + row * a.k + g * kGroup + sub * 8) = c;
    }
}

template <int DT, int AF>
hipError_t rows(const Fp8QuantizeArgs& a, hipStream_t stream) {
    const uint32_t groups = uint32_t(a.k / kGroup), total = uint32_t(a.m) * groups;
    const uint32_t grid = uint32_t(ceil_div(total, 16 * kRowGroups));
    fp8_rows_kernel<DT, AF><<<dim3(grid), dim3(256), 0, stream>>>(a, groups, total);
    return hipGetLastError();
}

template <int DT>
hipError_t rows_by_act(const Fp8QuantizeArgs& a, int act_fn, hipStream_t stream) {
    switch (act_fn) {
        case kActFnSwiglu: return rows<DT, kActFnSwiglu>(a, stream);
        case kActFnGeluTanh: return rows<DT, kActFnGeluTanh>(a, stream);
        default: return rows<DT, kActFnNone>(a, stream);
    }
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8QuantizeArgs& a, int dtype, int act_fn, hipStream_t stream) {
    if (dtype == kActBf16) return rows_by_act<kActBf16>(a, act_fn, stream);
    if (dtype == kActF16) return rows_by_act<kActF16>(a, act_fn, stream);
    return rows<0, kActFnNone>(a, stream);
}

hipError_t launch_fp8_quantize_blocks(const Fp8QuantizeArgs& a, int dtype, hipStream_t stream) {
    const uint32_t groups = uint32_t(a.k / kGroup), grid = uint32_t(ceil_div(a.m, int64_t(128))) * groups;
    if (dtype == kActBf16) fp8_blocks_kernel<kActBf16><<<dim3(grid), dim3(256), 0, stream>>>(a, groups);
    else if (dtype == kActF16) fp8_blocks_kernel<kActF16><<<dim3(grid), dim3(256), 0, stream>>>(a, groups);
    else fp8_blocks_kernel<0><<<dim3(grid), dim3(256), 0, stream>>>(a, groups);
    return hipGetLastError();
}

}  // namespace w4a16
