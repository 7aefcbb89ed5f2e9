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

// Rows: 16 lanes a group, 8 values a lane; N groups a lane, all loaded first.
template <int DT, int AF, int N, bool BY_GROUP>
__global__ __launch_bounds__(256) void fp8_rows_kernel(Fp8QuantizeArgs a, uint32_t groups, uint32_t total) {
    const int sub = threadIdx.x % 16;
    const uint32_t first = blockIdx.x * uint32_t(16 * N) + threadIdx.x / 16;
    float v[N][8];
    uint32_t by_group[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const uint32_t at = min(first + 16 * u, total - 1);
        const uint32_t row = at / groups, g = at - row * groups;
        const int64_t in = int64_t(row) * a.ldx + int64_t(g) * kGroup + sub * 8;
        fp8_load8<DT, AF>(a.x, in, a.k, v[u]);
        by_group[u] = g * uint32_t(a.m) + row;
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const uint32_t at = first + 16 * u;
        const uint32_t top = fp8_group_top(v[u]);
        const float s = fp8_scale(top);
        const uint2 c = fp8_codes8(v[u], s, top);
        if (at < total) {
            *reinterpret_cast<uint2*>(a.codes + int64_t(at) * kGroup + sub * 8) = c;
            if (sub == 0) a.scales[BY_GROUP ? by_group[u] : at] = s;
        }
    }
}

// Blocks: one workgroup a block of 128 x 128, 16 rows at a time, everything in
// registers between the maximum and the codes.  Large weights are bound by HBM:
// 28672 x 8192 from bf16 125 to 150 us (705 MB, 4.7 to 5.6 TB/s), from FP32 206 (1.2
// GB, 5.7 TB/s), 32768 x 2048 from bf16 40 us; 2560 x 2048 7.4 us, 320 workgroups and
// two latencies.
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
        fp8_load8<DT, kActFnNone>(a.x, row * a.ldx + g * kGroup + sub * 8, 0, v[u]);
        top = max(top, fp8_top8(v[u]));
    }
    top = fp8_max_xor<16>(fp8_max_xor<8>(fp8_max_xor<4>(fp8_max_xor<2>(fp8_max_xor<1>(top)))));
    top = max(top, uint32_t(__shfl_xor(int(top), 32)));
    if (lane == 0) tops[threadIdx.x / 64] = top;
    __syncthreads();
    top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    const float s = fp8_scale(top);
    if (threadIdx.x == 0) a.scales[blockIdx.x] = s;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        const int64_t row = block * 128 + u * 16 + threadIdx.x / 16;
        const uint2 c = fp8_codes8(v[u], s, top);
        if (row < a.m) *reinterpret_cast<uint2*>(a.codes + row * a.k + g * kGroup + sub * 8) = c;
    }
}

// Below so many groups a lane takes one, more waves the sooner; above it four, whose loads fill memory's queue.  us on one and
// on four, rows x columns: 1 x 2048 2.3 and 3.7, 777 x 4096 4.7 and 6.1, 4096 x 4096 12.9 and 14.3, 4096 x 16384 (524288
// groups) 44.6 and 45.6, 8192 x 16384 89 and 84 (4.79 TB/s, a large copy's rate); with SwiGLU 2048 x 4096 11.5 and 13.2.  (In a run of the
// last calls 78 to 86 us, and 95 to 114 while the card's power control settles.)  tanh-GELU is bound by its arithmetic: 2048 x
// 8192 18.6 us, without it 13.3.
constexpr uint32_t kOneGroup = 600000;

template <int DT, int AF, bool BY_GROUP>
hipError_t rows(const Fp8QuantizeArgs& a, hipStream_t stream) {
    const uint32_t groups = uint32_t(a.k / kGroup), total = uint32_t(a.m) * groups;
    if (total < kOneGroup) fp8_rows_kernel<DT, AF, 1, BY_GROUP><<<dim3(uint32_t(ceil_div(total, 16))), dim3(256), 0, stream>>>(a, groups, total);
    else fp8_rows_kernel<DT, AF, 4, BY_GROUP><<<dim3(uint32_t(ceil_div(total, 64))), dim3(256), 0, stream>>>(a, groups, total);
    return hipGetLastError();
}

template <int DT, int AF>
hipError_t rows(const Fp8QuantizeArgs& a, hipStream_t stream) {
    return a.by_group ? rows<DT, AF, true>(a, stream) : rows<DT, AF, false>(a, stream);
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
    return rows<0, kActFnNone, false>(a, stream);
}

hipError_t launch_fp8_quantize_blocks(const Fp8QuantizeArgs& a, int dtype, hipStream_t stream) {
    const uint32_t groups = uint32_t(a.k / kGroup), grid = uint32_t(ceil_div(a.m, int64_t(128))) * groups;
    if (dtype == kActBf16) fp8_blocks_kernel<kActBf16><<<dim3(grid), dim3(256), 0, stream>>>(a, groups);
    else if (dtype == kActF16) fp8_blocks_kernel<kActF16><<<dim3(grid), dim3(256), 0, stream>>>(a, groups);
    else fp8_blocks_kernel<0><<<dim3(grid), dim3(256), 0, stream>>>(a, groups);
    return hipGetLastError();
}

}  // namespace w4a16
