// Append to the 4-bit paged cache (kv4.h) and read back from it.
//
// Append takes the fused projection's rows [q heads | k heads | v heads],
// rotates queries and keys by the token's position, quantizes keys and values
// round-to-nearest to INT4 with one FP32 scale per token, head and group of W
// channels (the weights' quantizer), and stores them at the token's slot.
#include "kv4.h"

namespace w4a16 {

namespace {

// The rotation's products and sums are single FP32 operations, not fused:
// the stored codes then depend on the inputs and the table alone and equal
// those of any implementation of the formula in IEEE FP32.
#pragma clang fp contract(off)
__device__ inline void rotate(float x, float y, float c, float s, float& rx, float& ry) {
    const float a = x * c, b = y * s, d = y * c, e = x * s;
    rx = a - b;
    ry = d + e;
}
#pragma clang fp contract(on)

template <int ACT>
__device__ inline void widen8(uint4 raw, float v[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = to_f32<ACT>(uint16_t(w[i] & 0xFFFFu));
        v[2 * i + 1] = to_f32<ACT>(uint16_t(w[i] >> 16));
    }
}

template <int ACT>
__device__ inline uint4 narrow8(const float v[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = uint32_t(from_f32<ACT>(v[2 * i])) | (uint32_t(from_f32<ACT>(v[2 * i + 1])) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread owns 8 channels of one head of one token (16 bytes in).  The W/8
// threads of a scale group are adjacent lanes.  Grid: x = token, y = parts of
// 256 threads of the row.
template <int ACT, int D>
__global__ __launch_bounds__(256) void kv4_append_kernel(Kv4AppendArgs a) {
    constexpr int W = kv4_width(D), NB = kv4_blocks(D);
    const int64_t t = blockIdx.x;
    const int part = blockIdx.y * 256 + threadIdx.x;
    const int head = part / (D / 8), d0 = part % (D / 8) * 8;
    const int heads = a.heads + 2 * a.kv_heads;
    if (head >= heads) return;  // whole heads: a scale group's lanes leave together

    const uint16_t* row = a.qkv + t * a.ldqkv + int64_t(head) * D;
    float v[8];
    widen8<ACT>(*reinterpret_cast<const uint4*>(row + d0), v);

    const bool is_v = head >= a.heads + a.kv_heads;
    bool known = true;
    if (a.rope) {
        const int64_t pos = a.positions[t];
        known = pos >= 0 && pos < a.rope_len;
        if (!is_v && d0 < a.rot) {
            const float* cs = a.rope + (known ? pos : 0) * a.rot;
            const int half = a.rot / 2;
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    rotate(v[2 * i], v[2 * i + 1], cs[d0 / 2 + i], cs[half + d0 / 2 + i], v[2 * i], v[2 * i + 1]);
            } else {
                const bool low = d0 < half;
                float w[8];
                widen8<ACT>(*reinterpret_cast<const uint4*>(row + (low ? d0 + half : d0 - half)), w);
                const float* c = cs + (low ? d0 : d0 - half);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float x, y;
                    if (low) rotate(v[i], w[i], c[i], c[half + i], x, y);
                    else rotate(w[i], v[i], c[i], c[half + i], x, y);
                    v[i] = low ? x : y;
                }
            }
        }
    }
    if (head < a.heads) {
        if (!known) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(0x7FC00000u);
        }
        *reinterpret_cast<uint4*>(a.q_out + (t * a.heads + head) * D + d0) = narrow8<ACT>(v);
        return;
    }
    const int64_t slot = a.slots[t];
    const bool stored = known && slot >= 0 && slot < a.pages * a.page;

    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = fmaxf(amax, lane_xor<1>(amax));
    amax = fmaxf(amax, lane_xor<2>(amax));
    amax = fmaxf(amax, lane_xor<4>(amax));
    if constexpr (W == 128) amax = fmaxf(amax, lane_xor<8>(amax));
    if (!stored) return;
    const float s = amax / 7.0f;
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float r = s != 0.0f ? rintf(v[i] / s) : 0.0f;
        r = fminf(fmaxf(r, -8.0f), 7.0f);
        u[i] = uint32_t(int(r) + 8);
    }

    const int64_t pg = slot / a.page;
    const int tok = int(slot - pg * a.page);
    const int kh = head - a.heads - (is_v ? a.kv_heads : 0);
    uint8_t* region = a.pool + (pg * a.kv_heads + kh) * kv4_region(a.page, D);
    const int b = d0 / W, e = d0 % W, tc = tok % kKvChunkTokens;
    const int64_t chunk = (int64_t(tok / kKvChunkTokens) * NB + b) * (8 * W);
    if (!is_v) {
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) word |= (u[2 * i] << (4 * i)) | (u[2 * i + 1] << (16 + 4 * i));
        *reinterpret_cast<uint32_t*>(region + chunk + (16 * (e % 32 / 8) + tc) * (W / 8) + 4 * (e / 32)) = word;
    } else {
        uint8_t* vr = region + int64_t(a.page) * D / 2 + chunk;
#pragma unroll
        for (int g = 0; g < 2; ++g) {  // two groups of 4 channels: groups h of one lane (W = 128) or two lanes
            const uint16_t half = uint16_t(u[4 * g] | (u[4 * g + 1] << 4) | (u[4 * g + 2] << 8) | (u[4 * g + 3] << 12));
            const int l = (e + 4 * g) / (W / 16), h = (e + 4 * g) % (W / 16) / 4;
            *reinterpret_cast<uint16_t*>(vr + (16 * (tc / 4) + l) * (W / 8) + 8 * h + 4 * (tc % 4 / 2) + 2 * (tc % 2)) = half;
        }
    }
    if (e == 0)
        reinterpret_cast<float*>(region + int64_t(a.page) * D)[(is_v ? NB + b : b) * int64_t(a.page) + tok] = s;
}

// A thread reads 8 channels of one head of one token of both sides.
template <int DT, int D>  // DT: 0 = f32, 1 = bf16, 2 = f16
__global__ __launch_bounds__(256) void kv4_read_kernel(Kv4ReadArgs a) {
    constexpr int W = kv4_width(D), NB = kv4_blocks(D);
    const int64_t t = blockIdx.x;
    const int part = blockIdx.y * 256 + threadIdx.x;
    const int head = part / (D / 8), d0 = part % (D / 8) * 8;
    if (head >= a.kv_heads) return;
    const int64_t slot = a.slots[t];
    const int64_t to = (t * a.kv_heads + head) * D + d0;
    float k[8], v[8];
    if (slot >= 0 && slot < a.pages * a.page) {
        const int64_t pg = slot / a.page;
        const int tok = int(slot - pg * a.page);
        const uint8_t* region = a.pool + (pg * a.kv_heads + head) * kv4_region(a.page, D);
        const int b = d0 / W, e = d0 % W, tc = tok % kKvChunkTokens;
        const int64_t chunk = (int64_t(tok / kKvChunkTokens) * NB + b) * (8 * W);
        const float* sc = reinterpret_cast<const float*>(region + int64_t(a.page) * D);
        const float ks = sc[int64_t(b) * a.page + tok], vs = sc[int64_t(NB + b) * a.page + tok];
        const uint32_t word =
            *reinterpret_cast<const uint32_t*>(region + chunk + (16 * (e % 32 / 8) + tc) * (W / 8) + 4 * (e / 32));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k[2 * i] = float(int((word >> (4 * i)) & 15u) - 8) * ks;
            k[2 * i + 1] = float(int((word >> (16 + 4 * i)) & 15u) - 8) * ks;
        }
        const uint8_t* vr = region + int64_t(a.page) * D / 2 + chunk;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int l = (e + 4 * g) / (W / 16), h = (e + 4 * g) % (W / 16) / 4;
            const uint32_t half =
                *reinterpret_cast<const uint16_t*>(vr + (16 * (tc / 4) + l) * (W / 8) + 8 * h + 4 * (tc % 4 / 2) + 2 * (tc % 2));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[4 * g + i] = float(int((half >> (4 * i)) & 15u) - 8) * vs;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = v[i] = 0.0f;
    }
    if constexpr (DT == 0) {
        float4* ko = reinterpret_cast<float4*>(static_cast<float*>(a.k) + to);
        float4* vo = reinterpret_cast<float4*>(static_cast<float*>(a.v) + to);
        ko[0] = make_float4(k[0], k[1], k[2], k[3]);
        ko[1] = make_float4(k[4], k[5], k[6], k[7]);
        vo[0] = make_float4(v[0], v[1], v[2], v[3]);
        vo[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        constexpr int ACT = DT == 1 ? int(kActBf16) : int(kActF16);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k) + to) = narrow8<ACT>(k);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v) + to) = narrow8<ACT>(v);
    }
}

template <int ACT>
hipError_t append_by_dim(const Kv4AppendArgs& a, hipStream_t stream) {
    const dim3 grid(unsigned(a.tokens), unsigned(ceil_div(int64_t(a.heads + 2 * a.kv_heads) * (a.dim / 8), 256)));
    switch (a.dim) {
        case 64: kv4_append_kernel<ACT, 64><<<grid, dim3(256), 0, stream>>>(a); break;
        case 128: kv4_append_kernel<ACT, 128><<<grid, dim3(256), 0, stream>>>(a); break;
        default: kv4_append_kernel<ACT, 256><<<grid, dim3(256), 0, stream>>>(a); break;
    }
    return hipGetLastError();
}

template <int DT>
hipError_t read_by_dim(const Kv4ReadArgs& a, hipStream_t stream) {
    const dim3 grid(unsigned(a.tokens), unsigned(ceil_div(int64_t(a.kv_heads) * (a.dim / 8), 256)));
    switch (a.dim) {
        case 64: kv4_read_kernel<DT, 64><<<grid, dim3(256), 0, stream>>>(a); break;
        case 128: kv4_read_kernel<DT, 128><<<grid, dim3(256), 0, stream>>>(a); break;
        default: kv4_read_kernel<DT, 256><<<grid, dim3(256), 0, stream>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_append(const Kv4AppendArgs& a, int act, hipStream_t stream) {
    return act == kActBf16 ? append_by_dim<kActBf16>(a, stream) : append_by_dim<kActF16>(a, stream);
}

hipError_t launch_kv4_read(const Kv4ReadArgs& a, int dtype, hipStream_t stream) {
    return dtype == 0 ? read_by_dim<0>(a, stream) : dtype == 1 ? read_by_dim<1>(a, stream) : read_by_dim<2>(a, stream);
}

}  // namespace w4a16
