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

// A thread owns 16 channels of one head of one token: two octets a, b that the
// rotation pairs (half layout: channels 8u.. and 8u + rot/2..; otherwise
// neighbours), so each is loaded once and one row of angles serves both.
//
// A workgroup takes 16 consecutive tokens and `passes` x (256 / D) heads: the
// tokens of a chunk are usually neighbours, and their words and half-words,
// which interleave in the same cache lines, then reach memory as whole lines
// from one L2.  The angles stay in registers over the heads.  HBM bounds it: 8192
// tokens of 48 heads of 128 channels, 181 MB, take 43 us, 4.2 TB/s, where a large
// copy reaches 4.8 (one workgroup a token, each thread one octet: 99 us, its
// lines written back in parts by several XCDs' L2s).
template <int ACT, int D>
__global__ __launch_bounds__(256) void kv4_append_kernel(Kv4AppendArgs a, int passes) {
    constexpr int W = kv4_width(D), NB = kv4_blocks(D), UNITS = D / 16, HEADS = 256 / (16 * UNITS);
    const int u = threadIdx.x % UNITS, row = threadIdx.x / UNITS;  // 16 tokens x HEADS heads
    const int64_t t = int64_t(blockIdx.x) * 16 + row % 16;
    if (t >= a.tokens) return;  // whole rows: a scale group's lanes leave together
    const int heads = a.heads + 2 * a.kv_heads;

    // octets, and whether they turn
    const int r8 = a.rot / 16;  // octets of half the rotated channels
    int oa = 2 * u, ob = 2 * u + 1;
    if (!a.interleaved) {
        oa = u < r8 ? u : 2 * u;
        ob = u < r8 ? u + r8 : 2 * u + 1;
    }
    const bool turns = u < r8;
    float c[8], s[8];
    bool known = true;
    if (a.rope) {
        const int64_t pos = a.positions[t];
        known = pos >= 0 && pos < a.rope_len;
        if (turns) {
            const float4* cs = reinterpret_cast<const float4*>(a.rope + (known ? pos : 0) * a.rot + 8 * u);
            const float4* sn = reinterpret_cast<const float4*>(a.rope + (known ? pos : 0) * a.rot + a.rot / 2 + 8 * u);
            const float4 x[4] = {cs[0], cs[1], sn[0], sn[1]};
            c[0] = x[0].x; c[1] = x[0].y; c[2] = x[0].z; c[3] = x[0].w;
            c[4] = x[1].x; c[5] = x[1].y; c[6] = x[1].z; c[7] = x[1].w;
            s[0] = x[2].x; s[1] = x[2].y; s[2] = x[2].z; s[3] = x[2].w;
            s[4] = x[3].x; s[5] = x[3].y; s[6] = x[3].z; s[7] = x[3].w;
        }
    }

    for (int p = 0; p < passes; ++p) {
        const int head = (int(blockIdx.y) * passes + p) * HEADS + row / 16;
        if (head >= heads) return;
        const uint16_t* src = a.qkv + t * a.ldqkv + int64_t(head) * D;
        float v[2][8];
        widen8<ACT>(*reinterpret_cast<const uint4*>(src + 8 * oa), v[0]);
        widen8<ACT>(*reinterpret_cast<const uint4*>(src + 8 * ob), v[1]);
        const bool is_v = head >= a.heads + a.kv_heads;
        if (turns && !is_v) {
            if (a.interleaved) {
#pragma unroll
                for (int o = 0; o < 2; ++o)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        rotate(v[o][2 * i], v[o][2 * i + 1], c[4 * o + i], s[4 * o + i], v[o][2 * i], v[o][2 * i + 1]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) rotate(v[0][i], v[1][i], c[i], s[i], v[0][i], v[1][i]);
            }
        }
        if (head < a.heads) {
            if (!known) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[0][i] = v[1][i] = __uint_as_float(0x7FC00000u);
            }
            uint16_t* dst = a.q_out + (t * a.heads + head) * D;
            *reinterpret_cast<uint4*>(dst + 8 * oa) = narrow8<ACT>(v[0]);
            *reinterpret_cast<uint4*>(dst + 8 * ob) = narrow8<ACT>(v[1]);
            continue;
        }
        const int64_t slot = a.slots[t];

        // largest magnitude of each block, over the head's lanes; one that is not finite leaves +inf (the
        // maximum of floats drops NaN, and its code would read back as an ordinary number)
        const int ba = 8 * oa / W, bb = 8 * ob / W;
        float amax[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) amax[b] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x = fabsf(v[0][i]), y = fabsf(v[1][i]);
            x = x < INFINITY ? x : INFINITY;
            y = y < INFINITY ? y : INFINITY;
            if constexpr (NB == 1) {
                amax[0] = fmaxf(amax[0], fmaxf(x, y));
            } else {
#pragma unroll
                for (int b = 0; b < NB; ++b) amax[b] = fmaxf(amax[b], fmaxf(ba == b ? x : 0.0f, bb == b ? y : 0.0f));
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            amax[b] = fmaxf(amax[b], lane_xor<1>(amax[b]));
            amax[b] = fmaxf(amax[b], lane_xor<2>(amax[b]));
            if constexpr (UNITS >= 8) amax[b] = fmaxf(amax[b], lane_xor<4>(amax[b]));
            if constexpr (UNITS >= 16) amax[b] = fmaxf(amax[b], lane_xor<8>(amax[b]));
        }
        if (!(known && slot >= 0 && slot < a.pages * a.page)) continue;
        float scale[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) scale[b] = amax[b] < INFINITY ? amax[b] / 7.0f : __uint_as_float(0x7FC00000u);

        const int64_t pg = slot / a.page;
        const int tok = int(slot - pg * a.page);
        const int kh = head - a.heads - (is_v ? a.kv_heads : 0);
        uint8_t* region = a.pool + (pg * a.kv_heads + kh) * kv4_region(a.page, D);
        const int tc = tok % kKvChunkTokens;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int octet = o ? ob : oa, b = o ? bb : ba, e = 8 * octet - W * b;
            const float f = NB == 1 || b == 0 ? scale[0] : scale[NB - 1];
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float r = f != 0.0f ? rintf(v[o][i] / f) : 0.0f;
                r = fminf(fmaxf(r, -8.0f), 7.0f);
                x[i] = uint32_t(int(r) + 8);
            }
            uint8_t* chunk = region + (int64_t(tok / kKvChunkTokens) * NB + b) * (8 * W);
            if (!is_v) {
                uint32_t word = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) word |= (x[2 * i] << (4 * i)) | (x[2 * i + 1] << (16 + 4 * i));
                *reinterpret_cast<uint32_t*>(chunk + (16 * (e % 32 / 8) + tc) * (W / 8) + 4 * (e / 32)) = word;
            } else {
                uint8_t* vr = chunk + int64_t(a.page) * D / 2;
#pragma unroll
                for (int g = 0; g < 2; ++g) {  // two groups of 4 channels: groups h of one lane (W = 128) or two lanes
                    const uint16_t half = uint16_t(x[4 * g] | (x[4 * g + 1] << 4) | (x[4 * g + 2] << 8) | (x[4 * g + 3] << 12));
                    const int l = (e + 4 * g) / (W / 16), h = (e + 4 * g) % (W / 16) / 4;
                    *reinterpret_cast<uint16_t*>(vr + (16 * (tc / 4) + l) * (W / 8) + 8 * h + 4 * (tc % 4 / 2) + 2 * (tc % 2)) = half;
                }
            }
        }
        if (u < NB)
            reinterpret_cast<float*>(region + int64_t(a.page) * D)[((is_v ? NB : 0) + u) * int64_t(a.page) + tok] =
                NB == 1 || u == 0 ? scale[0] : scale[NB - 1];
    }
}

// A thread reads 8 channels of one head of one token of both sides (8192 tokens
// of 8 heads of 128: 12 us for 43 MB, 3.5 TB/s; 14 us with one token a
// workgroup).  Its loads of 4 and 2 bytes, gathered from the chunks, hold it below
// a copy's rate.
template <int DT, int D>  // DT: 0 = f32, 1 = bf16, 2 = f16
__global__ __launch_bounds__(256) void kv4_read_kernel(Kv4ReadArgs a, int tokens) {
    constexpr int W = kv4_width(D), NB = kv4_blocks(D);
    // a workgroup takes `tokens` whole tokens, or 256 threads of one at a time (y)
    const int row = a.kv_heads * (D / 8);
    const int in = tokens > 1 ? int(threadIdx.x) / row : 0;
    const int64_t t = int64_t(blockIdx.x) * tokens + in;
    const int part = blockIdx.y * 256 + threadIdx.x - in * row;
    const int head = part / (D / 8), d0 = part % (D / 8) * 8;
    if (in >= tokens || t >= a.tokens || head >= a.kv_heads) return;
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
    // heads of a workgroup's pass, and as many passes (up to 4) as leave two workgroups a CU
    const int64_t per = 256 / a.dim, blocks = ceil_div(a.tokens, 16), rows = ceil_div(int64_t(a.heads + 2 * a.kv_heads), per);
    int passes = 4;
    while (passes > 1 && blocks * ceil_div(rows, passes) < 512) passes /= 2;
    const dim3 grid(unsigned(blocks), unsigned(ceil_div(rows, passes)));
    switch (a.dim) {
        case 64: kv4_append_kernel<ACT, 64><<<grid, dim3(256), 0, stream>>>(a, passes); break;
        case 128: kv4_append_kernel<ACT, 128><<<grid, dim3(256), 0, stream>>>(a, passes); break;
        default: kv4_append_kernel<ACT, 256><<<grid, dim3(256), 0, stream>>>(a, passes); break;
    }
    return hipGetLastError();
}

template <int DT>
hipError_t read_by_dim(const Kv4ReadArgs& a, hipStream_t stream) {
    const int row = a.kv_heads * (a.dim / 8), tokens = row < 256 ? 256 / row : 1;
    const dim3 grid(unsigned(ceil_div(a.tokens, tokens)), unsigned(ceil_div(row, 256)));
    switch (a.dim) {
        case 64: kv4_read_kernel<DT, 64><<<grid, dim3(256), 0, stream>>>(a, tokens); break;
        case 128: kv4_read_kernel<DT, 128><<<grid, dim3(256), 0, stream>>>(a, tokens); break;
        default: kv4_read_kernel<DT, 256><<<grid, dim3(256), 0, stream>>>(a, tokens); break;
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
