// Low-rank adapters of many requests beside a shared projection:
//
//   out[i] = y[i] + scale[l] (x[i] A_l^T) B_l^T,   l = index[i], none if l is
//                                                  not an adapter
//
// Two launches.  The first contracts K: t = x A^T in FP32, per part of K.
// The second adds the parts, contracts the rank and adds y.  Both take tiles
// of 16 rows in the order given: a tile's distinct adapters are found from
// its 16 indices, and each is one product in which the rows of other adapters
// are computed and dropped (matrix instructions are idle here; the weights'
// bytes are what counts, and each adapter's are read once a tile).
#include "common.h"
#include "kernels.h"
#include "lora.h"

namespace w4a16 {

namespace {

template <int ACT>
__device__ inline f32x4_t mfma16(uint4 a, uint4 b, f32x4_t c) {
    if constexpr (ACT == kActBf16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

// The distinct adapters among a tile's rows, taken one by one; lanes 0..15
// of `mine` (and their copies) hold the rows' indices.
struct Distinct {
    int mine;
    uint64_t left;
    __device__ Distinct(const int32_t* index, int64_t row0, int64_t m, int adapters, int lane) {
        const int64_t row = row0 + lane % 16;
        mine = row < m ? index[row] : -1;
        if (mine >= adapters) mine = -1;
        left = __ballot(mine >= 0) & 0xFFFFull;
    }
    __device__ int next() {
        const int l = __builtin_amdgcn_readlane(mine, __ffsll((unsigned long long)left) - 1);
        left &= ~__ballot(mine == l);
        return l;
    }
};

constexpr int kWaves = 4;

// t[split][row][r] = sum over the split's columns of x[row] A_l[r].
// Grid: x = row tile, y = slot, z = split.  The waves take 32-column steps in
// turn and add up in LDS.
template <int ACT, int RT>  // RT: 16-row tiles of the rank
__global__ __launch_bounds__(256) void lora_shrink_kernel(LoraArgs a, int slots, int kspan, float* t) {
    __shared__ float lds[kWaves][RT * 4][64];
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int col = lane % 16, kq = lane / 16;
    const int64_t row0 = int64_t(blockIdx.x) * 16;
    Distinct d(a.index, row0, a.m, a.adapters, lane);
    const int64_t k0 = int64_t(blockIdx.z) * kspan, k1 = k0 + kspan < a.k ? k0 + kspan : a.k;
    const int64_t row = row0 + col < a.m ? row0 + col : a.m - 1;
    const uint16_t* xr = a.x + row * a.ldx + 8 * kq;
    for (int seen = 0; d.left; ++seen) {
        const int l = d.next();
        if (seen % slots != int(blockIdx.y)) continue;
        const uint16_t* ar[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int r = min(16 * i + col, a.rank - 1);
            ar[i] = a.a + (int64_t(l) * a.rank + r) * a.k + 8 * kq;
        }
        f32x4_t acc[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i] = f32x4_t{0, 0, 0, 0};
        for (int64_t k = k0 + 32 * wave; k < k1; k += 32 * kWaves) {
            // K is a multiple of 8: a lane's 8 columns are inside or outside together
            const bool in = k + 8 * kq < k1;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const uint4 xv = in ? *reinterpret_cast<const uint4*>(xr + k) : zero;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const uint4 av = in ? *reinterpret_cast<const uint4*>(ar[i] + k) : zero;
                acc[i] = mfma16<ACT>(av, xv, acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) lds[wave][4 * i + j][lane] = acc[i][j];
        __syncthreads();
        // wave w adds and stores the rank tiles w, w + 4, ..
        for (int i = wave; i < RT; i += kWaves) {
            float s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[j] = lds[0][4 * i + j][lane] + lds[1][4 * i + j][lane] + lds[2][4 * i + j][lane] + lds[3][4 * i + j][lane];
            const int r = 16 * i + 4 * kq;
            if (d.mine == l && row0 + col < a.m && r < a.rank)
                *reinterpret_cast<float4*>(t + (int64_t(blockIdx.z) * a.m + row0 + col) * a.rank + r) = make_float4(s[0], s[1], s[2], s[3]);
        }
        __syncthreads();
    }
}

// out[row] = y[row] + scale t[row] B_l^T.  Grid: x = 256 columns, y = row
// tile, z = slot.  A wave computes 64 columns as two pairs of MFMA tiles whose
// output rows interleave, so a lane holds 8 consecutive columns of its row.
// t enters as a high and a low 16-bit part (16 or more significant bits in
// all), scaled by a power of two per row so that f16 neither overflows nor
// loses bits.
template <int ACT, int RS>  // RS: 32-wide steps of the rank
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs a, int slots, int splits, const float* t) {
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int col = lane % 16, kq = lane / 16;
    const int64_t row0 = int64_t(blockIdx.y) * 16;
    const int64_t n0 = int64_t(blockIdx.x) * 256 + 64 * wave;
    if (n0 >= a.n) return;
    Distinct d(a.index, row0, a.m, a.adapters, lane);
    const int64_t row = row0 + col;
    const bool real = row < a.m;
    float add[2][8];
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) add[g][i] = 0.0f;
    // rows without an adapter are copied by the first slot
    bool write = real && d.mine < 0 && blockIdx.z == 0;
    for (int seen = 0; d.left; ++seen) {
        const int l = d.next();
        if (seen % slots != int(blockIdx.z)) continue;
        const bool mine = real && d.mine == l;
        write |= mine;
        const float scale = a.scales ? a.scales[l] : 1.0f;
        float v[RS][8];
        float big = 0.0f;
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            const int r = 32 * s + 8 * kq;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[s][i] = 0.0f;
            if (mine && r < a.rank) {
                for (int p = 0; p < splits; ++p) {
                    const float4* src = reinterpret_cast<const float4*>(t + (int64_t(p) * a.m + row) * a.rank + r);
                    const float4 lo = src[0], hi = src[1];
                    v[s][0] += lo.x; v[s][1] += lo.y; v[s][2] += lo.z; v[s][3] += lo.w;
                    v[s][4] += hi.x; v[s][5] += hi.y; v[s][6] += hi.z; v[s][7] += hi.w;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[s][i] *= scale;
                big = fmaxf(big, fabsf(v[s][i]));
            }
        }
        big = max_xor32(fmaxf(big, lane_xor<16>(big)));
        const int e = big > 0.0f && big < 3e38f ? int(__float_as_uint(big) >> 23) - 127 : 0;
        uint4 hi[RS], lo[RS];
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            uint32_t h[4], w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = ldexpf(v[s][2 * i], -e), q = ldexpf(v[s][2 * i + 1], -e);
                const uint16_t ph = from_f32<ACT>(p), qh = from_f32<ACT>(q);
                h[i] = uint32_t(ph) | (uint32_t(qh) << 16);
                w[i] = uint32_t(from_f32<ACT>(p - to_f32<ACT>(ph))) | (uint32_t(from_f32<ACT>(q - to_f32<ACT>(qh))) << 16);
            }
            hi[s] = make_uint4(h[0], h[1], h[2], h[3]);
            lo[s] = make_uint4(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            f32x4_t acc[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // MFMA row `col` of half h is column 8 (col / 4) + 4 h + col % 4
                const int64_t n = n0 + 32 * g + 8 * (col / 4) + 4 * h + col % 4;
                const uint16_t* br = a.b + (int64_t(l) * a.n + (n < a.n ? n : a.n - 1)) * a.rank + 8 * kq;
                acc[h] = f32x4_t{0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < RS; ++s) {
                    const uint4 bv = 32 * s + 8 * kq < a.rank ? *reinterpret_cast<const uint4*>(br + 32 * s) : make_uint4(0, 0, 0, 0);
                    acc[h] = mfma16<ACT>(bv, hi[s], acc[h]);
                    acc[h] = mfma16<ACT>(bv, lo[s], acc[h]);
                }
            }
            if (mine) {
#pragma unroll
                for (int i = 0; i < 8; ++i) add[g][i] = ldexpf(acc[i / 4][i % 4], e);
            }
        }
    }
    if (!write) return;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int64_t n = n0 + 32 * g + 8 * kq;
        const uint16_t* src = a.y + row * a.ldy + n;
        uint16_t* dst = a.out + row * a.ldo + n;
        const bool wide = n + 8 <= a.n && a.ldy % 8 == 0 && a.ldo % 8 == 0 &&
                          ((reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
        if (wide) {
            const uint4 raw = *reinterpret_cast<const uint4*>(src);
            const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = uint32_t(from_f32<ACT>(to_f32<ACT>(uint16_t(in[i])) + add[g][2 * i])) |
                       (uint32_t(from_f32<ACT>(to_f32<ACT>(uint16_t(in[i] >> 16)) + add[g][2 * i + 1])) << 16);
            *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (n + i < a.n) dst[i] = from_f32<ACT>(to_f32<ACT>(src[i]) + add[g][i]);
        }
    }
}

template <int ACT, int RT>
hipError_t run(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
    float* t = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kSyncBytes);
    const unsigned tiles = unsigned(ceil_div(a.m, 16));
    lora_shrink_kernel<ACT, RT><<<dim3(tiles, unsigned(p.slots), unsigned(p.splits)), dim3(256), 0, stream>>>(a, p.slots, int(p.kspan), t);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    lora_expand_kernel<ACT, (RT + 1) / 2><<<dim3(unsigned(ceil_div(a.n, 256)), tiles, unsigned(p.slots)), dim3(256), 0, stream>>>(a, p.slots, p.splits, t);
    return hipGetLastError();
}

template <int ACT>
hipError_t run_by_rank(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
    if (a.rank <= 16) return run<ACT, 1>(a, p, stream);
    if (a.rank <= 32) return run<ACT, 2>(a, p, stream);
    if (a.rank <= 64) return run<ACT, 4>(a, p, stream);
    return run<ACT, 8>(a, p, stream);
}

}  // namespace

// Rows of one launch: its row tiles are the grid's second dimension, at most 65535.
constexpr int64_t kMaxRows = int64_t(1) << 19;

LoraPlan plan_lora(int64_t m, int64_t n, int64_t k, int adapters, int rank) {
    LoraPlan p{};
    if (m > kMaxRows) m = kMaxRows;
    const int64_t tiles = ceil_div(m, 16);
    const int64_t most = m < 16 ? m : 16;
    p.slots = int(tiles >= 64 ? 1 : most < adapters ? most : adapters);
    if (p.slots < 1) p.slots = 1;
    int64_t splits = ceil_div(512, tiles * p.slots);
    if (splits > ceil_div(k, 512)) splits = ceil_div(k, 512);
    if (splits > 16) splits = 16;
    p.kspan = ceil_div(ceil_div(k, splits), 32) * 32;
    p.splits = int(ceil_div(k, p.kspan));
    p.workspace = size_t(p.splits) * size_t(m) * size_t(rank) * 4;
    return p;
}

hipError_t launch_lora(const LoraArgs& a, int act, hipStream_t stream) {
    for (int64_t r0 = 0; r0 < a.m; r0 += kMaxRows) {
        LoraArgs c = a;
        c.m = a.m - r0 < kMaxRows ? a.m - r0 : kMaxRows;
        c.x += r0 * a.ldx;
        c.y += r0 * a.ldy;
        c.out += r0 * a.ldo;
        c.index += r0;
        const LoraPlan p = plan_lora(c.m, a.n, a.k, a.adapters, a.rank);
        const hipError_t e = act == kActBf16 ? run_by_rank<kActBf16>(c, p, stream) : run_by_rank<kActF16>(c, p, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace w4a16
