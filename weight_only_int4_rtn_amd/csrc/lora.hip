// Low-rank adapters of many requests beside a shared projection:
//
//   out[i] = y[i] + scale[l] (x[i] A_l^T) B_l^T,   l = index[i], none if l is
//                                                  not an adapter
//
// Two launches.  The first contracts K: t = x A^T in FP32, per part of K.
// The second adds the parts, contracts the rank and adds y.  Both take tiles of
// rows in the order given: a tile's distinct adapters are found from its
// indices, and each is one product in which the rows of other adapters are
// computed and dropped (matrix instructions are idle here; the weights' bytes
// are what counts, and each adapter's are read once a tile).  With few rows a
// tile's adapters go to workgroups of their own (slots).
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

// The distinct adapters among a tile's ROWS rows (at most 64), taken one by one;
// lane L holds row L % ROWS's index in `mine`.
template <int ROWS>
struct Distinct {
    int mine;
    uint64_t left;
    __device__ Distinct(const int32_t* index, int64_t row0, int64_t m, int adapters, int lane) {
        const int64_t row = row0 + lane % ROWS;
        mine = row < m ? index[row] : -1;
        if (mine >= adapters) mine = -1;
        left = __ballot(mine >= 0) & (~0ull >> (64 - ROWS));
    }
    // the next adapter, and its rows (a bit each)
    __device__ int next(uint64_t& rows) {
        const int l = __builtin_amdgcn_readlane(mine, __ffsll((unsigned long long)left) - 1);
        rows = __ballot(mine == l) & left;
        left &= ~rows;
        return l;
    }
};

// Position of the n-th set bit (n from 0; any position if there are not so many).
__device__ inline int nth_bit(uint64_t mask, int n) {
    int at = 0;
#pragma unroll
    for (int w = 32; w > 0; w /= 2) {
        const uint64_t low = mask & ((uint64_t(1) << w) - 1);
        const int have = __popcll(low);
        const bool up = n >= have;
        at += up ? w : 0;
        n -= up ? have : 0;
        mask = up ? mask >> w : low;
    }
    return at;
}

// One row's t (this lane's channels of it) as MFMA operands: a high and a low
// 16-bit part, scaled by 2^-e so that the row's largest lies in [1, 2) for bf16
// and in [2^14, 2^15) for f16, near the top of its range: the low parts of small
// channels then keep 16 or more significant bits together with the high ones, in
// bf16 at any size, in f16 down to 2^-22 of the row's largest, whose 2^-38 is
// f16's smallest step (with the largest at 1, 12.6 bits at 2^-14).  Returns e.
template <int ACT, int RS>  // RS: 32-wide steps of the rank
__device__ inline int operands_of(const float (&v)[RS][8], uint4 (&hi)[RS], uint4 (&lo)[RS]) {
    float big = 0.0f;
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(v[s][i]));
    big = max_xor32(fmaxf(big, lane_xor<16>(big)));
    const int e = big > 0.0f && big < INFINITY ? int(__float_as_uint(big) >> 23) - 127 - (ACT == kActF16 ? 14 : 0) : 0;
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
    return e;
}

// The same of a row's sums in the workspace (their parts added, times the adapter's scale).
template <int ACT, int RS>
__device__ inline int row_operand(const LoraArgs& a, const float* t, int splits, int64_t row, bool mine, float scale, int kq,
                                  uint4 (&hi)[RS], uint4 (&lo)[RS]) {
    float v[RS][8];
#pragma unroll
    for (int s = 0; s < RS; ++s) {
        const int r = 32 * s + 8 * kq;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[s][i] = 0.0f;
        if (mine && r < a.rank) {
#pragma unroll 4
            for (int p = 0; p < splits; ++p) {
                const float4* src = reinterpret_cast<const float4*>(t + (int64_t(p) * a.m + row) * a.rank + r);
                const float4 x = src[0], y = src[1];
                v[s][0] += x.x; v[s][1] += x.y; v[s][2] += x.z; v[s][3] += x.w;
                v[s][4] += y.x; v[s][5] += y.y; v[s][6] += y.z; v[s][7] += y.w;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[s][i] *= scale;
    }
    return operands_of<ACT, RS>(v, hi, lo);
}


// x A_l^T of 16 rows (lane L: row at xr, quarter L / 16 of each 32 columns) over
// columns [k0, k1), by a whole workgroup: the waves take runs of columns in turn
// and add up in LDS.  Left in sum: place p = component p / 64 of lane p % 64 (rank
// index 16 (p / 256) + 4 (lane / 16) + p / 64 % 4 of row lane % 16).
template <int ACT, int RT, int WAVES>  // RT: 16-row tiles of the rank
__device__ inline void contract(const LoraArgs& a, int l, const uint16_t* xr, int64_t k0, int64_t k1, int wave, int lane,
                                float (*lds)[RT * 4 * 64]) {
    constexpr int UN = RT >= 8 ? 2 : 4;
    const int col = lane % 16, kq = lane / 16;
    const uint16_t* ar[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int r = min(16 * i + col, a.rank - 1);
        ar[i] = a.a + (int64_t(l) * a.rank + r) * a.k + 8 * kq;
    }
    f32x4_t acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = f32x4_t{0, 0, 0, 0};
    // A wave takes runs of 32 UN columns in turn, all of a run's loads in flight
    // together; of the last run the columns that exist (K is a multiple of 8: a
    // lane's 8 columns are inside or outside together).
    for (int64_t k = k0 + 32 * UN * wave; k < k1; k += 32 * UN * WAVES) {
        if (k + 32 * UN <= k1) {
            uint4 xv[UN], av[UN][RT];
#pragma unroll
            for (int n = 0; n < UN; ++n) {
                xv[n] = *reinterpret_cast<const uint4*>(xr + k + 32 * n);
#pragma unroll
                for (int i = 0; i < RT; ++i) av[n][i] = *reinterpret_cast<const uint4*>(ar[i] + k + 32 * n);
            }
#pragma unroll
            for (int n = 0; n < UN; ++n)
#pragma unroll
                for (int i = 0; i < RT; ++i) acc[i] = mfma16<ACT>(av[n][i], xv[n], acc[i]);
            continue;
        }
        for (int64_t kk = k; kk < k1; kk += 32) {
            uint4 xv = make_uint4(0, 0, 0, 0), av[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) av[i] = xv;
            if (kk + 8 * kq < k1) {
                xv = *reinterpret_cast<const uint4*>(xr + kk);
#pragma unroll
                for (int i = 0; i < RT; ++i) av[i] = *reinterpret_cast<const uint4*>(ar[i] + kk);
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) acc[i] = mfma16<ACT>(av[i], xv, acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) lds[wave][(4 * i + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int p = threadIdx.x; p < RT * 4 * 64; p += 64 * WAVES) {
        float x = lds[0][p];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) x += lds[w][p];
        lds[0][p] = x;
    }
    __syncthreads();
}

// The operands of the sums that contract() left, times the adapter's scale.  Returns e.
template <int ACT, int RT>
__device__ inline int contracted_operand(const LoraArgs& a, const float* sum, float scale, int lane, uint4 (&hi)[(RT + 1) / 2],
                                         uint4 (&lo)[(RT + 1) / 2]) {
    constexpr int RS = (RT + 1) / 2;
    const int col = lane % 16, kq = lane / 16;
    float v[RS][8];
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // rank index 32 s + 8 kq + i: rank tile 2 s + kq / 2, quarter 2 (kq % 2) + i / 4 of its rows
            const int tile = min(2 * s + kq / 2, RT - 1), from = (2 * (kq % 2) + i / 4) * 16 + col;
            const float x = sum[(4 * tile + i % 4) * 64 + from] * scale;
            v[s][i] = 32 * s + 8 * kq < a.rank ? x : 0.0f;
        }
    return operands_of<ACT, RS>(v, hi, lo);
}

// t[split][row][r] = sum over the split's columns of x[row] A_l[r].
// Grid: x = tile of TILE rows, y = slot, z = split.  An adapter's rows are
// gathered, 16 to a product, so its weights are read once a tile wherever its
// rows stand.
//
// OPERANDS (one split, tiles of 16 rows in place): instead of sums, the rows'
// operands for the second launch (operands_of): [row tile][32-wide step of the
// rank][high, low][lane].
template <int ACT, int RT, int TILE, bool OPERANDS>  // RT: 16-row tiles of the rank
__global__ __launch_bounds__(OPERANDS ? 512 : 256) void lora_shrink_kernel(LoraArgs a, int slots, int kspan, float* t, uint4* operands, float* factors) {
    constexpr int WAVES = OPERANDS ? 8 : 4;
    __shared__ float lds[WAVES][RT * 4 * 64];
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int col = lane % 16, kq = lane / 16;
    const int64_t row0 = int64_t(blockIdx.x) * TILE;
    Distinct<TILE> d(a.index, row0, a.m, a.adapters, lane);
    const int64_t k0 = int64_t(blockIdx.z) * kspan, k1 = k0 + kspan < a.k ? k0 + kspan : a.k;
    for (int seen = 0; d.left; ++seen) {
        uint64_t rows;
        const int l = d.next(rows);
        if (seen % slots != int(blockIdx.y)) continue;
        const float scale = OPERANDS && a.scales ? a.scales[l] : 1.0f;
        const int count = __popcll(rows);
        for (int first = 0; first < (OPERANDS ? 1 : count); first += 16) {
            const bool mine = OPERANDS ? (rows >> col & 1) : first + col < count;
            const int at = OPERANDS ? col : nth_bit(rows, mine ? first + col : first);
            const int64_t row = row0 + at < a.m ? row0 + at : a.m - 1;
            const uint16_t* xr = a.x + row * a.ldx + 8 * kq;
            contract<ACT, RT, WAVES>(a, l, xr, k0, k1, wave, lane, lds);
            if constexpr (OPERANDS) {
                if (wave == 0) {
                    constexpr int RS = (RT + 1) / 2;
                    uint4 hi[RS], lo[RS];
                    const int e = contracted_operand<ACT, RT>(a, lds[0], scale, lane, hi, lo);
                    if (mine) {
                        uint4* to = operands + int64_t(blockIdx.x) * RS * 128 + lane;
#pragma unroll
                        for (int s = 0; s < RS; ++s) {
                            to[(2 * s) * 64] = hi[s];
                            to[(2 * s + 1) * 64] = lo[s];
                        }
                        if (kq == 0) factors[row] = ldexpf(1.0f, e);
                    }
                }
            } else {
                for (int i = wave; i < RT; i += WAVES) {
                    const int r = 16 * i + 4 * kq;
                    if (mine && r < a.rank)
                        *reinterpret_cast<float4*>(t + (int64_t(blockIdx.z) * a.m + row) * a.rank + r) =
                            make_float4(lds[0][(4 * i) * 64 + lane], lds[0][(4 * i + 1) * 64 + lane], lds[0][(4 * i + 2) * 64 + lane],
                                        lds[0][(4 * i + 3) * 64 + lane]);
                }
            }
            __syncthreads();
        }
    }
}

// MFMA row `col` of half h of a 32-column group: columns interleave so that a
// lane's two times four results are 8 consecutive columns.
__device__ inline int column_of(int col, int h) { return 8 * (col / 4) + 4 * h + col % 4; }

// 8 columns of a row, of which `left` (any number) exist.
__device__ inline uint4 load_columns(const uint16_t* src, int64_t left) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) w[i / 2] |= uint32_t(src[i]) << (16 * (i % 2));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ inline void store_columns(uint16_t* dst, int64_t left, uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) dst[i] = uint16_t(w[i / 2] >> (16 * (i % 2)));
}

// y + f acc on 8 columns, rounded once
template <int ACT>
__device__ inline uint4 add_columns(uint4 y, f32x4_t lo, f32x4_t hi, float f) {
    const uint32_t in[4] = {y.x, y.y, y.z, y.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float p = i < 2 ? lo[2 * i] : hi[2 * i - 4], q = i < 2 ? lo[2 * i + 1] : hi[2 * i - 3];
        o[i] = uint32_t(from_f32<ACT>(fmaf(p, f, to_f32<ACT>(uint16_t(in[i]))))) |
               (uint32_t(from_f32<ACT>(fmaf(q, f, to_f32<ACT>(uint16_t(in[i] >> 16))))) << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Few rows: out[row] = y[row] + scale t[row] B_l^T.  Grid: x = 256 columns, y =
// tile of TILE rows, z = slot.  A wave computes 64 columns of an adapter's rows,
// gathered 16 to a product; the operands of B are read once a tile.  Latency
// bounds the pair of launches: 64 rows, 48 adapters of rank 16, 4096 x 4096: 7 and
// 8 us for 14 MB.  Part of it is each slot's way to its adapter, a ballot and a
// lane read for every adapter of the tile before it, before its first load.
template <int ACT, int RS, int TILE>
__global__ __launch_bounds__(256) void lora_expand_kernel(LoraArgs a, int slots, int splits, const float* t) {
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int col = lane % 16, kq = lane / 16;
    const int64_t row0 = int64_t(blockIdx.y) * TILE;
    const int64_t n0 = int64_t(blockIdx.x) * 256 + 64 * wave;
    if (n0 >= a.n) return;
    Distinct<TILE> d(a.index, row0, a.m, a.adapters, lane);
    const bool aligned = a.ldy % 8 == 0 && a.ldo % 8 == 0 && ((reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
    auto add = [&](int64_t row, const f32x4_t (&acc)[2][2], float f) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int64_t n = n0 + 32 * g + 8 * kq;
            const uint16_t* src = a.y + row * a.ldy + n;
            uint16_t* dst = a.out + row * a.ldo + n;
            if (aligned && n + 8 <= a.n) *reinterpret_cast<uint4*>(dst) = add_columns<ACT>(*reinterpret_cast<const uint4*>(src), acc[g][0], acc[g][1], f);
            else store_columns(dst, a.n - n, add_columns<ACT>(load_columns(src, a.n - n), acc[g][0], acc[g][1], f));
        }
    };
    if (blockIdx.z == 0 && a.out != a.y) {
        // rows without an adapter are copied by the first slot
        const uint64_t none = __ballot(d.mine < 0 && lane < TILE && row0 + lane < a.m);
        const f32x4_t zero[2][2] = {};
        for (int first = 0; first < __popcll(none); first += 16)
            if (first + col < __popcll(none)) add(row0 + nth_bit(none, first + col), zero, 0.0f);
    }
    for (int seen = 0; d.left; ++seen) {
        uint64_t rows;
        const int l = d.next(rows);
        if (seen % slots != int(blockIdx.z)) continue;
        const float scale = a.scales ? a.scales[l] : 1.0f;
        uint4 bv[2][2][RS];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t n = n0 + 32 * g + column_of(col, h);
                const uint16_t* br = a.b + (int64_t(l) * a.n + (n < a.n ? n : a.n - 1)) * a.rank + 8 * kq;
#pragma unroll
                for (int s = 0; s < RS; ++s) {
                    bv[g][h][s] = make_uint4(0, 0, 0, 0);
                    if (32 * s + 8 * kq < a.rank) bv[g][h][s] = *reinterpret_cast<const uint4*>(br + 32 * s);
                }
            }
        const int count = __popcll(rows);
        for (int first = 0; first < count; first += 16) {
            const bool mine = first + col < count;
            const int64_t row = row0 + nth_bit(rows, mine ? first + col : first);
            uint4 hi[RS], lo[RS];
            const int e = row_operand<ACT, RS>(a, t, splits, row, mine, scale, kq, hi, lo);
            f32x4_t acc[2][2];
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    acc[g][h] = f32x4_t{0, 0, 0, 0};
#pragma unroll
                    for (int s = 0; s < RS; ++s) {
                        acc[g][h] = mfma16<ACT>(bv[g][h][s], hi[s], acc[g][h]);
                        acc[g][h] = mfma16<ACT>(bv[g][h][s], lo[s], acc[g][h]);
                    }
                }
            if (mine) add(row, acc, ldexpf(1.0f, e));
        }
    }
}

// A row or two: both steps in one launch.  Grid: x = 256 columns; every
// workgroup contracts K for itself, which the L2 serves, and saves the second
// launch and the way through memory between the two.
template <int ACT, int RT>
__global__ __launch_bounds__(512) void lora_one_kernel(LoraArgs a) {
    constexpr int WAVES = 8, RS = (RT + 1) / 2;
    __shared__ float lds[WAVES][RT * 4 * 64];
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int col = lane % 16, kq = lane / 16;
    const int64_t n0 = int64_t(blockIdx.x) * 256 + 32 * wave;
    Distinct<16> d(a.index, 0, a.m, a.adapters, lane);
    const int64_t row = col < a.m ? col : a.m - 1;
    const int64_t n = n0 + 8 * kq;
    const uint16_t* src = a.y + row * a.ldy + n;
    uint16_t* dst = a.out + row * a.ldo + n;
    const bool whole = n + 8 <= a.n && a.ldy % 8 == 0 && a.ldo % 8 == 0 &&
                       ((reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
    uint4 y = make_uint4(0, 0, 0, 0);
    if (whole) y = *reinterpret_cast<const uint4*>(src);
    else y = load_columns(src, a.n - n);
    f32x4_t add[2] = {f32x4_t{0, 0, 0, 0}, f32x4_t{0, 0, 0, 0}};
    float f = 0.0f;
    while (d.left) {
        uint64_t rows;
        const int l = d.next(rows);
        const float scale = a.scales ? a.scales[l] : 1.0f;
        uint4 bv[2][RS];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t c = n0 + column_of(col, h);
            const uint16_t* br = a.b + (int64_t(l) * a.n + (c < a.n ? c : a.n - 1)) * a.rank + 8 * kq;
#pragma unroll
            for (int s = 0; s < RS; ++s) {
                bv[h][s] = make_uint4(0, 0, 0, 0);
                if (32 * s + 8 * kq < a.rank) bv[h][s] = *reinterpret_cast<const uint4*>(br + 32 * s);
            }
        }
        contract<ACT, RT, WAVES>(a, l, a.x + row * a.ldx + 8 * kq, 0, a.k, wave, lane, lds);
        uint4 hi[RS], lo[RS];
        const int e = contracted_operand<ACT, RT>(a, lds[0], scale, lane, hi, lo);
        f32x4_t acc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            acc[h] = f32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < RS; ++s) {
                acc[h] = mfma16<ACT>(bv[h][s], hi[s], acc[h]);
                acc[h] = mfma16<ACT>(bv[h][s], lo[s], acc[h]);
            }
        }
        if (rows >> col & 1) {
            add[0] = acc[0];
            add[1] = acc[1];
            f = ldexpf(1.0f, e);
        }
        __syncthreads();
    }
    if (col >= a.m) return;
    const uint4 o = add_columns<ACT>(y, add[0], add[1], f);
    if (whole) *reinterpret_cast<uint4*>(dst) = o;
    else store_columns(dst, a.n - n, o);
}

// Many rows.  Grid: x = kTallCols columns, y = tile of 64 rows.  A wave takes a
// quarter of the columns of all 64 rows, 64 at a time (a row's line of 128
// bytes is read and written in one go), so each operand of B serves four
// products; t comes as operands.  A tile's adapters are taken one after another,
// each reading and writing the rows that are its own.  4099 rows by 32768
// columns at rank 64, 537 MB of y and out, take 147 us, 3.7 TB/s, and the first
// launch 23 (t turned into operands by every workgroup here: 200 and 19; 32 or 16
// rows a wave 160 and 210, as B comes from the L2 once for each).  A wave
// loads y and B of the next columns only after these are stored: nothing is in
// flight meanwhile.
constexpr int kTallCols = 512, kTallGroups = 4, kTallRows = 16 * kTallGroups;

template <int ACT, int RS>
__global__ __launch_bounds__(256) void lora_expand_rows_kernel(LoraArgs a, const uint4* operands, const float* factors) {
    constexpr int PAIR = RS > 2 ? 1 : 2;  // groups of 32 columns at a time, as registers go
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int col = lane % 16, kq = lane / 16;
    const int64_t row0 = int64_t(blockIdx.y) * kTallRows;
    const int64_t n0 = int64_t(blockIdx.x) * kTallCols + kTallCols / 4 * wave;
    if (n0 >= a.n) return;
    const int64_t n1 = n0 + kTallCols / 4 < a.n ? n0 + kTallCols / 4 : a.n;
    Distinct<kTallRows> d(a.index, row0, a.m, a.adapters, lane);
    int index[kTallGroups];  // of this lane's row in each group of 16
    const uint16_t* src[kTallGroups];
    uint16_t* dst[kTallGroups];
#pragma unroll
    for (int g = 0; g < kTallGroups; ++g) {
        index[g] = __shfl(d.mine, 16 * g + col);
        const int64_t row = row0 + 16 * g + col < a.m ? row0 + 16 * g + col : a.m - 1;
        src[g] = a.y + row * a.ldy + 8 * kq;
        dst[g] = a.out + row * a.ldo + 8 * kq;
    }
    const bool aligned = a.ldy % 8 == 0 && a.ldo % 8 == 0 && ((reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
    while (d.left) {
        uint64_t rows;
        const int l = d.next(rows);
        uint4 hi[kTallGroups][RS], lo[kTallGroups][RS];
        float f[kTallGroups];
#pragma unroll
        for (int g = 0; g < kTallGroups; ++g) {
            f[g] = 0.0f;
#pragma unroll
            for (int s = 0; s < RS; ++s) hi[g][s] = lo[g][s] = make_uint4(0, 0, 0, 0);
            if (index[g] == l) {
                const uint4* from = operands + (int64_t(blockIdx.y) * kTallGroups + g) * RS * 128 + lane;
                f[g] = factors[row0 + 16 * g + col];
#pragma unroll
                for (int s = 0; s < RS; ++s) {
                    hi[g][s] = from[(2 * s) * 64];
                    lo[g][s] = from[(2 * s + 1) * 64];
                }
            }
        }
        const uint16_t* b = a.b + int64_t(l) * a.n * a.rank + 8 * kq;
#pragma unroll 1
        for (int64_t c0 = n0; c0 < n1; c0 += 32 * PAIR) {
            const bool whole = aligned && c0 + 32 * PAIR <= a.n;
            uint4 bv[PAIR][2][RS], yv[PAIR][kTallGroups];
#pragma unroll
            for (int p = 0; p < PAIR; ++p) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int64_t n = c0 + 32 * p + column_of(col, h);
                    const uint16_t* br = b + (n < a.n ? n : a.n - 1) * a.rank;
#pragma unroll
                    for (int s = 0; s < RS; ++s) {
                        bv[p][h][s] = make_uint4(0, 0, 0, 0);
                        if (32 * s + 8 * kq < a.rank) bv[p][h][s] = *reinterpret_cast<const uint4*>(br + 32 * s);
                    }
                }
#pragma unroll
                for (int g = 0; g < kTallGroups; ++g)
                    if (index[g] == l)
                        yv[p][g] = whole ? *reinterpret_cast<const uint4*>(src[g] + c0 + 32 * p)
                                         : load_columns(src[g] + c0 + 32 * p, a.n - (c0 + 32 * p + 8 * kq));
            }
#pragma unroll
            for (int g = 0; g < kTallGroups; ++g) {
                if (!__any(index[g] == l)) continue;
#pragma unroll
                for (int p = 0; p < PAIR; ++p) {
                    f32x4_t acc[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        acc[h] = f32x4_t{0, 0, 0, 0};
#pragma unroll
                        for (int s = 0; s < RS; ++s) {
                            acc[h] = mfma16<ACT>(bv[p][h][s], hi[g][s], acc[h]);
                            acc[h] = mfma16<ACT>(bv[p][h][s], lo[g][s], acc[h]);
                        }
                    }
                    if (index[g] == l) {
                        const uint4 o = add_columns<ACT>(yv[p][g], acc[0], acc[1], f[g]);
                        if (whole) *reinterpret_cast<uint4*>(dst[g] + c0 + 32 * p) = o;
                        else store_columns(dst[g] + c0 + 32 * p, a.n - (c0 + 32 * p + 8 * kq), o);
                    }
                }
            }
        }
    }
    // rows without an adapter
#pragma unroll
    for (int g = 0; g < kTallGroups; ++g) {
        if (index[g] >= 0 || row0 + 16 * g + col >= a.m || a.out == a.y) continue;
        for (int64_t c0 = n0; c0 < n1; c0 += 32) {
            if (aligned && c0 + 32 <= a.n) *reinterpret_cast<uint4*>(dst[g] + c0) = *reinterpret_cast<const uint4*>(src[g] + c0);
            else store_columns(dst[g] + c0, a.n - (c0 + 8 * kq), load_columns(src[g] + c0, a.n - (c0 + 8 * kq)));
        }
    }
}

template <int ACT, int RT>
hipError_t run(const LoraArgs& a, const LoraPlan& p, hipStream_t stream) {
    float* t = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kSyncBytes);
    const unsigned tiles = unsigned(ceil_div(a.m, p.tile));
    constexpr int RS = (RT + 1) / 2;
    const dim3 grid(tiles, unsigned(p.slots), unsigned(p.splits));
    if (p.one) {
        lora_one_kernel<ACT, RT><<<dim3(unsigned(ceil_div(a.n, 256))), dim3(512), 0, stream>>>(a);
    } else if (p.tall) {
        uint4* operands = reinterpret_cast<uint4*>(t);
        float* factors = reinterpret_cast<float*>(operands + int64_t(tiles) * RS * 128);
        lora_shrink_kernel<ACT, RT, 16, true><<<grid, dim3(512), 0, stream>>>(a, p.slots, int(p.kspan), t, operands, factors);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        lora_expand_rows_kernel<ACT, RS><<<dim3(unsigned(ceil_div(a.n, kTallCols)), unsigned(ceil_div(a.m, kTallRows))), dim3(256), 0, stream>>>(a, operands, factors);
    } else {
        const bool wide = p.tile == 64;
        if (wide) lora_shrink_kernel<ACT, RT, 64, false><<<grid, dim3(256), 0, stream>>>(a, p.slots, int(p.kspan), t, nullptr, nullptr);
        else lora_shrink_kernel<ACT, RT, 16, false><<<grid, dim3(256), 0, stream>>>(a, p.slots, int(p.kspan), t, nullptr, nullptr);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        const dim3 columns(unsigned(ceil_div(a.n, 256)), tiles, unsigned(p.slots));
        if (wide) lora_expand_kernel<ACT, RS, 64><<<columns, dim3(256), 0, stream>>>(a, p.slots, p.splits, t);
        else lora_expand_kernel<ACT, RS, 16><<<columns, dim3(256), 0, stream>>>(a, p.slots, p.splits, t);
    }
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
    // One launch for a row or two whose workgroups read no more than 128 KB of A each (2048 x 2560, rank 16: 1 row 5.3 us
    // against 7.9 in two launches, 2 rows 6.6 against 8.2; rank 64, twice that limit: 11.7 against 10.2).
    p.one = m <= 2 && m * rank * k <= int64_t(1) << 16;
    p.tall = ceil_div(m, kTallRows) * ceil_div(n, kTallCols) >= 512;
    // Few rows: a tile of 64 reads an adapter's weights once where a tile of 16 reads them up to four times (64 rows, 16
    // adapters of rank 64, 4096 x 16384: 26 us against 42), but a few adapters make too few workgroups of it (64 rows, 2
    // adapters, 4096 x 4096: 22 us against 15).
    p.tile = p.tall || m <= 16 || adapters < 8 ? 16 : 64;
    const int64_t tiles = ceil_div(m, p.tile);
    // Slots: one for every adapter while the launches are small; a tall call's tile of 16 seldom holds more than the
    // end of one request and the start of the next.
    int64_t slots = p.tall ? 2 : ceil_div(1024, tiles * ceil_div(n, 256));
    if (slots > p.tile) slots = p.tile;
    if (slots > adapters) slots = adapters;
    if (slots > m) slots = m;
    p.slots = int(slots);
    // parts of K that make 256 workgroups, in whole turns of their waves (64 rows, 48 adapters of rank 16, 4096 x 4096:
    // 12.9 us; 512 workgroups 13.7, 128 14.8: each part is another read of the second launch)
    int64_t splits = p.tall ? 1 : ceil_div(256, tiles * slots);
    if (splits > 16) splits = 16;
    const int64_t turn = rank > 64 ? 256 : 512;
    p.kspan = p.tall ? k : ceil_div(ceil_div(k, splits), turn) * turn;
    p.splits = int(ceil_div(k, p.kspan));
    // sums [split][row][rank], or operands (2 KB a row tile and 32-wide step of the rank) and a factor a row
    p.workspace = p.one    ? 0
                  : p.tall ? size_t(tiles) * (size_t(rank <= 32 ? 1 : rank <= 64 ? 2 : 4) * 2048 + 64)
                           : size_t(p.splits) * size_t(m) * size_t(rank) * 4;
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
