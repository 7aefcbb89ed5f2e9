// Attention over the 4-bit paged cache (kv4.h):
//
//   o[i, h] = sum_t p[t] v[t],  p = softmax over the visible t of
//             scale q[i, h] . k[t],  k[t] = ks[t] ck[t], v[t] = vs[t] cv[t]
//
// with FP32 scales ks, vs per token, head and block of W channels and codes
// ck, cv.  Query heads share key heads: the rows of one (request, key head)
// are its query tokens times the heads that share it, cut into tiles of 16.
//
// The codes go to the matrix cores as exact f16 integers and the scales are
// applied in FP32 outside: the key's to the product, the value's to the
// probability before its rounding to f16.  Queries enter as f16 scaled by a
// power of two per row (exact for bf16 and f16 inputs up to f16's subnormals
// 34 binades below the row's largest).  The weights p vs are rounded to f16
// relative to the row's largest of them (Running), so they use f16's range
// whatever the values' size.  Their rounding (2^-11 of each) is an eighth of a
// bf16 output's own and as coarse as an f16 output's: against 64 bits f16 rows
// are off by 2.9e-4 where FP32 weights give 2.1e-4 (bf16 1.67e-3 and 1.66e-3).
// A second f16 part of the weights takes that away and costs f16 calls a second
// product (prompt of 4096 tokens 194 -> 234 us, 4 of 131072 104 -> 116, 12
// windowed pieces 29 -> 33); one part is kept for both types, as the codes in the
// cache are themselves off by up to 1/14 of a group's largest value.  The sum and
// the output accumulate in FP32.
#include "kernels.h"
#include "kv4.h"

namespace w4a16 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ inline f32x4_t mfma(uint4 a, uint4 b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
}

__device__ inline uint32_t pack_f16(float a, float b) {
    const f16x2_t v = {_Float16(a), _Float16(b)};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ inline float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// max / sum over the four lanes of one row (lanes differing in bits 4 and 5)
__device__ inline float row_max(float v) { return max_xor32(fmaxf(v, lane_xor<16>(v))); }
__device__ inline float row_sum(float v) { return sum_xor32(v + lane_xor<16>(v)); }

// What a tile of rows sees.
struct Tile {
    int64_t q0;   // first query token of the request
    int r0, rows; // first row of the tile, rows of the request
    int b, kv, qn;
    __device__ int position(int i) const { return kv - qn + i; }
};

struct View {
    int causal, window;
    __device__ int lo(int pos) const { return window ? max(0, pos - window + 1) : 0; }
    __device__ int hi(int pos, int kv) const {
        return max(0, causal ? min(kv, pos + 1) : window ? min(kv, pos + window) : kv);
    }
};

// What a launch computes: a whole attention, the part of it over the groups'
// shared prefixes, whose splits leave their sums as they are, the part over the
// requests' own tokens, which begins with those sums, or each request's prefix
// and own tokens one after the other.
enum Part { kWhole = 0, kPrefix = 1, kOwn = 2, kBoth = 3 };

// First query token of group j (a request outside the batch is its end).
__device__ inline int64_t group_start(const Kv4AttentionArgs& a, int64_t j) {
    int64_t b = a.cu_groups ? a.cu_groups[j] : j ? a.batch : 0;
    b = b < 0 ? 0 : b > a.batch ? a.batch : b;
    return a.cu_q ? a.cu_q[b] : b;
}

// The group of request b (-1: none), and how many tokens its prefix has.
__device__ inline int group_of(const Kv4AttentionArgs& a, int b) {
    if (!a.cu_groups) return 0;
    int lo = 0, hi = int(a.groups) - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.cu_groups[mid] <= b) lo = mid;
        else hi = mid - 1;
    }
    return b >= a.cu_groups[lo] && b < a.cu_groups[lo + 1] ? lo : -1;
}
__device__ inline int prefix_len(const Kv4AttentionArgs& a, int group) {
    const int64_t n = a.prefix_lens[group], room = a.prefix_width * a.page;
    return int(n < 0 ? 0 : n > room ? room : n);
}

// Tokens of a part where `tokens` are cut into at most `splits` parts (kPrefix, kBoth): even ones of at least 128 tokens and
// sqrt(kPartRoot tokens).  The host knows how far a table reaches, the device how long a sequence is, and tables of captured
// steps have room: parts cut from their width left 64 x 32/8 heads on 8192 tokens in a table of 131072 two parts of 25, 155
// us, where an exact table took 48.  So the width bounds the grid and the length cuts the parts, by this function in both
// launches alike.
template <int PART>
constexpr int kPartRoot = PART == kPrefix ? 48 : 12;
template <int PART>
__host__ __device__ inline int part_span(int tokens, int splits) {
    const int even = (tokens + splits - 1) / splits, least = int(ceilf(sqrtf(float(kPartRoot<PART>) * float(tokens))));
    const int span = even > least ? even : least;
    return span <= 128 ? 128 : (span + 63) / 64 * 64;
}

// Tiles are numbered without a table: request b's start at
// floor(cu_q[b] share / ROWS) + b, which leaves room for the ragged last tile
// of every request (a few tiles stay empty).  Over the prefixes a group takes a
// request's place, with the queries of all its requests.
template <int ROWS, int PART>
__device__ inline bool find_tile(const Kv4AttentionArgs& a, int64_t x, Tile& t) {
    const int share = a.heads / a.kv_heads;
    if (PART != kPrefix && !a.cu_q) {
        const int per = (share + ROWS - 1) / ROWS;
        t.b = int(x / per);
        t.q0 = t.b;
        t.qn = 1;
        t.r0 = int(x % per) * ROWS;
    } else {
        auto first = [&](int64_t b) -> int64_t {
            if constexpr (PART == kPrefix) return group_start(a, b);
            else return a.cu_q[b];
        };
        int lo = 0, hi = int(PART == kPrefix ? a.groups : a.batch) - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            const int64_t start = first(mid) * share / ROWS + mid;
            if (start <= x) lo = mid;
            else hi = mid - 1;
        }
        t.b = lo;
        const int64_t c0 = first(lo), c1 = first(lo + 1);
        t.q0 = c0 < 0 ? 0 : c0 > a.tokens ? a.tokens : c0;
        const int64_t q1 = c1 < t.q0 ? t.q0 : c1 > a.tokens ? a.tokens : c1;
        t.qn = int(q1 - t.q0);
        const int64_t r0 = (x - (c0 * share / ROWS + lo)) * ROWS;
        if (r0 < 0 || r0 >= int64_t(t.qn) * share) return false;
        t.r0 = int(r0);
    }
    t.rows = t.qn * share;
    const int64_t room = a.table_width * a.page;
    const int64_t kv = a.kv_lens[t.b];
    t.kv = int(kv < 0 ? 0 : kv > room ? room : kv);
    return true;
}

// Where the 16-token chunks of a wave's steps lie, for 32 steps at a time: lane
// L holds chunk L % 2 of step L / 2, so a step finds its chunks with scalar
// reads of lanes instead of a page lookup (a scalar load and its wait) each.
// Offsets are in units of 128 bytes (codes) and 64 bytes (scales): 32 bits
// reach every pool that fits a GPU.
struct Chunks {
    uint32_t code, scale;
    uint64_t there;  // bit L: lane L's chunk is on a page of the pool
    // stride: chunks between a wave's steps; end: tokens
    __device__ void find(const Kv4AttentionArgs& a, uint32_t magic, const int32_t* row, int64_t region, int chunk_bytes,
                         int first, int stride, int end, int lane) {
        const int c = first + lane / 2 * stride + lane % 2;
        const int per = a.page / 16;
        const int p = per == 1 ? c : int(__umulhi(uint32_t(c), magic));
        const int in = c - p * per;
        int id = -1;
        if (c * 16 < end && p < int(a.table_width)) id = row[p];
        place(a, id, in, region, chunk_bytes);
    }
    // The same along a prefix of `len` tokens, padded to `own` (a multiple of 32), and the request's tokens behind it.
    __device__ void find_both(const Kv4AttentionArgs& a, uint32_t magic, const int32_t* prefix, int len, int own, const int32_t* row,
                              int64_t region, int chunk_bytes, int first, int stride, int end, int lane) {
        const int at = first + lane / 2 * stride + lane % 2;
        const bool mine = at * 16 >= own;
        const int c = mine ? at - own / 16 : at;
        const int per = a.page / 16;
        const int p = per == 1 ? c : int(__umulhi(uint32_t(c), magic));
        const int in = c - p * per;
        int id = -1;
        if (mine ? at * 16 < end && p < int(a.table_width) : c * 16 < len && p < int(a.prefix_width)) id = mine ? row[p] : prefix[p];
        place(a, id, in, region, chunk_bytes);
    }
    __device__ void place(const Kv4AttentionArgs& a, int id, int in, int64_t region, int chunk_bytes) {
        const bool ok = id >= 0 && id < a.pages;
        const uint64_t at = uint64_t(ok ? id : 0) * uint64_t(a.kv_heads * region);
        code = ok ? uint32_t((at + uint64_t(in) * chunk_bytes) >> 7) : 0;
        scale = ok ? uint32_t((at + uint64_t(a.page) * a.dim + in * 64) >> 6) : 0;
        there = __ballot(ok);
    }
    __device__ uint64_t code_at(int i) const { return uint64_t(uint32_t(__builtin_amdgcn_readlane(int(code), i))) << 7; }
    __device__ uint64_t scale_at(int i) const { return uint64_t(uint32_t(__builtin_amdgcn_readlane(int(scale), i))) << 6; }
};

// One side (keys or values) of 32 tokens of one key head, as loaded.
template <int D>
struct Side {
    static constexpr int W = kv4_width(D), NB = kv4_blocks(D);
    uint32_t w[2][NB][W / 32];
    float4 s[2][NB];

    __device__ static void words(const uint8_t* p, uint32_t (&w)[W / 32]) {
        if constexpr (W == 128) {
            const uint4 x = load_stream16(p);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else {
            typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
            const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
            w[0] = x.x; w[1] = x.y;
        }
    }
    // codes, scales: this head's region of page 0, at the side
    __device__ void load(const uint8_t* codes, const uint8_t* scales, const Chunks& ch, int step, int page, int lane) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint8_t* p = codes + ch.code_at(2 * step + c);
            const uint8_t* q = scales + ch.scale_at(2 * step + c);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                words(p + b * (8 * W) + uint32_t(lane * (W / 8)), w[c][b]);
                s[c][b] = *reinterpret_cast<const float4*>(q + b * page * 4 + uint32_t(lane / 16 * 16));
            }
        }
    }
};

// Workspace of a split: per (tile, key head, split) the accumulators in lane
// order, then the 16 rows' references and sums.
template <int D>
constexpr int64_t partial_floats() { return 16 * D + 32; }

// One row's queries as f16, scaled by 2^e; what undoes it in the logits' base-2
// exponent; and -24 sum(q) per block.
template <int ACT, int D>
__device__ inline float load_queries(const uint16_t* src, float scale, uint4 (&q)[kv4_blocks(D)][kv4_width(D) / 32],
                                     float (&offset)[kv4_blocks(D)]) {
    constexpr int W = kv4_width(D), NB = kv4_blocks(D);
    uint4 raw[NB][W / 32];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int s = 0; s < W / 32; ++s) raw[b][s] = *reinterpret_cast<const uint4*>(src + W * b + 32 * s);
    float big = 0.0f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int s = 0; s < W / 32; ++s) {
            const uint32_t w[4] = {raw[b][s].x, raw[b][s].y, raw[b][s].z, raw[b][s].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                big = fmaxf(big, fmaxf(fabsf(to_f32<ACT>(uint16_t(w[i]))), fabsf(to_f32<ACT>(uint16_t(w[i] >> 16)))));
        }
    big = row_max(big);
    const int e = big > 0.0f && big < INFINITY ? 10 - (int(__float_as_uint(big) >> 23) - 127) : 0;
    const float sign = scale < 0.0f ? -1.0f : 1.0f;  // the logits' factor is positive
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        float sum = 0.0f;
#pragma unroll
        for (int s = 0; s < W / 32; ++s) {
            const uint32_t w[4] = {raw[b][s].x, raw[b][s].y, raw[b][s].z, raw[b][s].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = pack_f16(sign * ldexpf(to_f32<ACT>(uint16_t(w[i])), e), sign * ldexpf(to_f32<ACT>(uint16_t(w[i] >> 16)), e));
            q[b][s] = make_uint4(o[0], o[1], o[2], o[3]);
            sum += sum8<kActF16>(q[b][s]);
        }
        offset[b] = -kKvOffset * row_sum(sum);
    }
    // never 0, which would make a masked logit (-inf) NaN
    return fmaxf(ldexpf(fabsf(scale) * kLog2e, -e), 1e-37f);
}

// A row's running softmax over some of its tokens: probabilities p = 2^(z - ref)
// in FP32 and weights p vs, which are rounded to f16.  The reference follows the
// largest weight, not the largest logit and value scale apart: a token with large
// values that the softmax leaves out must not push the others' weights below f16's
// normal numbers.  A new reference puts the largest weight seen at 2^5, and the
// next comes when one exceeds 2^15, so the sums so far are rescaled a few times a
// row instead of at every new maximum (prompt of 4096 tokens: 237 -> 209 us).
// Weights then have all of f16's 11 bits down to 2^-19 of the row's largest or
// lower, and an absolute error of 2^-30 of it below.  Scales count from 2^-80 up:
// tokens without values have p of at most 2^85, whose sum FP32 holds.
struct Running {
    static constexpr float kTop = 5.0f, kMaxWeight = 32768.0f, kMaxP = 0x1p+90f, kMinScale = 0x1p-80f;
    float ref = -INFINITY;
    float sum = 0.0f;  // this lane's part of the row's sum
    // what logits (base 2) are relative to; before the first reference so low that any logit calls for one
    __device__ float base() const { return fmaxf(ref, -3e38f); }
    // a new reference from the row's largest log2 of a weight; returns what the sums so far are to be multiplied by
    __device__ float raise(float top) {
        const float now = fmaxf(ref, top - kTop);
        const float f = ref == -INFINITY ? 0.0f : exp2_fast(ref - now);
        ref = now;
        sum *= f;
        return f;
    }
};

// One step's probabilities and weights of a row: z (logits before the factor zf,
// -inf where masked), vs (0 where masked).  scale(f) multiplies the output sums so far.
template <int NB, typename F>
__device__ inline void weigh(Running& run, const float (&z)[2][4], float zf, const float (&vs)[2][NB][4], float (&p)[2][4],
                             float (&w)[2][NB][4], F&& scale) {
    auto compute = [&]() {
        const float base = run.base();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[c][i] = exp2_fast(fmaf(z[c][i], zf, -base));
#pragma unroll
                for (int b = 0; b < NB; ++b) w[c][b][i] = p[c][i] * vs[c][b][i];
            }
    };
    compute();
    float pm = 0.0f, wm = 0.0f;
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            pm = fmaxf(pm, p[c][i]);
#pragma unroll
            for (int b = 0; b < NB; ++b) wm = fmaxf(wm, w[c][b][i]);
        }
    if (__any(pm > Running::kMaxP || wm > Running::kMaxWeight)) {
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v = Running::kMinScale;
#pragma unroll
                for (int b = 0; b < NB; ++b) v = fmaxf(v, vs[c][b][i]);
                top = fmaxf(top, fmaf(z[c][i], zf, __builtin_amdgcn_logf(v)));
            }
        scale(run.raise(row_max(top)));
        compute();
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) run.sum += p[c][i];
}

// The weights of a block as an operand of the second product.
template <int NB>
__device__ inline uint4 weights(const float (&w)[2][NB][4], int b) {
    return make_uint4(pack_f16(w[0][b][0], w[0][b][1]), pack_f16(w[0][b][2], w[0][b][3]),
                      pack_f16(w[1][b][0], w[1][b][1]), pack_f16(w[1][b][2], w[1][b][3]));
}

// What a split of the prefixes' launch leaves of a row, and where its request's own part begins.
struct Left {
    float *sums, *stats;  // a lane's channels: CH consecutive ones for each block and register; {reference, sum of probabilities}
    __device__ Left(const Kv4AttentionArgs& a, int split, int64_t token, int head) {
        const int64_t rows = a.tokens * a.heads, row = split * rows + token * a.heads + head;
        sums = a.parts + row * a.dim;
        stats = a.parts + a.prefix_splits * rows * a.dim + row * 2;
    }
};

template <int D>
__device__ inline void leave(const Left& to, const f32x4_t (&acc)[kv4_blocks(D)][kv4_width(D) / 16], float ref, float sum, int kq) {
    constexpr int W = kv4_width(D), NB = kv4_blocks(D), CH = W / 16;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < CH; i += 4)
                *reinterpret_cast<float4*>(to.sums + W * b + CH * (4 * kq + j) + i) =
                    make_float4(acc[b][i][j], acc[b][i + 1][j], acc[b][i + 2][j], acc[b][i + 3][j]);
    if (kq == 0) *reinterpret_cast<float2*>(to.stats) = make_float2(ref, sum);
}

// Splits of the prefix that request b shares (0: it is in no group), as the prefixes' launch cut it.
__device__ inline int prefix_splits(const Kv4AttentionArgs& a, int b) {
    const int group = group_of(a, b);
    if (group < 0) return 0;
    const int len = prefix_len(a, group), span = part_span<kPrefix>(len, a.prefix_splits);
    return max(1, min(a.prefix_splits, (len + span - 1) / span));
}

// A wave begins its running softmax of a row with the prefix's splits first, first + step, ... < live: they are as good as
// tokens that it has seen before its own.
template <int D>
__device__ inline void take(const Kv4AttentionArgs& a, int first, int live, int step, int64_t token, int head, int kq, Running& run,
                            f32x4_t (&acc)[kv4_blocks(D)][kv4_width(D) / 16]) {
    constexpr int W = kv4_width(D), NB = kv4_blocks(D), CH = W / 16;
    for (int s = first; s < live; s += step) {
        const Left from(a, s, token, head);
        const float2 st = *reinterpret_cast<const float2*>(from.stats);
        float4 v[NB][4][CH / 4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < CH / 4; ++i) v[b][j][i] = *reinterpret_cast<const float4*>(from.sums + W * b + CH * (4 * kq + j) + 4 * i);
        const float now = fmaxf(run.ref, st.x);
        const float f0 = run.ref == -INFINITY ? 0.0f : exp2_fast(run.ref - now);
        const float f1 = st.x == -INFINITY ? 0.0f : exp2_fast(st.x - now);
        run.ref = now;
        run.sum = run.sum * f0 + (kq == 0 ? st.y * f1 : 0.0f);  // the lanes of a row add theirs at the end
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < CH / 4; ++i) {
                    acc[b][4 * i][j] = acc[b][4 * i][j] * f0 + v[b][j][i].x * f1;
                    acc[b][4 * i + 1][j] = acc[b][4 * i + 1][j] * f0 + v[b][j][i].y * f1;
                    acc[b][4 * i + 2][j] = acc[b][4 * i + 2][j] * f0 + v[b][j][i].z * f1;
                    acc[b][4 * i + 3][j] = acc[b][4 * i + 3][j] * f0 + v[b][j][i].w * f1;
                }
    }
}

constexpr uint32_t kOnes = 0x3C003C00u;  // two f16 ones

// One workgroup: 16 rows of one key head over one split of the tokens.  Its
// four waves take steps of 32 tokens in turn, each with its own running
// softmax, and meet in LDS at the end.  The next step's keys are loaded as soon
// as this step's have been used, and the values likewise, so each side has one
// set of registers and half a step or more of work to arrive behind, and three
// waves fit a SIMD (four for D = 64, two for D = 256).  Splits are joined by the
// last of a tile's workgroups to finish, in split order.
//
// HBM bounds long contexts: 4 requests of 131072 tokens, 8 heads of 128, 570 MB,
// take 98 to 105 us, 5.4 to 5.8 TB/s.  Shorter ones are bounded by the chain of
// dependent accesses of a part (lengths, pages, codes, join; 5 to 8 us): 64
// requests of 0 to 8192 tokens 84 us (3.4 TB/s), 1 of 1000 tokens 10.5 us at D =
// 256.  Equal stretches of all requests' tokens a workgroup, in one round, pay
// that chain twice and were slower (95 us, where these splits took 89).
template <int ACT, int D, int PART>
__global__ __launch_bounds__(256, D == 256 ? 2 : D == 128 ? 3 : 4) void kv4_attention_kernel(Kv4AttentionArgs a, int span, int splits,
                                                                              uint32_t magic, unsigned* counters,
                                                                              float* partials) {
    constexpr int W = kv4_width(D), NB = kv4_blocks(D), CH = W / 16;
    constexpr int WAVES = 4;
    __shared__ float lds[WAVES / 2][NB * CH * 4 + 2][64];
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int col = lane % 16, kq = lane / 16;
    const int kh = blockIdx.y, share = a.heads / a.kv_heads;

    Tile t;
    if (!find_tile<16, PART>(a, blockIdx.x, t)) return;
    const View view{a.causal, int(a.window)};
    const int last = min(t.r0 + 15, t.rows - 1);
    const int p_first = t.position(t.r0 / share), p_last = t.position(last / share);
    // kBoth: tokens [0, len) are the prefix's, those from `own` on the request's
    const int group = PART == kBoth ? group_of(a, t.b) : -1, len = group < 0 ? 0 : prefix_len(a, group), own = (len + 31) / 32 * 32;
    const int begin = view.lo(p_first) / 32 * 32, end = own + view.hi(p_last, t.kv);
    if constexpr (PART == kPrefix || PART == kBoth) span = part_span<PART>(end, splits);  // (no window: they begin at 0)
    const int live = max(1, min(splits, (end - begin + span - 1) / span));  // splits with tokens
    if (int(blockIdx.z) >= live) return;
    const int s0 = begin + int(blockIdx.z) * span, s1 = min(end, s0 + span);
    // every row of the tile sees [all_lo, all_hi)
    const int all_lo = view.lo(p_last), all_hi = min(own + view.hi(p_first, t.kv), s1);

    const int64_t region = kv4_region(a.page, D);
    const uint8_t* pool = a.pool + kh * region;
    const int32_t* row = a.table + int64_t(t.b) * a.ldt;
    const int first = s0 + 32 * wave, steps = max(0, (s1 - first + 32 * WAVES - 1) / (32 * WAVES));
    Chunks ch;
    auto find = [&](int chunk) {
        if constexpr (PART == kBoth)
            ch.find_both(a, magic, a.prefix_table + (group < 0 ? 0 : group) * a.ldp, len, own, row, region, NB * 8 * W, chunk, 2 * WAVES, s1, lane);
        else ch.find(a, magic, row, region, NB * 8 * W, chunk, 2 * WAVES, s1, lane);
    };
    find(first / 16);
    Side<D> k, v;
    if (steps > 0) {
        k.load(pool, pool, ch, 0, a.page, lane);
        v.load(pool + a.page * (D / 2), pool + NB * a.page * 4, ch, 0, a.page, lane);
    }

    // columns past the last row repeat it, and are dropped at the end
    const int r = min(t.r0 + col, last);
    const int qi = r / share, hd = kh * share + r % share;
    const int pos = t.position(qi);
    const int lo = view.lo(pos), hi = min(own + view.hi(pos, t.kv), s1);
    uint4 q[NB][W / 32];
    float offset[NB];
    const float zf = load_queries<ACT, D>(a.q + (t.q0 + qi) * a.ldq + int64_t(hd) * D + 8 * kq, a.scale, q, offset);

    f32x4_t acc[NB][CH], ps[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        ps[b] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < CH; ++i) acc[b][i] = f32x4_t{0, 0, 0, 0};
    }
    Running run;

    if constexpr (PART == kOwn) {
        if (blockIdx.z == 0) take<D>(a, wave, prefix_splits(a, t.b), WAVES, t.q0 + qi, hd, kq, run, acc);
    }
    for (int step = 0; step < steps; ++step) {
        const int tok = first + step * 32 * WAVES;
        const uint32_t there = uint32_t(ch.there >> (2 * (step % 32))) & 3;
        float z[2][4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                f32x4_t s = {offset[b], offset[b], offset[b], offset[b]};
#pragma unroll
                for (int ks = 0; ks < W / 32; ks += 2) {
                    uint32_t x[4], y[4];
                    kv4_pairs(k.w[c][b][ks], k.w[c][b][ks + 1], x, y);
                    s = mfma(make_uint4(x[0], x[1], x[2], x[3]), q[b][ks], s);
                    s = mfma(make_uint4(y[0], y[1], y[2], y[3]), q[b][ks + 1], s);
                }
                const float4 f = k.s[c][b];
                const float y[4] = {s[0] * f.x, s[1] * f.y, s[2] * f.z, s[3] * f.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) z[c][i] = b == 0 ? y[i] : z[c][i] + y[i];
            }
        }
        const bool more = step + 1 < steps;
        if (more) {
            if ((step + 1) % 32 == 0) find((tok + 32 * WAVES) / 16);
            k.load(pool, pool, ch, (step + 1) % 32, a.page, lane);
        }
        float vs[2][NB][4];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                vs[c][b][0] = v.s[c][b].x; vs[c][b][1] = v.s[c][b].y; vs[c][b][2] = v.s[c][b].z; vs[c][b][3] = v.s[c][b].w;
            }
        if (!(tok >= all_lo && tok + 32 <= all_hi && there == 3) || (PART == kBoth && tok < own && tok + 32 > len)) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = tok + 16 * c + 4 * kq + i;
                    const bool seen = (there >> c & 1) && at >= lo && at < hi && (PART != kBoth || at < len || at >= own);
                    z[c][i] = seen ? z[c][i] : -INFINITY;
#pragma unroll
                    for (int b = 0; b < NB; ++b) vs[c][b][i] = seen ? vs[c][b][i] : 0.0f;
                }
        }
        float p[2][4], w[2][NB][4];
        weigh<NB>(run, z, zf, vs, p, w, [&](float f) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                ps[b] *= f;
#pragma unroll
                for (int i = 0; i < CH; ++i) acc[b][i] *= f;
            }
        });
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint4 pw = weights<NB>(w, b);
            ps[b] = mfma(make_uint4(kOnes, kOnes, kOnes, kOnes), pw, ps[b]);
#pragma unroll
            for (int h = 0; h < CH / 4; ++h) {
                uint32_t x[2][4], y[2][4];
#pragma unroll
                for (int c = 0; c < 2; ++c) kv4_pairs(v.w[c][b][2 * h], v.w[c][b][2 * h + 1], x[c], y[c]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[b][4 * h + i] = mfma(make_uint4(x[0][i], y[0][i], x[1][i], y[1][i]), pw, acc[b][4 * h + i]);
            }
        }
        if (more) v.load(pool + a.page * (D / 2), pool + NB * a.page * 4, ch, (step + 1) % 32, a.page, lane);
    }

    // take the offset out, then join the waves two and two
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < CH; ++i) acc[b][i] -= kKvOffset * ps[b];
    float ref = run.ref, sum = run.sum;
#pragma unroll
    for (int half = WAVES / 2; half > 0; half /= 2) {
        if (wave >= half && wave < 2 * half) {
            float(*o)[64] = lds[wave - half];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < CH; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[(b * CH + i) * 4 + j][lane] = acc[b][i][j];
            o[NB * CH * 4][lane] = ref;
            o[NB * CH * 4 + 1][lane] = sum;
        }
        __syncthreads();
        if (wave < half) {
            const float(*o)[64] = lds[wave];
            const float other = o[NB * CH * 4][lane];
            const float now = fmaxf(ref, other);
            const float f0 = ref == -INFINITY ? 0.0f : exp2_fast(ref - now);
            const float f1 = other == -INFINITY ? 0.0f : exp2_fast(other - now);
            ref = now;
            sum = sum * f0 + o[NB * CH * 4 + 1][lane] * f1;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < CH; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[b][i][j] = acc[b][i][j] * f0 + o[(b * CH + i) * 4 + j][lane] * f1;
        }
        __syncthreads();
    }
    uint16_t* dst = a.out + (t.q0 + qi) * a.ldo + int64_t(hd) * D;
    if (PART == kPrefix || live == 1) {
        if (wave != 0 || t.r0 + col > last) return;
        sum = row_sum(sum);
        if constexpr (PART == kPrefix) {
            leave<D>(Left(a, int(blockIdx.z), t.q0 + qi, hd), acc, ref, sum, kq);
            return;
        }
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t w[CH / 2];
#pragma unroll
                for (int i = 0; i < CH / 2; ++i)
                    w[i] = uint32_t(from_f32<ACT>(acc[b][2 * i][j] * inv)) | (uint32_t(from_f32<ACT>(acc[b][2 * i + 1][j] * inv)) << 16);
                uint16_t* to = dst + W * b + CH * (4 * kq + j);
                if constexpr (CH == 8) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
                else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
            }
        return;
    }

    // A split stores its sums past the L2 (SC1: the XCDs' L2s are not coherent)
    // and counts itself; the one that completes the count joins them all and
    // clears the counter for the next call.  Nobody waits.
    const int64_t tile = int64_t(blockIdx.x) * a.kv_heads + kh;
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    constexpr int kSlot = int(partial_floats<D>() * 4), kRefs = 16 * D * 4;
    const __amdgpu_buffer_rsrc_t slots = buffer_rsrc(partials + tile * splits * partial_floats<D>(), int64_t(splits) * kSlot);
    int* last_one = reinterpret_cast<int*>(&lds[1][0][0]);  // the second join round read lds[0] only
    if (wave == 0) {
        sum = row_sum(sum);
        const int at = int(blockIdx.z) * kSlot;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < CH; ++i)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[b][i]), slots,
                                                       at + ((b * CH + i) * 64 + lane) * 16, 0, kCoherent);
        if (kq == 0) {
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(ref), slots, at + kRefs + col * 4, 0, kCoherent);
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sum), slots, at + kRefs + 64 + col * 4, 0, kCoherent);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if (lane == 0) {
            const unsigned before = __hip_atomic_fetch_add(counters + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            *last_one = before == unsigned(live - 1);
            if (*last_one) __hip_atomic_store(counters + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    __syncthreads();
    if (!*last_one) return;
    // wave w joins the accumulators i = PER w .. PER w + PER - 1 of each block
    constexpr int PER = CH / WAVES;
    float total = 0.0f;
    ref = -INFINITY;
    f32x4_t out[NB][PER];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < PER; ++i) out[b][i] = f32x4_t{0, 0, 0, 0};
    constexpr int BATCH = 8;
    for (int sp = 0; sp < live; sp += BATCH) {
        u32x4 part[BATCH][NB][PER];
        float refs[BATCH], sums[BATCH];
#pragma unroll
        for (int g = 0; g < BATCH; ++g) {
            const int at = min(sp + g, live - 1) * kSlot;
            refs[g] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(slots, at + kRefs + col * 4, 0, kCoherent));
            sums[g] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(slots, at + kRefs + 64 + col * 4, 0, kCoherent));
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    part[g][b][i] = __builtin_amdgcn_raw_buffer_load_b128(slots, at + ((b * CH + PER * wave + i) * 64 + lane) * 16, 0, kCoherent);
        }
        float now = ref;
#pragma unroll
        for (int g = 0; g < BATCH; ++g) now = fmaxf(now, refs[g]);
        const float keep = ref == -INFINITY ? 0.0f : exp2_fast(ref - now);
        ref = now;
        total *= keep;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < PER; ++i) out[b][i] *= keep;
#pragma unroll
        for (int g = 0; g < BATCH; ++g) {
            const float f = sp + g < live && refs[g] > -INFINITY ? exp2_fast(refs[g] - now) : 0.0f;
            total += sums[g] * f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < PER; ++i) out[b][i] += __builtin_bit_cast(f32x4_t, part[g][b][i]) * f;
        }
    }
    if (t.r0 + col > last) return;
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint16_t* to = dst + W * b + CH * (4 * kq + j) + PER * wave;
            if constexpr (PER == 2)
                *reinterpret_cast<uint32_t*>(to) = uint32_t(from_f32<ACT>(out[b][0][j] * inv)) | (uint32_t(from_f32<ACT>(out[b][1][j] * inv)) << 16);
            else
                *to = from_f32<ACT>(out[b][0][j] * inv);
        }
}

// ---------------------------------------------------------------------------
// Many rows of a request (prompts, prompt pieces, action chunks).
//
// One workgroup: 64 rows of one key head over one split of the tokens.  Each of
// the four waves owns 16 rows and all walk the same tokens, so the codes become
// f16 once a workgroup: each wave turns a quarter of the next step's codes into
// matrix operands in LDS (in operand order: reads and writes of 16 bytes a lane,
// no conflicts) while this step is computed, one barrier a step, raw codes
// loaded a step before that.  32 rows a wave halve the operand reads but leave
// registers for two waves a SIMD instead of four, which costs more (16 x 64
// queries on 1000 tokens, D = 128: 54 us against 44; prompt of 4096: 205 against
// 193).  What bounds it is the issue of instructions: over a prompt of 4096 (186
// to 212 us) matrix units are busy 30 % of the cycles and vector units 65 %, and
// beside 70.7 M vector (9.0 M of them matrix) and 13.1 M LDS instructions stand
// 34.1 M scalar ones, mostly chunk addresses and mask bounds; copies that leave
// out the staging, the exponentials or the products each save what those cost.
// ---------------------------------------------------------------------------
template <int D>
struct Stage {
    static constexpr int W = kv4_width(D), NB = kv4_blocks(D), CH = W / 16;
    static constexpr int SUB = D == 64 ? 2 : 1;       // 32-token parts of a step
    static constexpr int KF = 2 * NB * (W / 32), VF = NB * CH;  // operands of a part, 1 KB each
    uint4 k[SUB][KF][64], v[SUB][VF][64];
    float ks[SUB][NB][32], vs[SUB][NB][32];
};

// A wave's quarter of a step: D >= 128: keys of chunk 0, of chunk 1, the values'
// words 0 and 1 of both chunks, words 2 and 3.  D = 64 (two parts a step): keys
// of part 0, of part 1, values of part 0, of part 1.
template <int D>
struct Quarter {
    using S = Stage<D>;
    static constexpr int W = S::W, NB = S::NB;
    uint32_t w[NB][4];
    float scale;

    __device__ static uint2 load8(const uint8_t* p) {
        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 x = *reinterpret_cast<const u32x2*>(p);
        return make_uint2(x.x, x.y);
    }
    // c0: the step's first chunk in ch
    __device__ void load(const uint8_t* pool, const Chunks& ch, int c0, int page, int wave, int lane) {
        const bool values = wave >= 2;
        const int u = wave & 1;
        const uint8_t* codes = pool + (values ? page * (D / 2) : 0);
        const uint8_t* scales = pool + (values ? NB * page * 4 : 0);
        const int ca = c0 + (D == 64 ? 2 * u : 0), cb = ca + 1;
        const uint64_t at0 = ch.code_at(ca), at1 = ch.code_at(cb), sc0 = ch.scale_at(ca), sc1 = ch.scale_at(cb);
        if (D != 64 && !values) {
            const uint8_t* p = codes + (u ? at1 : at0) + uint32_t(lane * 16);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint4 x = *reinterpret_cast<const uint4*>(p + b * (8 * W));
                w[b][0] = x.x; w[b][1] = x.y; w[b][2] = x.z; w[b][3] = x.w;
            }
        } else {
            const uint32_t in = uint32_t(lane * (W / 8) + (D == 64 ? 0 : 8 * u));
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint2 x = load8(codes + at0 + b * (8 * W) + in), y = load8(codes + at1 + b * (8 * W) + in);
                w[b][0] = x.x; w[b][1] = x.y; w[b][2] = y.x; w[b][3] = y.y;
            }
        }
        // scales: 16 lanes a chunk and block
        const int g = lane / 16;
        const bool both = D == 64 || values;  // of both chunks, else of chunk u
        const int c = both ? g & 1 : u, b = both ? g >> 1 : g;
        if (b < NB && !(D != 64 && values && u))
            scale = *reinterpret_cast<const float*>(scales + (c ? sc1 : sc0) + (b * page + lane % 16) * 4);
    }
    __device__ void store(S& st, int wave, int lane) const {
        const bool values = wave >= 2;
        const int u = wave & 1, part = D == 64 ? u : 0;
        if (!values) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // D = 64: words (chunk i / 2, k-step i % 2); else chunk u, k-step i
                    const int f = D == 64 ? i : (u * NB + b) * 4 + i;
                    st.k[part][f][lane] = make_uint4(kv4_pair<0>(w[b][i]), kv4_pair<1>(w[b][i]), kv4_pair<2>(w[b][i]), kv4_pair<3>(w[b][i]));
                }
        } else {
#pragma unroll
            for (int b = 0; b < NB; ++b)
                static_for<0, 4>([&](auto ic) {
                    constexpr int i = ic;
                    const int f = D == 64 ? i : b * S::CH + 4 * u + i;
                    st.v[part][f][lane] = make_uint4(kv4_pair<i>(w[b][0]), kv4_pair<i>(w[b][1]), kv4_pair<i>(w[b][2]), kv4_pair<i>(w[b][3]));
                });
        }
        const int g = lane / 16;
        const bool both = D == 64 || values;
        const int c = both ? g & 1 : u, b = both ? g >> 1 : g;
        if (b < NB && !(D != 64 && values && u)) (values ? st.vs : st.ks)[part][b][16 * c + lane % 16] = scale;
    }
};

template <int ACT, int D, int PART>
__global__ __launch_bounds__(256, D == 256 ? 2 : 4) void kv4_rows_kernel(Kv4AttentionArgs a, int64_t tiles, int span, int splits,
                                                                        uint32_t magic, unsigned* counters, float* partials) {
    using S = Stage<D>;
    constexpr int W = S::W, NB = S::NB, CH = S::CH, SUB = S::SUB, ROWS = 64, STEP = 32 * SUB;
    extern __shared__ uint4 lds_raw[];
    S* const stage = reinterpret_cast<S*>(lds_raw);
    __shared__ int last_one;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int col = lane % 16, kq = lane / 16;
    // consecutive workgroups take the key heads of one tile (each XCD then keeps to few heads), the
    // tiles from the last: under a causal mask those see most
    const int kh = int(blockIdx.x % unsigned(a.kv_heads)), share = a.heads / a.kv_heads;
    const int64_t x = tiles - 1 - int64_t(blockIdx.x / unsigned(a.kv_heads));

    Tile t;
    if (!find_tile<ROWS, PART>(a, x, t)) return;
    const View view{a.causal, int(a.window)};
    const int last = min(t.r0 + ROWS - 1, t.rows - 1);
    const int begin = view.lo(t.position(t.r0 / share)) / STEP * STEP, end = view.hi(t.position(last / share), t.kv);
    if constexpr (PART == kPrefix) span = part_span<PART>(end, splits);
    const int live = max(1, min(splits, (end - begin + span - 1) / span));
    if (int(blockIdx.y) >= live) return;
    const int s0 = begin + int(blockIdx.y) * span, s1 = min(end, s0 + span);
    const int steps = max(0, (s1 - s0 + STEP - 1) / STEP);

    // this wave's rows
    const int w0 = min(t.r0 + 16 * wave, last), w1 = min(w0 + 15, last);
    const bool idle = t.r0 + 16 * wave > last;
    const int all_lo = view.lo(t.position(w1 / share)), all_hi = min(view.hi(t.position(w0 / share), t.kv), s1);
    const int any_lo = view.lo(t.position(w0 / share)), any_hi = idle ? 0 : min(view.hi(t.position(w1 / share), t.kv), s1);

    const int64_t region = kv4_region(a.page, D);
    const uint8_t* pool = a.pool + kh * region;
    const int32_t* table = a.table + int64_t(t.b) * a.ldt;
    constexpr int PER = 64 / (2 * SUB);  // steps whose chunks the lanes hold
    Chunks ch;
    Quarter<D> raw;
    uint32_t there[3] = {0, 0, 0};  // chunks on pages of the pool, of this step, the next and the one after
    int loaded = 0;
    auto load = [&]() {
        const int at = loaded % PER;
        if (at == 0) ch.find(a, magic, table, region, NB * 8 * W, s0 / 16 + loaded * 2 * SUB, 2, s1, lane);
        raw.load(pool, ch, at * 2 * SUB, a.page, wave, lane);
        const uint32_t on = uint32_t(ch.there >> (at * 2 * SUB)) & ((1u << (2 * SUB)) - 1);
        ++loaded;
        return on;
    };
    if (steps > 0) there[1] = load();

    const int r = min(t.r0 + 16 * wave + col, last);
    const int qi = r / share, hd = kh * share + r % share;
    const int lo = view.lo(t.position(qi)), hi = min(view.hi(t.position(qi), t.kv), s1);
    uint4 q[NB][W / 32];
    float offset[NB];
    const float zf = load_queries<ACT, D>(a.q + (t.q0 + qi) * a.ldq + int64_t(hd) * D + 8 * kq, a.scale, q, offset);
    f32x4_t acc[NB][CH], ps[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        ps[b] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < CH; ++i) acc[b][i] = f32x4_t{0, 0, 0, 0};
    }
    Running run;

    if constexpr (PART == kOwn) {
        if (blockIdx.y == 0) take<D>(a, 0, prefix_splits(a, t.b), 1, t.q0 + qi, hd, kq, run, acc);
    }
    if (steps > 0) raw.store(stage[0], wave, lane);
    if (steps > 1) there[2] = load();
    for (int step = 0; step < steps; ++step) {
        lds_barrier();  // this step's operands are there, and nobody reads the other buffer any more
        there[0] = there[1];
        there[1] = there[2];
        if (step + 1 < steps) raw.store(stage[(step + 1) & 1], wave, lane);
        if (step + 2 < steps) there[2] = load();
        const S& st = stage[step & 1];
#pragma unroll
        for (int sub = 0; sub < SUB; ++sub) {
            const int tok = s0 + step * STEP + 32 * sub;
            if (tok + 32 <= any_lo || tok >= any_hi) continue;
            const uint32_t on = there[0] >> (2 * sub) & 3;
            float z[2][4];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    f32x4_t s = {offset[b], offset[b], offset[b], offset[b]};
#pragma unroll
                    for (int ks = 0; ks < W / 32; ++ks) s = mfma(st.k[sub][(c * NB + b) * (W / 32) + ks][lane], q[b][ks], s);
                    const float4 f = *reinterpret_cast<const float4*>(&st.ks[sub][b][16 * c + 4 * kq]);
                    const float y[4] = {s[0] * f.x, s[1] * f.y, s[2] * f.z, s[3] * f.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[c][i] = b == 0 ? y[i] : z[c][i] + y[i];
                }
            float vs[2][NB][4];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const float4 f = *reinterpret_cast<const float4*>(&st.vs[sub][b][16 * c + 4 * kq]);
                    vs[c][b][0] = f.x; vs[c][b][1] = f.y; vs[c][b][2] = f.z; vs[c][b][3] = f.w;
                }
            if (!(tok >= all_lo && tok + 32 <= all_hi && on == 3)) {
                // a value scale that was never written is not a number one can multiply by 0
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = tok + 16 * c + 4 * kq + i;
                        const bool seen = (on >> c & 1) && at >= lo && at < hi;
                        z[c][i] = seen ? z[c][i] : -INFINITY;
#pragma unroll
                        for (int b = 0; b < NB; ++b) vs[c][b][i] = seen ? vs[c][b][i] : 0.0f;
                    }
            }
            float p[2][4], w[2][NB][4];
            weigh<NB>(run, z, zf, vs, p, w, [&](float f) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    ps[b] *= f;
#pragma unroll
                    for (int i = 0; i < CH; ++i) acc[b][i] *= f;
                }
            });
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint4 pw = weights<NB>(w, b);
                ps[b] = mfma(make_uint4(kOnes, kOnes, kOnes, kOnes), pw, ps[b]);
#pragma unroll
                for (int i = 0; i < CH; ++i) acc[b][i] = mfma(st.v[sub][b * CH + i][lane], pw, acc[b][i]);
            }
        }
    }

    const int64_t tile = x * a.kv_heads + kh;
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    constexpr int kGroupBytes = int(partial_floats<D>() * 4), kSlot = kGroupBytes * (ROWS / 16), kRefs = 16 * D * 4;
    const __amdgpu_buffer_rsrc_t slots =
        buffer_rsrc(live > 1 ? partials + tile * splits * (kSlot / 4) : partials, live > 1 ? int64_t(splits) * kSlot : 0);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < CH; ++i) acc[b][i] -= kKvOffset * ps[b];
    float sum = row_sum(run.sum), ref = run.ref;
    if (PART != kPrefix && live > 1) {
        // as in the kernel above: the last split to finish joins them all
        const int mine = int(blockIdx.y) * kSlot + wave * kGroupBytes;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < CH; ++i)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[b][i]), slots,
                                                       mine + ((b * CH + i) * 64 + lane) * 16, 0, kCoherent);
        if (kq == 0) {
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(run.ref), slots, mine + kRefs + col * 4, 0, kCoherent);
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(sum), slots, mine + kRefs + 64 + col * 4, 0, kCoherent);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) {
            const unsigned before = __hip_atomic_fetch_add(counters + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last_one = before == unsigned(live - 1);
            if (last_one) __hip_atomic_store(counters + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (!last_one) return;
        ref = -INFINITY;
        sum = 0.0f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < CH; ++i) acc[b][i] = f32x4_t{0, 0, 0, 0};
        for (int sp = 0; sp < live; ++sp) {
            const int at = sp * kSlot + wave * kGroupBytes;
            const float other = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(slots, at + kRefs + col * 4, 0, kCoherent));
            const float more = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(slots, at + kRefs + 64 + col * 4, 0, kCoherent));
            f32x4_t part[NB][CH];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < CH; ++i)
                    part[b][i] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                                 slots, at + ((b * CH + i) * 64 + lane) * 16, 0, kCoherent));
            const float now = fmaxf(ref, other);
            const float f0 = ref == -INFINITY ? 0.0f : exp2_fast(ref - now);
            const float f1 = other == -INFINITY ? 0.0f : exp2_fast(other - now);
            ref = now;
            sum = sum * f0 + more * f1;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < CH; ++i) acc[b][i] = acc[b][i] * f0 + part[b][i] * f1;
        }
    }
    if (t.r0 + 16 * wave + col > last) return;
    if constexpr (PART == kPrefix) {
        leave<D>(Left(a, int(blockIdx.y), t.q0 + qi, hd), acc, ref, sum, kq);
        return;
    }
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    uint16_t* dst = a.out + (t.q0 + qi) * a.ldo + int64_t(hd) * D;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[CH / 2];
#pragma unroll
            for (int i = 0; i < CH / 2; ++i)
                w[i] = uint32_t(from_f32<ACT>(acc[b][2 * i][j] * inv)) | (uint32_t(from_f32<ACT>(acc[b][2 * i + 1][j] * inv)) << 16);
            uint16_t* to = dst + W * b + CH * (4 * kq + j);
            if constexpr (CH == 8) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        }
}

// Dynamic LDS beyond 64 KB has to be allowed for a kernel first.
hipError_t allow_lds(const void* kernel, size_t bytes) {
    return bytes <= 65536 ? hipSuccess : hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

template <int ACT, int D, int PART>
hipError_t run(const Kv4AttentionArgs& a, const Kv4Plan& p, float* partials, hipStream_t stream) {
    const int per = a.page / 16;
    const uint32_t magic = per == 1 ? 0 : uint32_t(((uint64_t(1) << 32) + per - 1) / per);
    unsigned* counters = static_cast<unsigned*>(a.workspace);
    if (p.splits < 2) partials = nullptr;
    if constexpr (PART != kBoth) {  // (tiles of 16 rows only)
        if (p.rows > 16) {
            const dim3 grid(unsigned(p.tiles * a.kv_heads), unsigned(p.splits));
            const size_t lds = 2 * sizeof(Stage<D>);
            const hipError_t e = allow_lds(reinterpret_cast<const void*>(&kv4_rows_kernel<ACT, D, PART>), lds);
            if (e != hipSuccess) return e;
            kv4_rows_kernel<ACT, D, PART><<<grid, dim3(256), lds, stream>>>(a, p.tiles, int(p.span), p.splits, magic, counters, partials);
            return hipGetLastError();
        }
    }
    const dim3 grid(unsigned(p.tiles), unsigned(a.kv_heads), unsigned(p.splits));
    kv4_attention_kernel<ACT, D, PART><<<grid, dim3(256), 0, stream>>>(a, int(p.span), p.splits, magic, counters, partials);
    return hipGetLastError();
}

template <int ACT, int PART>
hipError_t run_by_dim(const Kv4AttentionArgs& a, const Kv4Plan& p, float* partials, hipStream_t stream) {
    switch (a.dim) {
        case 64: return run<ACT, 64, PART>(a, p, partials, stream);
        case 128: return run<ACT, 128, PART>(a, p, partials, stream);
        default: return run<ACT, 256, PART>(a, p, partials, stream);
    }
}

template <int PART>
hipError_t run_by_type(const Kv4AttentionArgs& a, const Kv4Plan& p, float* partials, int act, hipStream_t stream) {
    return act == kActBf16 ? run_by_dim<kActBf16, PART>(a, p, partials, stream) : run_by_dim<kActF16, PART>(a, p, partials, stream);
}

float* after_header(void* workspace, size_t bytes) { return reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kSyncBytes + bytes); }

}  // namespace

Kv4Plan plan_kv4_attention(int64_t tokens, int64_t batch, int heads, int kv_heads, int dim, int64_t capacity, bool ragged,
                           bool causal, int64_t window) {
    Kv4Plan p{};
    const int64_t share = heads / kv_heads;
    p.rows = 16;
    // A window of the whole capacity hides nothing.  Left as given (any int64), it would overflow the sums below, and a
    // caller's workspace would be checked against another plan than the one launched.
    if (window >= capacity) window = 0;
    // the tokens a tile can see: its window, the queries of its rows, an aligned begin
    auto reach = [&](int rows) {
        const int64_t r = (causal ? window : 2 * window) + (ragged ? rows : 1) + 64;
        return window > 0 && r < capacity ? r : capacity;
    };
    // Tiles of 64 rows share the codes' conversion but have fewer workgroups to
    // spread over the chip: they lead where a request has 16 rows or more and the
    // call 4 M pairs of a row and a token.  us on tiles of 64 against 16, queries x
    // heads / key heads on tokens, with the pairs in M:
    //   D = 128  128 x 32/8 on 1024 (4.2) 17 against 20, 200 x 32/8 on 700 (4.5) 16
    //            against 21, 512 x 8/8 on 1024 (4.2) 16 against 20, 50 x 32/8 on 1024
    //            (1.6) 16 against 13; but 64 x 32/8 on 2048 (4.2) 21 against 19
    //   D = 64   256 x 16/16 on 1024 (4.2) 12.5 against 14.2, 50 x 16/16 on 1074 (0.9)
    //            12 against 10
    //   D = 256  512 x 8/1 on 1024 (4.2) 25 against 29, 768 x 8/1 on 1024 (6.3) 29
    //            against 34, 1024 x 8/1 on 1024 (8.4) 29 against 28, 512 x 8/1 on 512
    //            (2.1) 20 against 17; but 128 x 8/1 on 4096 (4.2) 42 against 25: few
    //            rows on long requests are better off on tiles of 16
    // (the grid of tiles of 64 is one line of tiles and key heads, which has to fit)
    if (ragged && tokens * share >= 16 * batch && tokens * heads * reach(64) >= int64_t(1) << 22 &&
        (tokens * share / 64 + batch) * kv_heads < int64_t(1) << 23)
        p.rows = 64;
    p.tiles = ragged ? tokens * share / p.rows + batch : batch * ceil_div(share, p.rows);
    const int64_t most = reach(p.rows);
    // Splits: with few tiles as many as fill the chip once (768 workgroups of D
    // = 128; 4 x 131072 tokens: 111 us, twice as many 119, four times 131), else
    // twice over, as lengths may differ (64 x 0..8192 tokens: 92 us, once 100,
    // four times 94).  Tiles of 64 rows count as three a CU though four of D = 64 and
    // 128 fit: four measured no better (200 queries x 32/8 heads of 128 on 30000
    // tokens 173 us, three 175; 4 x 128 on 4096 69 and 69; D = 64: 300 x 8/1 on
    // 30000 60 and 57).  A tile's splits share a counter of the workspace's header.
    const int64_t base = p.tiles * kv_heads;
    const int64_t room = 256 * (dim == 256 ? 2 : dim == 128 || p.rows > 16 ? 3 : 4);
    const int64_t want = base >= int64_t(kSyncBytes / 4) ? 1 : 4 * base <= room ? room / (base > 0 ? base : 1) : ceil_div(2 * room, base);
    int64_t span = ceil_div(ceil_div(most, want), 128) * 128;
    // Each part costs the join a read, each step of 128 tokens the walk a turn: at least sqrt(12 tokens), and 128, or 256
    // for tiles of many queries.  us with sqrt of 3, 12 and 48 tokens: D = 128, 32/8 heads, one request of 2000 9.6, 8.7,
    // 9.2, of 30000 26, 22, 22; D = 256, 8/1, of 4000 15, 13, 14, of 131072 54, 42, 48; D = 64, 16/16, of 30000 27, 24, 21.
    int64_t least = ragged ? 256 : 128;
    while (least * least < 12 * most) least += 128;
    if (span < least) span = least;
    p.span = span;
    p.splits = int(ceil_div(most, span));
    if (p.splits < 1) p.splits = 1;
    if (p.splits > 1) p.workspace = size_t(base) * size_t(p.splits) * size_t(p.rows / 16) * size_t(16 * dim + 32) * 4;
    return p;
}

hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, int act, hipStream_t stream) {
    const Kv4Plan p = plan_kv4_attention(a.tokens, a.batch, a.heads, a.kv_heads, a.dim, a.table_width * a.page,
                                         a.cu_q != nullptr, a.causal != 0, a.window);
    return run_by_type<kWhole>(a, p, after_header(a.workspace, 0), act, stream);
}

Kv4PrefixPlan plan_kv4_prefix(int64_t tokens, int64_t batch, int64_t groups, int heads, int kv_heads, int dim,
                              int64_t prefix_capacity, int64_t capacity, bool ragged, bool causal) {
    Kv4PrefixPlan p{};
    const int64_t share = heads / kv_heads;
    // Parts of `most` tokens that fill the chip once; fewer tokens are cut anew on the device (part_span).
    auto cut = [&](Kv4Plan& q, int64_t most, auto span_of) {
        const int64_t base = q.tiles * kv_heads, room = 256 * (dim == 256 ? 2 : dim == 64 || q.rows > 16 ? 4 : 3);
        q.span = span_of(int(most), int(base < room ? room / base : 1));
        q.splits = int(ceil_div(most, q.span));
    };
    // The prefixes.  Tiles of 64 rows share the codes' conversion, tiles of 16 have more workgroups and no barriers in
    // their steps.  us on tiles of 16 against 64, requests x heads / key heads on tokens, with the pairs of a row and a token
    // in M:  D = 128  64 x 32/8 on 8192 (17) 43 against 46, on 16384 (34) 66 against 61, 128 x 32/8 on 8192 (34) 72 against 68,
    // 3 x 8 of 20 queries x 32/8 on 2000 (31) 72 against 60, four groups of 48 x 32/8 on 20000 to 32768 (160) 248 against
    // 176, but 16 x 32/8 on 65536 (34) 68 against 75;  D = 256  256 x 8/1 on 4096 (8) 44 against 49;  D = 64  256 x 8/2
    // on 8192 (17) 29 and 29.  A part leaves its sums in memory for the other launch instead of joining them, but that
    // launch has to read them: parts of at least sqrt(48 tokens) (2 x 32/8 on 16384, D = 128: 23 us, sqrt(12 tokens) 24,
    // sqrt(tokens) 29, sqrt(100 tokens) 26); twice as many as fill the chip 49 us for 64 x 32/8 on 8192, 43 once.
    // A group's last tile is padded: tiles of 64 need 48 rows a group.  us on tiles of 16 against 64, groups x requests on
    // tokens, 32/8 heads of 128: 64 x 2 on 8192 (8 rows) 127 against 267, 64 x 8 on 2817 (32) 132 against 134, on 16384 502
    // against 549, 16 x 12 on 6645 with 32/4 (96) 101 against 75.  Over 700 such calls 64 takes on average 1.13 times as
    // long at 30 to 33 rows a group, 1.01 at 44 to 49, 0.93 at 60 to 65.
    // (the grid of tiles of 64 is one line of tiles and key heads, which has to fit)
    const bool tall = tokens * heads * prefix_capacity >= int64_t(24) << 20 && tokens * share >= 48 * groups &&
                      (tokens * share / 64 + groups) * kv_heads < int64_t(1) << 23;
    p.prefix.rows = tall ? 64 : 16;
    p.prefix.tiles = tokens * share / p.prefix.rows + groups;
    cut(p.prefix, prefix_capacity, part_span<kPrefix>);
    // The requests' own tokens, few as a rule: once over the chip where kv4_attention goes twice (64 x 32/8 on 4096, up to
    // 500 of their own: 35 us against 42; up to 4000: 71 and 71).
    p.own = plan_kv4_attention(tokens, batch, heads, kv_heads, dim, capacity, ragged, causal, 0);
    if (!ragged && p.own.splits > 1) {
        cut(p.own, capacity, part_span<kOwn>);
        p.own.workspace = p.own.splits > 1 ? size_t(p.own.tiles * kv_heads) * size_t(p.own.splits) * size_t(p.own.rows / 16) * size_t(16 * dim + 32) * 4 : 0;
    }
    // One launch for both where sharing saves little: every request's tiles (of 16 rows) then walk the prefix too.  What two
    // launches save are tile-tokens; what they cost, a launch and sums that pass through memory, grows with the rows, and a
    // tile that many heads share holds more of them: with 4 heads a key head and more the bound grows with them.  us together
    // against apart, with the saved tile-tokens in thousands, requests x heads / key heads on tokens, exact tables:
    //   D = 64   8 x 8/1 on 1000 (3) 8.5 and 11.6, 8 x 16/16 on 1000 (115) 10.8 and 11.8, on 4000 (452) 18.1 and 14.9, 32 x 32/8
    //            on 1000 (188) 12.9 and 13.4, 64 x 32/8 (385) 17.1 and 15.6, 20 x 16/2 on 12000 (217) 17.9 and 19.5
    //   D = 128  4 x 32/8 on 1000 (16) 11.2 and 14.2, 150 x 16/2 on 1000 (152) 18.3 and 20.4, 4 x 8/8 on 8000 (192) 18.5 and
    //            18.7, 32 x 8/8 on 1000 (238) 15.9 and 14.4, 64 x 32/8 on 1000 (385) 20.5 and 21.5, 64 x 8/1 on 16000 (496)
    //            29.3 and 31.1
    //   D = 256  2 x 8/1 on 800 (0) 11.3 and 18.8, 64 x 8/1 on 8000 (248) 30.9 and 37.1, 40 x 16/4 on 2500 (297) 28.4 and 28.1,
    //            64 x 4/4 on 2000 (483) 30.6 and 22.4
    // Over 17000 random calls the routes taken are 1.3 % behind the best of each; with 200000 for all of them 1.9 %.
    const int64_t tiles = ragged ? tokens * share / 16 + batch : batch * ceil_div(share, int64_t(16)), shared = tokens * share / 16 + groups;
    // (one request a group shares nothing: 64 x 1 on 16384, D = 128, 223 us together, 244 apart)
    const int64_t grown = (dim == 128 ? 100000 : 65000) * share;
    const int64_t little = share < 4 ? 200000 : grown < 500000 ? grown : 500000;
    if (!tall && (tiles - shared) * kv_heads * prefix_capacity <= little) {
        p.together = true;
        p.own = Kv4Plan{};
        p.own.rows = 16;
        p.own.tiles = tiles;
        cut(p.own, prefix_capacity + 32 + capacity, part_span<kBoth>);
        if (p.own.splits > 1) p.workspace = size_t(tiles * kv_heads) * size_t(p.own.splits) * size_t(16 * dim + 32) * 4;
        return p;
    }
    p.parts = size_t(p.prefix.splits) * size_t(tokens) * size_t(heads) * size_t(dim + 2) * 4;
    p.parts = (p.parts + 15) / 16 * 16;
    p.workspace = p.parts + p.own.workspace;
    return p;
}

hipError_t launch_kv4_prefix(const Kv4AttentionArgs& a, int act, hipStream_t stream) {
    Kv4AttentionArgs o = a;
    const Kv4PrefixPlan p = plan_kv4_prefix(o.tokens, o.batch, o.groups, o.heads, o.kv_heads, o.dim, o.prefix_width * o.page,
                                            o.table_width * o.page, o.cu_q != nullptr, o.causal != 0);
    if (p.together) return run_by_type<kBoth>(o, p.own, after_header(o.workspace, 0), act, stream);
    o.prefix_splits = p.prefix.splits;
    Kv4AttentionArgs f = o;
    f.table = a.prefix_table;
    f.table_width = a.prefix_width;
    f.ldt = a.ldp;
    f.kv_lens = a.prefix_lens;
    f.causal = 0;
    const hipError_t e = run_by_type<kPrefix>(f, p.prefix, nullptr, act, stream);
    return e == hipSuccess ? run_by_type<kOwn>(o, p.own, after_header(o.workspace, p.parts), act, stream) : e;
}

}  // namespace w4a16
