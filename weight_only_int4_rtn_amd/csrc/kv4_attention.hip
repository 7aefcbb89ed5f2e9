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
// 34 binades below the row's largest).  Probabilities are p 2^-E vs with E
// the exponent of the largest value scale so far, folded into the running
// maximum, so they use f16's range whatever the values' size; their rounding
// (2^-11 of each) is an eighth of the bf16 output's.  The running maximum,
// the sum and the output accumulate in FP32.
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

// Tiles are numbered without a table: request b's start at
// floor(cu_q[b] share / ROWS) + b, which leaves room for the ragged last tile
// of every request (a few tiles stay empty).
template <int ROWS>
__device__ inline bool find_tile(const Kv4AttentionArgs& a, int64_t x, Tile& t) {
    const int share = a.heads / a.kv_heads;
    if (!a.cu_q) {
        const int per = (share + ROWS - 1) / ROWS;
        t.b = int(x / per);
        t.q0 = t.b;
        t.qn = 1;
        t.r0 = int(x % per) * ROWS;
    } else {
        int lo = 0, hi = int(a.batch) - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            const int64_t start = int64_t(a.cu_q[mid]) * share / ROWS + mid;
            if (start <= x) lo = mid;
            else hi = mid - 1;
        }
        t.b = lo;
        const int64_t c0 = a.cu_q[lo], c1 = a.cu_q[lo + 1];
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

// Chunks of 16 tokens -> their place in the pool.
struct Pages {
    const int32_t* row;
    int width, per;      // pages a row holds, chunks per page
    uint32_t magic;      // floor(c / per) = (c magic) >> 32 for c < 2^24, per <= 256
    int64_t pages;
    const uint8_t* pool; // of this key head
    int64_t stride;      // bytes between pages
    __device__ const uint8_t* region(int chunk, int end, int& in_page, bool& ok) const {
        const int p = per == 1 ? chunk : int(__umulhi(uint32_t(chunk), magic));
        in_page = chunk - p * per;
        int id = -1;
        if (chunk * 16 < end && p < width) id = row[p];
        ok = id >= 0 && id < pages;
        return pool + (ok ? int64_t(id) * stride : 0);
    }
};

// 32 tokens of one key head, as loaded.
template <int D>
struct Step {
    static constexpr int W = kv4_width(D), NB = kv4_blocks(D);
    uint32_t k[2][NB][W / 32], v[2][NB][W / 32];
    float4 ks[2][NB], vs[2][NB];
    bool ok[2];

    __device__ static void words(const uint8_t* p, uint32_t (&w)[W / 32]) {
        if constexpr (W == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x; w[1] = x.y;
        }
    }
    __device__ void load(const Pages& pg, int token, int end, int page, int lane) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            int in_page;
            const uint8_t* r = pg.region(token / 16 + c, end, in_page, ok[c]);
            const float* sc = reinterpret_cast<const float*>(r + page * D) + in_page * 16 + 4 * (lane / 16);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint8_t* p = r + (in_page * NB + b) * (8 * W) + lane * (W / 8);
                words(p, k[c][b]);
                words(p + page * (D / 2), v[c][b]);
                ks[c][b] = *reinterpret_cast<const float4*>(sc + b * page);
                vs[c][b] = *reinterpret_cast<const float4*>(sc + (NB + b) * page);
            }
        }
    }
};

// Workspace of a split: per (tile, key head, split) the accumulators in lane
// order, then the 16 rows' references and sums.
template <int D>
constexpr int64_t partial_floats() { return 16 * D + 32; }

// One workgroup: 16 rows of one key head over one split of the tokens.  Its
// four waves take steps of 32 tokens in turn, each with its own running
// maximum, and meet in LDS at the end.
template <int ACT, int D>
__global__ __launch_bounds__(256) void kv4_attention_kernel(Kv4AttentionArgs a, int span, int splits, uint32_t magic,
                                                            float* partials) {
    constexpr int W = kv4_width(D), NB = kv4_blocks(D), CH = W / 16;
    constexpr int WAVES = 4;
    __shared__ float lds[WAVES / 2][NB * CH * 4 + 2][64];
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
    const int col = lane % 16, kq = lane / 16;
    const int kh = blockIdx.y, share = a.heads / a.kv_heads;

    Tile t;
    if (!find_tile<16>(a, blockIdx.x, t)) return;
    const View view{a.causal, int(a.window)};
    const int last = min(t.r0 + 15, t.rows - 1);
    const int p_first = t.position(t.r0 / share), p_last = t.position(last / share);
    const int begin = view.lo(p_first) / 32 * 32, end = view.hi(p_last, t.kv);
    const int s0 = begin + int(blockIdx.z) * span, s1 = min(end, s0 + span);
    if (splits > 1 && s0 >= end) return;
    // every row of the tile sees [all_lo, all_hi)
    const int all_lo = view.lo(p_last), all_hi = view.hi(p_first, t.kv);

    // columns past the last row repeat it, and are dropped at the end
    const int r = min(t.r0 + col, last);
    const int qi = r / share, hd = kh * share + r % share;
    const int pos = t.position(qi);
    const int lo = view.lo(pos), hi = view.hi(pos, t.kv);

    // queries: f16, scaled by 2^(10 - e), and -24 sum(q) per block
    uint4 q[NB][W / 32];
    f32x4_t init[NB];
    float zf;
    {
        const uint16_t* src = a.q + (t.q0 + qi) * a.ldq + int64_t(hd) * D + 8 * kq;
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
        const int e = big > 0.0f && big < 3e38f ? 10 - (int(__float_as_uint(big) >> 23) - 127) : 0;
        zf = ldexpf(a.scale * kLog2e, -e);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float sum = 0.0f;
#pragma unroll
            for (int s = 0; s < W / 32; ++s) {
                const uint32_t w[4] = {raw[b][s].x, raw[b][s].y, raw[b][s].z, raw[b][s].w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = pack_f16(ldexpf(to_f32<ACT>(uint16_t(w[i])), e), ldexpf(to_f32<ACT>(uint16_t(w[i] >> 16)), e));
                q[b][s] = make_uint4(o[0], o[1], o[2], o[3]);
                sum += sum8<kActF16>(q[b][s]);
            }
            sum = -kKvOffset * row_sum(sum);
            init[b] = f32x4_t{sum, sum, sum, sum};
        }
    }

    Pages pg;
    pg.row = a.table + int64_t(t.b) * a.ldt;
    pg.width = int(a.table_width);
    pg.per = a.page / 16;
    pg.magic = magic;
    pg.pages = a.pages;
    pg.stride = a.kv_heads * kv4_region(a.page, D);
    pg.pool = a.pool + kh * kv4_region(a.page, D);

    f32x4_t acc[NB][CH], ps[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        ps[b] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < CH; ++i) acc[b][i] = f32x4_t{0, 0, 0, 0};
    }
    float top = -INFINITY;   // running maximum of the row's logits (base 2)
    int vexp = -60;          // exponent of the largest value scale so far (never below 2^-60)
    float ref = -INFINITY;   // top + vexp: what the probabilities are relative to
    float sum = 0.0f;        // this lane's part of the row's sum

    Step<D> cur, next;
    int tok = s0 + 32 * wave;
    if (tok < s1) cur.load(pg, tok, s1, a.page, lane);
    for (; tok < s1; tok += 32 * WAVES) {
        if (tok + 32 * WAVES < s1) next.load(pg, tok + 32 * WAVES, s1, a.page, lane);
        float z[2][4], vs[2][NB][4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[c][i] = 0.0f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                f32x4_t s = init[b];
#pragma unroll
                for (int ks = 0; ks < W / 32; ++ks) {
                    const uint32_t w = cur.k[c][b][ks];
                    s = mfma(make_uint4(kv4_pair<0>(w), kv4_pair<1>(w), kv4_pair<2>(w), kv4_pair<3>(w)), q[b][ks], s);
                }
                const float4 kf = cur.ks[c][b], vf = cur.vs[c][b];
                z[c][0] += s[0] * kf.x; z[c][1] += s[1] * kf.y; z[c][2] += s[2] * kf.z; z[c][3] += s[3] * kf.w;
                vs[c][b][0] = vf.x; vs[c][b][1] = vf.y; vs[c][b][2] = vf.z; vs[c][b][3] = vf.w;
            }
        }
        const bool whole = tok >= all_lo && tok + 32 <= all_hi && tok + 32 <= s1 && cur.ok[0] && cur.ok[1];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) z[c][i] *= zf;
        if (!whole) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = tok + 16 * c + 4 * kq + i;
                    const bool seen = cur.ok[c] && at >= lo && at < min(hi, s1);
                    z[c][i] = seen ? z[c][i] : -INFINITY;
#pragma unroll
                    for (int b = 0; b < NB; ++b) vs[c][b][i] = seen ? vs[c][b][i] : 0.0f;
                }
        }
        // new references where a logit or a value scale exceeds the old ones
        float zm = z[0][0], vm = vs[0][0][0];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                zm = fmaxf(zm, z[c][i]);
#pragma unroll
                for (int b = 0; b < NB; ++b) vm = fmaxf(vm, vs[c][b][i]);
            }
        if (__any(zm > top || vm > ldexpf(1.0f, vexp))) {
            top = fmaxf(top, row_max(zm));
            vm = row_max(vm);
            vexp = max(vexp, int(__float_as_uint(vm) >> 23) - 126);
            const float now = top + float(vexp);
            const float f = ref == -INFINITY ? 0.0f : exp2_fast(ref - now);
            ref = now;
            sum *= f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                ps[b] *= f;
#pragma unroll
                for (int i = 0; i < CH; ++i) acc[b][i] *= f;
            }
        }
        const float base = ref == -INFINITY ? 0.0f : ref;
        float p[2][4];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[c][i] = exp2_fast(z[c][i] - base);
                sum += p[c][i];
            }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint4 pw = make_uint4(pack_f16(p[0][0] * vs[0][b][0], p[0][1] * vs[0][b][1]),
                                        pack_f16(p[0][2] * vs[0][b][2], p[0][3] * vs[0][b][3]),
                                        pack_f16(p[1][0] * vs[1][b][0], p[1][1] * vs[1][b][1]),
                                        pack_f16(p[1][2] * vs[1][b][2], p[1][3] * vs[1][b][3]));
            ps[b] = mfma(make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u), pw, ps[b]);
            static_for<0, CH>([&](auto ic) {
                constexpr int i = ic, h = i / 4, ii = i % 4;
                acc[b][i] = mfma(make_uint4(kv4_pair<ii>(cur.v[0][b][2 * h]), kv4_pair<ii>(cur.v[0][b][2 * h + 1]),
                                            kv4_pair<ii>(cur.v[1][b][2 * h]), kv4_pair<ii>(cur.v[1][b][2 * h + 1])),
                                 pw, acc[b][i]);
            });
        }
        cur = next;
    }

    // take the offset out, then join the waves two and two
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < CH; ++i) acc[b][i] -= kKvOffset * ps[b];
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
    if (wave != 0) return;
    sum = row_sum(sum);
    if (splits > 1) {
        float* o = partials + ((int64_t(blockIdx.x) * a.kv_heads + kh) * splits + blockIdx.z) * partial_floats<D>();
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[((b * CH + i) * 4 + j) * 64 + lane] = acc[b][i][j];
        if (kq == 0) {
            o[16 * D + col] = ref;
            o[16 * D + 16 + col] = sum;
        }
        return;
    }
    if (t.r0 + col > last) return;
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

// Joins the splits of one tile and key head: wave j takes the accumulators'
// component j, which hold whole runs of CH channels of the output.
template <int ACT, int D>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4AttentionArgs a, int span, int splits, const float* partials) {
    constexpr int W = kv4_width(D), NB = kv4_blocks(D), CH = W / 16;
    const int lane = threadIdx.x % 64, j = threadIdx.x / 64;
    const int col = lane % 16, kq = lane / 16;
    const int kh = blockIdx.y, share = a.heads / a.kv_heads;
    Tile t;
    if (!find_tile<16>(a, blockIdx.x, t)) return;
    const View view{a.causal, int(a.window)};
    const int last = min(t.r0 + 15, t.rows - 1);
    const int begin = view.lo(t.position(t.r0 / share)) / 32 * 32, end = view.hi(t.position(last / share), t.kv);
    const int live = min(splits, max(0, (end - begin + span - 1) / span));
    const float* o = partials + (int64_t(blockIdx.x) * a.kv_heads + kh) * splits * partial_floats<D>();
    float ref = -INFINITY;
    for (int s = 0; s < live; ++s) ref = fmaxf(ref, o[s * partial_floats<D>() + 16 * D + col]);
    float sum = 0.0f, acc[NB][CH];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < CH; ++i) acc[b][i] = 0.0f;
    if (ref > -INFINITY) {
#pragma unroll 4
        for (int s = 0; s < live; ++s) {
            const float* p = o + s * partial_floats<D>();
            const float f = exp2_fast(p[16 * D + col] - ref);
            sum += p[16 * D + 16 + col] * f;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < CH; ++i) acc[b][i] += p[((b * CH + i) * 4 + j) * 64 + lane] * f;
        }
    }
    if (t.r0 + col > last) return;
    const int r = t.r0 + col;
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    uint16_t* dst = a.out + (t.q0 + r / share) * a.ldo + int64_t(kh * share + r % share) * D;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        uint32_t w[CH / 2];
#pragma unroll
        for (int i = 0; i < CH / 2; ++i)
            w[i] = uint32_t(from_f32<ACT>(acc[b][2 * i] * inv)) | (uint32_t(from_f32<ACT>(acc[b][2 * i + 1] * inv)) << 16);
        uint16_t* to = dst + W * b + CH * (4 * kq + j);
        if constexpr (CH == 8) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    }
}

template <int ACT, int D>
hipError_t run(const Kv4AttentionArgs& a, const Kv4Plan& p, hipStream_t stream) {
    const int per = a.page / 16;
    const uint32_t magic = per == 1 ? 0 : uint32_t(((uint64_t(1) << 32) + per - 1) / per);
    float* partials = p.splits > 1 ? reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kSyncBytes) : nullptr;
    const dim3 grid(unsigned(p.tiles), unsigned(a.kv_heads), unsigned(p.splits));
    kv4_attention_kernel<ACT, D><<<grid, dim3(256), 0, stream>>>(a, int(p.span), p.splits, magic, partials);
    if (p.splits > 1) {
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        kv4_join_kernel<ACT, D><<<dim3(unsigned(p.tiles), unsigned(a.kv_heads)), dim3(256), 0, stream>>>(a, int(p.span), p.splits, partials);
    }
    return hipGetLastError();
}

template <int ACT>
hipError_t run_by_dim(const Kv4AttentionArgs& a, const Kv4Plan& p, hipStream_t stream) {
    switch (a.dim) {
        case 64: return run<ACT, 64>(a, p, stream);
        case 128: return run<ACT, 128>(a, p, stream);
        default: return run<ACT, 256>(a, p, stream);
    }
}

}  // namespace

Kv4Plan plan_kv4_attention(int64_t tokens, int64_t batch, int heads, int kv_heads, int dim, int64_t capacity, bool ragged,
                           bool causal, int64_t window) {
    Kv4Plan p{};
    const int64_t share = heads / kv_heads;
    p.rows = 16;
    p.tiles = ragged ? tokens * share / p.rows + batch : batch * ceil_div(share, p.rows);
    // the tokens a tile can see: its window, the queries of its rows, an aligned begin
    int64_t most = capacity;
    if (window > 0) {
        const int64_t reach = (causal ? window : 2 * window) + (ragged ? p.rows : 1) + 32;
        most = most < reach ? most : reach;
    }
    const int64_t base = p.tiles * kv_heads;
    const int64_t want = ceil_div(2048, base > 0 ? base : 1);
    int64_t span = ceil_div(ceil_div(most, want), 128) * 128;
    if (span < 256) span = 256;
    p.span = span;
    p.splits = int(ceil_div(most, span));
    if (p.splits < 1) p.splits = 1;
    if (p.splits > 1) p.workspace = size_t(base) * size_t(p.splits) * size_t(16 * dim + 32) * 4;
    return p;
}

hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, int act, hipStream_t stream) {
    const Kv4Plan p = plan_kv4_attention(a.tokens, a.batch, a.heads, a.kv_heads, a.dim, a.table_width * a.page,
                                         a.cu_q != nullptr, a.causal != 0, a.window);
    return act == kActBf16 ? run_by_dim<kActBf16>(a, p, stream) : run_by_dim<kActF16>(a, p, stream);
}

}  // namespace w4a16
