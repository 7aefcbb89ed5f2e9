// The 4-bit paged cache of keys and values: its layout and the launch plans
// of the kernels that write and read it (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "common.h"

namespace w4a16 {

// ---------------------------------------------------------------------------
// Layout.  The pool is [pages][kv_heads] regions; a region holds one page (P
// tokens, a multiple of 16) of one head of D channels, so a (page, head) is
// one contiguous run of memory.  W = min(D, 128) channels share a scale (the
// weights' group), NB = D / W blocks:
//
//   [0, PD/2)           key codes: chunks of 16 tokens x W channels, chunk
//                       (c, b) = tokens 16c.., block b at (c NB + b) 8W
//   [PD/2, PD)          value codes, chunks of the same size and order
//   [PD, PD + 4 P NB)   key scales FP32 [NB][P]
//   then 4 P NB bytes   value scales FP32 [NB][P]
//
// A chunk is read by a wave with one contiguous load: lane L owns its bytes
// [L W/8, (L+1) W/8), W/32 words, and each side's words are the operands of
// v_mfma_f32_16x16x32_f16 without any shuffle:
//   keys    S^T = K Q^T contracts channels: lane L is token L % 16, and word s
//           holds channels 32s + 8(L/16) + j with the weights' nibble order
//           (nibble i = 2i, nibble i + 4 = 2i + 1), one word per k-step.
//   values  O^T = V^T P^T contracts tokens: lane L is channel lane l = L % 16
//           and its token quarter kq = L / 16; word 2h + a holds tokens
//           4kq + 2a (low half) and 4kq + 2a + 1 (high half), nibble i of a
//           half = channel (W/16) l + 4h + i.  The tokens 4kq .. 4kq + 3 are
//           the rows of S^T that the same lane quarter computes, so the
//           probabilities are the other operand where they stand.
// A token owns whole bytes on both sides (words of keys, half-words of
// values), so appends of different tokens never touch the same byte.
//
// Codes are offset-binary nibbles u = q + 8, as in the packed weights.
// ---------------------------------------------------------------------------
constexpr int kKvChunkTokens = 16;

__host__ __device__ inline constexpr int kv4_width(int d) { return d < 128 ? d : 128; }
__host__ __device__ inline constexpr int kv4_blocks(int d) { return d / kv4_width(d); }
__host__ __device__ inline int64_t kv4_region(int64_t page, int d) { return page * d + 8 * page * kv4_blocks(d); }

// A nibble as a 16-bit float: bits 9:6 of the mantissa above exponent 4, so
// 0x4C00 | (u << 6) = 16 + u = 24 + q exactly (f16).  The small offset keeps
// the cancellation of sum(x (24 + q)) - 24 sum(x) at 24/2.5 of the values'
// size, an FP32 sum away from mattering.
constexpr uint32_t kKvMagic = 0x4C004C00u;
constexpr uint32_t kKvMask = 0x03C003C0u;
constexpr float kKvOffset = 24.0f;

// nibbles i and i + 4 of a word as an f16 pair 24 + q
template <int I>
__device__ inline uint32_t kv4_pair(uint32_t w) {
    constexpr int shift = 6 - 4 * I;
    uint32_t v;
    if constexpr (shift > 0) v = w << shift;
    else v = w >> -shift;
    return and_or(v, kKvMask, kKvMagic);
}

// The four f16 pairs 24 + q of each of two words (pair i: nibbles i and i + 4).
// The words go through 64-bit shifts together: half the shifts, and the bits that
// one word hands the other fall outside the mask.  The 16-row tiles use it (64
// ragged sequences 91 -> 85 us, 4 of 131072 tokens 109 -> 104); the 64-row tiles,
// which convert once for four waves, keep single words (a prompt of 4096 tokens
// 192 us, 196 with pairs of words).
template <int N>
__device__ inline uint64_t shl64(uint64_t v) {
    uint64_t d;
    asm("v_lshlrev_b64 %0, %1, %2" : "=v"(d) : "i"(N), "v"(v));
    return d;
}
__device__ inline void kv4_pairs(uint32_t a, uint32_t b, uint32_t (&pa)[4], uint32_t (&pb)[4]) {
    const uint64_t v = uint64_t(a) | (uint64_t(b) << 32);
    const uint64_t s[4] = {shl64<6>(v), shl64<2>(v), shr64<2>(v), shr64<6>(v)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        pa[i] = and_or(uint32_t(s[i]), kKvMask, kKvMagic);
        pb[i] = and_or(uint32_t(s[i] >> 32), kKvMask, kKvMagic);
    }
}

// ---------------------------------------------------------------------------
// Launch arguments
// ---------------------------------------------------------------------------
struct Kv4AppendArgs {
    const uint16_t* qkv;
    int64_t ldqkv;
    int64_t tokens;
    int heads, kv_heads, dim;
    uint8_t* pool;
    int64_t pages;
    int page;
    const int64_t* slots;
    const int32_t* positions;
    const float* rope;
    int64_t rope_len;
    int rot, interleaved;
    uint16_t* q_out;
};
hipError_t launch_kv4_append(const Kv4AppendArgs& a, int act, hipStream_t stream);

struct Kv4ReadArgs {
    const uint8_t* pool;
    int64_t pages;
    int page, kv_heads, dim;
    const int64_t* slots;
    int64_t tokens;
    void *k, *v;
};
hipError_t launch_kv4_read(const Kv4ReadArgs& a, int dtype, hipStream_t stream);

struct Kv4AttentionArgs {
    const uint16_t* q;
    int64_t ldq;  // elements between query tokens
    int64_t tokens;
    int heads, kv_heads, dim;
    const uint8_t* pool;
    int64_t pages;
    int page;
    const int32_t* table;
    int64_t table_width;  // pages a request's row can hold
    int64_t ldt;          // elements between rows
    const int32_t* kv_lens;
    const int32_t* cu_q;  // null: one query token a request
    int64_t batch;
    int causal;
    int64_t window;  // 0: none
    float scale;
    uint16_t* out;
    int64_t ldo;
    void* workspace;
};

struct Kv4Plan {
    int rows;          // rows (query token x shared head) of one tile
    int64_t tiles;     // row tiles per key head (at most: some may be empty)
    int64_t span;      // tokens of one split
    int splits;
    size_t workspace;  // after the header; 0 without splits
};
Kv4Plan plan_kv4_attention(int64_t tokens, int64_t batch, int heads, int kv_heads, int dim, int64_t capacity,
                           bool ragged, bool causal, int64_t window);
hipError_t launch_kv4_attention(const Kv4AttentionArgs& a, int act, hipStream_t stream);

}  // namespace w4a16
