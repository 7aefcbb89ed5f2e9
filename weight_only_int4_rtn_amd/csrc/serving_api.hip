// C entry points of the serving operators (include/w4a16.h): the 4-bit paged
// cache, attention over it, and low-rank adapters.  Argument checks from host
// metadata only, then launches.
#include <cmath>

#include "w4a16.h"

#include "kernels.h"
#include "kv4.h"
#include "lora.h"

using namespace w4a16;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxPage = 4096;
constexpr int64_t kMaxTokens = int64_t(1) << 28;  // of one request in the cache
constexpr int64_t kMaxRows = int64_t(1) << 26;    // query tokens x heads of a call: a launch's work items fit 32 bits
constexpr int64_t kMaxBatch = int64_t(1) << 20;
constexpr int64_t kMaxCacheTokens = int64_t(1) << 23;         // appended or read by a call
constexpr uint64_t kMaxPoolBytes = uint64_t(1) << 38;         // scales are addressed in units of 64 bytes
constexpr int64_t kMaxLoraRank = 128;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
    if (!a || !b || an == 0 || bn == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + bn && b0 < a0 + an;
}

size_t span_bytes(int64_t rows, int64_t cols, int64_t ld, size_t elem) {
    if (rows <= 0 || cols <= 0) return 0;
    return (size_t(rows - 1) * size_t(ld) + size_t(cols)) * elem;
}

w4a16_status_t from_hip(hipError_t e) { return e == hipSuccess ? W4A16_OK : W4A16_EHIP; }

bool act_dtype(w4a16_dtype_t t) { return t == W4A16_BF16 || t == W4A16_F16; }
int act_of(w4a16_dtype_t t) { return t == W4A16_BF16 ? kActBf16 : kActF16; }

bool valid_pool(int64_t pages, int64_t page, int64_t kv_heads, int64_t dim) {
    return pages >= 1 && pages <= (int64_t(1) << 31) - 1 && page >= 16 && page <= kMaxPage && page % 16 == 0 &&
           kv_heads >= 1 && kv_heads <= kMaxHeads && (dim == 64 || dim == 128 || dim == 256) &&
           uint64_t(pages) * uint64_t(kv_heads) * uint64_t(kv4_region(page, int(dim))) <= kMaxPoolBytes;
}

}  // namespace

extern "C" {

size_t kv4_pool_bytes(int64_t pages, int64_t page_size, int64_t kv_heads, int64_t head_dim) {
    if (!valid_pool(pages, page_size, kv_heads, head_dim)) return 0;
    return size_t(pages) * size_t(kv_heads) * size_t(kv4_region(page_size, int(head_dim)));
}

w4a16_status_t kv4_append(const void* qkv, w4a16_dtype_t dtype, int64_t tokens, int64_t ldqkv, int64_t heads,
                          int64_t kv_heads, int64_t head_dim, const float* rope, int64_t rope_len, int64_t rot_dim,
                          int interleaved, const int32_t* positions, const int64_t* slots, void* pool, int64_t pages,
                          int64_t page_size, void* q_out, void* stream) {
    if (!act_dtype(dtype)) return W4A16_EUNSUPPORTED;
    if (!valid_pool(pages, page_size, kv_heads, head_dim) || heads < 0 || heads > kMaxHeads) return W4A16_EINVAL;
    const int64_t width = (heads + 2 * kv_heads) * head_dim;
    if (tokens < 0 || tokens > kMaxCacheTokens || ldqkv < width || ldqkv > kMaxDim || ldqkv % 8 != 0) return W4A16_EINVAL;
    if ((rope == nullptr) != (positions == nullptr)) return W4A16_EINVAL;
    if (rope && (rope_len < 1 || rope_len > kMaxTokens || rot_dim < 16 || rot_dim > head_dim || rot_dim % 16 != 0 ||
                 !aligned(rope, 16) || !aligned(positions, 4)))
        return W4A16_EINVAL;
    if (tokens == 0) return W4A16_OK;
    if (!qkv || !slots || !pool || (heads > 0 && !q_out)) return W4A16_EINVAL;
    if (!aligned(qkv, 16) || !aligned(slots, 8) || !aligned(pool, 16) || !aligned(q_out, 16)) return W4A16_EINVAL;
    const size_t in = span_bytes(tokens, width, ldqkv, 2), pb = kv4_pool_bytes(pages, page_size, kv_heads, head_dim),
                 qb = size_t(tokens) * size_t(heads) * size_t(head_dim) * 2,
                 rb = rope ? size_t(rope_len) * size_t(rot_dim) * 4 : 0, sb = size_t(tokens) * 8,
                 ob = rope ? size_t(tokens) * 4 : 0;
    if (overlap(pool, pb, qkv, in) || overlap(pool, pb, rope, rb) || overlap(pool, pb, slots, sb) ||
        overlap(pool, pb, positions, ob) || overlap(q_out, qb, qkv, in) || overlap(q_out, qb, pool, pb) ||
        overlap(q_out, qb, rope, rb) || overlap(q_out, qb, slots, sb) || overlap(q_out, qb, positions, ob))
        return W4A16_EINVAL;
    Kv4AppendArgs a{};
    a.qkv = static_cast<const uint16_t*>(qkv);
    a.ldqkv = ldqkv;
    a.tokens = tokens;
    a.heads = int(heads);
    a.kv_heads = int(kv_heads);
    a.dim = int(head_dim);
    a.pool = static_cast<uint8_t*>(pool);
    a.pages = pages;
    a.page = int(page_size);
    a.slots = slots;
    a.positions = positions;
    a.rope = rope;
    a.rope_len = rope_len;
    a.rot = rope ? int(rot_dim) : 0;
    a.interleaved = interleaved != 0;
    a.q_out = static_cast<uint16_t*>(q_out);
    return from_hip(launch_kv4_append(a, act_of(dtype), static_cast<hipStream_t>(stream)));
}

w4a16_status_t kv4_read(const void* pool, int64_t pages, int64_t page_size, int64_t kv_heads, int64_t head_dim,
                        const int64_t* slots, int64_t tokens, w4a16_dtype_t out_dtype, void* k, void* v, void* stream) {
    if (out_dtype != W4A16_F32 && !act_dtype(out_dtype)) return W4A16_EUNSUPPORTED;
    if (!valid_pool(pages, page_size, kv_heads, head_dim) || tokens < 0 || tokens > kMaxCacheTokens) return W4A16_EINVAL;
    if (tokens == 0) return W4A16_OK;
    if (!pool || !slots || !k || !v || !aligned(pool, 16) || !aligned(slots, 8) || !aligned(k, 16) || !aligned(v, 16))
        return W4A16_EINVAL;
    const size_t pb = kv4_pool_bytes(pages, page_size, kv_heads, head_dim), sb = size_t(tokens) * 8,
                 ob = size_t(tokens) * size_t(kv_heads) * size_t(head_dim) * (out_dtype == W4A16_F32 ? 4 : 2);
    if (overlap(k, ob, v, ob) || overlap(k, ob, pool, pb) || overlap(v, ob, pool, pb) || overlap(k, ob, slots, sb) ||
        overlap(v, ob, slots, sb))
        return W4A16_EINVAL;
    Kv4ReadArgs a{};
    a.pool = static_cast<const uint8_t*>(pool);
    a.pages = pages;
    a.page = int(page_size);
    a.kv_heads = int(kv_heads);
    a.dim = int(head_dim);
    a.slots = slots;
    a.tokens = tokens;
    a.k = k;
    a.v = v;
    return from_hip(launch_kv4_read(a, int(out_dtype), static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

bool valid_attention(int64_t tokens, int64_t batch, int64_t heads, int64_t kv_heads, int64_t head_dim,
                     int64_t table_width, int64_t page_size, bool ragged, int64_t window) {
    if (!valid_pool(1, page_size, kv_heads, head_dim)) return false;
    if (heads < 1 || heads > kMaxHeads || heads % kv_heads != 0) return false;
    if (tokens < 0 || tokens > kMaxDim || batch < 0 || batch > kMaxBatch || tokens * heads > kMaxRows) return false;
    if (!ragged && tokens != batch) return false;
    if (tokens > 0 && batch == 0) return false;
    if (table_width < 1 || table_width * page_size >= kMaxTokens) return false;
    return window >= 0;
}

}  // namespace

extern "C" {

size_t kv4_attention_workspace_bytes(int64_t tokens, int64_t batch, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                     int64_t table_width, int64_t page_size, int ragged, int causal, int64_t window) {
    if (!valid_attention(tokens, batch, heads, kv_heads, head_dim, table_width, page_size, ragged != 0, window) || tokens == 0)
        return 0;
    const size_t w = plan_kv4_attention(tokens, batch, int(heads), int(kv_heads), int(head_dim), table_width * page_size,
                                        ragged != 0, causal != 0, window).workspace;
    return w ? kSyncBytes + w : 0;
}

int kv4_attention_tile_rows(int64_t tokens, int64_t batch, int64_t heads, int64_t kv_heads, int64_t head_dim,
                            int64_t table_width, int64_t page_size, int ragged, int causal, int64_t window) {
    if (!valid_attention(tokens, batch, heads, kv_heads, head_dim, table_width, page_size, ragged != 0, window) || tokens == 0)
        return 0;
    return plan_kv4_attention(tokens, batch, int(heads), int(kv_heads), int(head_dim), table_width * page_size, ragged != 0,
                              causal != 0, window).rows;
}

w4a16_status_t kv4_attention(const void* q, w4a16_dtype_t dtype, int64_t tokens, int64_t ldq, int64_t heads,
                             int64_t kv_heads, int64_t head_dim, const void* pool, int64_t pages, int64_t page_size,
                             const int32_t* table, int64_t table_width, int64_t ldt, const int32_t* kv_lens,
                             const int32_t* cu_q, int64_t batch, int causal, int64_t window, float scale, void* out,
                             int64_t ldo, void* workspace, size_t workspace_bytes, void* stream) {
    if (!act_dtype(dtype)) return W4A16_EUNSUPPORTED;
    if (!valid_attention(tokens, batch, heads, kv_heads, head_dim, table_width, page_size, cu_q != nullptr, window) ||
        !valid_pool(pages, page_size, kv_heads, head_dim))
        return W4A16_EINVAL;
    const int64_t width = heads * head_dim;
    if (ldq < width || ldq > kMaxDim || ldq % 8 != 0 || ldo < width || ldo > kMaxDim || ldo % 8 != 0 ||
        ldt < table_width || ldt > kMaxTokens || !std::isfinite(scale))
        return W4A16_EINVAL;
    if (tokens == 0) return W4A16_OK;
    if (!q || !pool || !table || !kv_lens || !out) return W4A16_EINVAL;
    if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(kv_lens, 4) ||
        !aligned(cu_q, 4))
        return W4A16_EINVAL;
    const size_t qb = span_bytes(tokens, width, ldq, 2), ob = span_bytes(tokens, width, ldo, 2),
                 pb = kv4_pool_bytes(pages, page_size, kv_heads, head_dim), tb = span_bytes(batch, table_width, ldt, 4),
                 lb = size_t(batch) * 4, cb = cu_q ? size_t(batch + 1) * 4 : 0;
    const size_t need = kv4_attention_workspace_bytes(tokens, batch, heads, kv_heads, head_dim, table_width, page_size,
                                                      cu_q != nullptr, causal, window);
    if (overlap(out, ob, q, qb) || overlap(out, ob, pool, pb) || overlap(out, ob, table, tb) || overlap(out, ob, kv_lens, lb) ||
        overlap(out, ob, cu_q, cb) || overlap(out, ob, workspace, need))
        return W4A16_EINVAL;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return W4A16_EWORKSPACE;
        if (!aligned(workspace, 16)) return W4A16_EINVAL;
        if (overlap(workspace, need, q, qb) || overlap(workspace, need, pool, pb) || overlap(workspace, need, table, tb) ||
            overlap(workspace, need, kv_lens, lb) || overlap(workspace, need, cu_q, cb))
            return W4A16_EINVAL;
    }
    Kv4AttentionArgs a{};
    a.q = static_cast<const uint16_t*>(q);
    a.ldq = ldq;
    a.tokens = tokens;
    a.heads = int(heads);
    a.kv_heads = int(kv_heads);
    a.dim = int(head_dim);
    a.pool = static_cast<const uint8_t*>(pool);
    a.pages = pages;
    a.page = int(page_size);
    a.table = table;
    a.table_width = table_width;
    a.ldt = ldt;
    a.kv_lens = kv_lens;
    a.cu_q = cu_q;
    a.batch = batch;
    a.causal = causal != 0;
    a.window = window < kMaxTokens ? window : kMaxTokens;
    a.scale = scale;
    a.out = static_cast<uint16_t*>(out);
    a.ldo = ldo;
    a.workspace = workspace;
    return from_hip(launch_kv4_attention(a, act_of(dtype), static_cast<hipStream_t>(stream)));
}

size_t lora_add_workspace_bytes(int64_t m, int64_t n, int64_t k, int64_t adapters, int64_t rank) {
    if (m <= 0 || m > kMaxDim || n <= 0 || n > kMaxDim || k <= 0 || k > kMaxDim || k % 8 != 0 || adapters <= 0 ||
        adapters > kMaxDim || rank <= 0 || rank > kMaxLoraRank || rank % 8 != 0)
        return 0;
    const size_t w = plan_lora(m, n, k, int(adapters), int(rank)).workspace;
    return w ? kSyncBytes + w : 0;
}

w4a16_status_t lora_add(const void* x, w4a16_dtype_t dtype, int64_t m, int64_t k, int64_t ldx, const void* a,
                        const void* b, int64_t adapters, int64_t rank, int64_t n, const int32_t* index,
                        const float* scales, const void* y, int64_t ldy, void* out, int64_t ldo, void* workspace,
                        size_t workspace_bytes, void* stream) {
    if (!act_dtype(dtype)) return W4A16_EUNSUPPORTED;
    if (m < 0 || m > kMaxDim || n < 0 || n > kMaxDim || k <= 0 || k > kMaxDim || k % 8 != 0 || adapters < 1 ||
        adapters > kMaxDim || rank < 8 || rank > kMaxLoraRank || rank % 8 != 0)
        return W4A16_EINVAL;
    if (ldx < k || ldx > kMaxDim || ldx % 8 != 0 || ldy < n || ldy > kMaxDim || ldo < n || ldo > kMaxDim) return W4A16_EINVAL;
    if (m == 0 || n == 0) return W4A16_OK;
    if (!x || !a || !b || !index || !y || !out) return W4A16_EINVAL;
    if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(index, 4) || !aligned(scales, 4) ||
        !aligned(y, 2) || !aligned(out, 2))
        return W4A16_EINVAL;
    const size_t xb = span_bytes(m, k, ldx, 2), yb = span_bytes(m, n, ldy, 2), ob = span_bytes(m, n, ldo, 2),
                 ab = size_t(adapters) * size_t(rank) * size_t(k) * 2, bb = size_t(adapters) * size_t(rank) * size_t(n) * 2,
                 ib = size_t(m) * 4, sb = scales ? size_t(adapters) * 4 : 0;
    const bool in_place = out == y && ldo == ldy;
    if ((!in_place && overlap(out, ob, y, yb)) || overlap(out, ob, x, xb) || overlap(out, ob, a, ab) || overlap(out, ob, b, bb) ||
        overlap(out, ob, index, ib) || overlap(out, ob, scales, sb))
        return W4A16_EINVAL;
    const size_t need = lora_add_workspace_bytes(m, n, k, adapters, rank);
    if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_EWORKSPACE;
    if (need > 0 && !aligned(workspace, 16)) return W4A16_EINVAL;
    if (overlap(workspace, need, x, xb) || overlap(workspace, need, y, yb) ||
        overlap(workspace, need, out, ob) || overlap(workspace, need, a, ab) || overlap(workspace, need, b, bb) ||
        overlap(workspace, need, index, ib) || overlap(workspace, need, scales, sb))
        return W4A16_EINVAL;
    LoraArgs p{};
    p.x = static_cast<const uint16_t*>(x);
    p.ldx = ldx;
    p.m = m;
    p.n = n;
    p.k = k;
    p.a = static_cast<const uint16_t*>(a);
    p.b = static_cast<const uint16_t*>(b);
    p.adapters = int(adapters);
    p.rank = int(rank);
    p.index = index;
    p.scales = scales;
    p.y = static_cast<const uint16_t*>(y);
    p.ldy = ldy;
    p.out = static_cast<uint16_t*>(out);
    p.ldo = ldo;
    p.workspace = workspace;
    return from_hip(launch_lora(p, act_of(dtype), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
