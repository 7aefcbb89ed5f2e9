// C entry points of the linear layer on 8-bit floats (include/w4a16.h): row and
// block quantization, the layer.  Argument checks from host metadata only, then
// launches.
#include "w4a16.h"

#include "checks.h"
#include "fp8.h"
#include "kernels.h"

using namespace w4a16;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 24;
constexpr int64_t kMaxK = int64_t(1) << 22;       // 256 rows of codes are addressed with 31 bits
constexpr int64_t kMaxGroups = int64_t(1) << 30;  // groups of a quantization, workgroups of a launch

size_t round16(size_t v) { return (v + 15) & ~size_t(15); }

int kernel_dtype(w4a16_dtype_t t) { return t == W4A16_BF16 ? kActBf16 : t == W4A16_F16 ? kActF16 : 0; }
size_t bytes_of(w4a16_dtype_t t) { return t == W4A16_F32 ? 4 : t == W4A16_E4M3 ? 1 : 2; }

// columns of x a row takes
int64_t width_of(w4a16_act_t act, int64_t k) { return act == W4A16_ACT_SWIGLU ? 2 * k : k; }

bool valid_act(w4a16_act_t act) { return act == W4A16_ACT_NONE || act == W4A16_ACT_SWIGLU || act == W4A16_ACT_GELU_TANH; }

bool valid_size(int64_t m, int64_t k) {
    return m >= 0 && m <= kMaxDim && k >= kGroup && k <= kMaxK && k % kGroup == 0 && m * (k / kGroup) <= kMaxGroups;
}

bool valid_linear(int64_t m, int64_t n, int64_t k) {
    if (!valid_size(m, k) || n < 0 || n > kMaxDim || ceil_div(n, int64_t(16)) * (k / kGroup) > kMaxGroups) return false;
    if (m == 0 || n == 0) return true;
    const Fp8Plan p = plan_fp8_linear(m, n, k);
    return p.mtiles * p.ntiles * p.splits <= kMaxGroups;
}

// codes and scales of x in the workspace, behind the header
size_t codes_bytes(int64_t m, int64_t k) { return round16(size_t(m) * size_t(k)); }
size_t scales_bytes(int64_t m, int64_t k) { return round16(size_t(m) * size_t(k / kGroup) * 4); }

w4a16_status_t quantize(const void* x, w4a16_dtype_t dtype, w4a16_act_t act, bool blocks, int64_t m, int64_t k, int64_t ldx, void* codes,
                        float* scales, void* stream) {
    if (!(blocks ? act_dtype(dtype) || dtype == W4A16_F32 : act_dtype(dtype))) return W4A16_EUNSUPPORTED;
    const size_t elem = bytes_of(dtype);
    const int64_t width = width_of(act, k);
    if (!valid_size(m, k) || ldx < width || ldx > kMaxDim || ldx * int64_t(elem) % 16 != 0) return W4A16_EINVAL;
    if (m == 0) return W4A16_OK;
    if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return W4A16_EINVAL;
    const size_t xb = span_bytes(m, width, ldx, elem), cb = size_t(m) * size_t(k),
                 sb = size_t(blocks ? ceil_div(m, int64_t(128)) : m) * size_t(k / kGroup) * 4;
    if (overlap(codes, cb, x, xb) || overlap(scales, sb, x, xb) || overlap(codes, cb, scales, sb)) return W4A16_EINVAL;
    const Fp8QuantizeArgs a{x, m, k, ldx, static_cast<uint8_t*>(codes), scales, false};
    hipStream_t s = static_cast<hipStream_t>(stream);
    return from_hip(blocks ? launch_fp8_quantize_blocks(a, kernel_dtype(dtype), s) : launch_fp8_quantize(a, kernel_dtype(dtype), int(act), s));
}

}  // namespace

extern "C" {

w4a16_status_t quantize_fp8_rows(const void* x, w4a16_dtype_t dtype, w4a16_act_t act, int64_t m, int64_t k, int64_t ldx, void* codes,
                                 float* scales, void* stream) {
    if (!valid_act(act)) return W4A16_EUNSUPPORTED;
    return quantize(x, dtype, act, false, m, k, ldx, codes, scales, stream);
}

w4a16_status_t quantize_fp8_blocks(const void* w, w4a16_dtype_t dtype, int64_t n, int64_t k, int64_t ldw, void* codes, float* scales,
                                   void* stream) {
    return quantize(w, dtype, W4A16_ACT_NONE, true, n, k, ldw, codes, scales, stream);
}

size_t fp8_linear_workspace_bytes(w4a16_dtype_t x_dtype, int64_t m, int64_t n, int64_t k) {
    if ((!act_dtype(x_dtype) && x_dtype != W4A16_E4M3) || !valid_linear(m, n, k) || m == 0 || n == 0) return 0;
    const Fp8Plan p = plan_fp8_linear(m, n, k);
    const size_t rows = x_dtype == W4A16_E4M3 || fp8_linear_quantizes(m, p) ? 0 : codes_bytes(m, k) + scales_bytes(m, k);
    return rows + p.workspace ? kSyncBytes + rows + p.workspace : 0;
}

int fp8_linear_tile(int64_t m, int64_t n, int64_t k, int* columns, int* splits) {
    const bool valid = valid_linear(m, n, k) && m > 0 && n > 0;
    const Fp8Plan p = valid ? plan_fp8_linear(m, n, k) : Fp8Plan{};
    if (columns) *columns = p.bn;
    if (splits) *splits = p.splits;
    return p.bm;
}

w4a16_status_t fp8_linear(const void* x, w4a16_dtype_t x_dtype, const float* x_scales, w4a16_act_t act, int64_t m, int64_t k, int64_t ldx,
                          const void* w, const float* w_scales, int64_t n, const void* bias, void* y, w4a16_dtype_t y_dtype, int64_t ldy,
                          void* workspace, size_t workspace_bytes, void* stream) {
    const bool codes = x_dtype == W4A16_E4M3;
    if ((!codes && !act_dtype(x_dtype)) || !act_dtype(y_dtype) || (!codes && x_dtype != y_dtype) || !valid_act(act) ||
        (codes && act != W4A16_ACT_NONE))
        return W4A16_EUNSUPPORTED;
    const int64_t width = width_of(act, k);
    const size_t elem = bytes_of(x_dtype);
    if (!valid_linear(m, n, k) || ldx < width || ldx > (codes ? kMaxK : kMaxDim) || ldx * int64_t(elem) % 16 != 0 || ldy < n || ldy > kMaxDim)
        return W4A16_EINVAL;
    if (m == 0 || n == 0) return W4A16_OK;  // (an empty tensor's scales have no address)
    if (!x || !w || !w_scales || !y || codes != (x_scales != nullptr)) return W4A16_EINVAL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(bias, 2) || !aligned(y, 2))
        return W4A16_EINVAL;
    const int64_t groups = k / kGroup;
    const size_t xb = span_bytes(m, width, ldx, elem), xsb = codes ? size_t(m) * size_t(groups) * 4 : 0, wb = size_t(n) * size_t(k),
                 wsb = size_t(ceil_div(n, int64_t(128))) * size_t(groups) * 4, bb = bias ? size_t(n) * 2 : 0, yb = span_bytes(m, n, ldy, 2);
    const size_t need = fp8_linear_workspace_bytes(x_dtype, m, n, k);
    if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_EWORKSPACE;
    if (need > 0 && !aligned(workspace, 16)) return W4A16_EINVAL;
    const struct { const void* p; size_t n; } in[] = {{x, xb}, {x_scales, xsb}, {w, wb}, {w_scales, wsb}, {bias, bb}};
    for (const auto& i : in)
        if (overlap(y, yb, i.p, i.n) || overlap(workspace, need, i.p, i.n)) return W4A16_EINVAL;
    if (overlap(workspace, need, y, yb)) return W4A16_EINVAL;

    hipStream_t s = static_cast<hipStream_t>(stream);
    uint8_t* at = static_cast<uint8_t*>(workspace) + (need ? kSyncBytes : 0);
    const Fp8Plan p = plan_fp8_linear(m, n, k);
    const bool inside = !codes && fp8_linear_quantizes(m, p);
    Fp8LinearArgs a{};
    if (codes || inside) {
        a.x = static_cast<const uint8_t*>(x);
        a.xs = x_scales;
        a.rs = groups;
        a.gs = 1;
        a.ldx = ldx;
    } else {
        // group by group: a step's scales are then one run of memory (4096 x 4096 x 16384: 222 us, row by row 242)
        a.rs = 1;
        a.gs = m;
        const Fp8QuantizeArgs q{x, m, k, ldx, at, reinterpret_cast<float*>(at + codes_bytes(m, k)), true};
        const hipError_t e = launch_fp8_quantize(q, kernel_dtype(x_dtype), int(act), s);
        if (e != hipSuccess) return W4A16_EHIP;
        a.x = q.codes;
        a.xs = q.scales;
        a.ldx = k;
        at += codes_bytes(m, k) + scales_bytes(m, k);
    }
    a.m = m;
    a.k = k;
    a.w = static_cast<const uint8_t*>(w);
    a.ws = w_scales;
    a.n = n;
    a.bias = static_cast<const uint16_t*>(bias);
    a.y = static_cast<uint16_t*>(y);
    a.ldy = ldy;
    a.counters = static_cast<unsigned*>(workspace);
    a.slots = reinterpret_cast<float*>(at);
    return from_hip(launch_fp8_linear(a, p, kernel_dtype(y_dtype), inside, int(act), s));
}

}  // extern "C"
