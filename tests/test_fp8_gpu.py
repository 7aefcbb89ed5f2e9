"""The 8-bit float layer on the GPU: quantizers byte for byte, products against
64 bits with tolerances from the kernel's arithmetic (fp8_ref.linear)."""
import numpy as np
import pytest
import torch

import weight_only_int4_rtn_amd as w4

from . import fp8_ref as R
from .gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = {"none": w4.Act.NONE, "swiglu": w4.Act.SWIGLU, "gelu_tanh": w4.Act.GELU_TANH}


def rows(m, k, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, k, generator=g) * torch.exp(spread * torch.randn(k, generator=g))).to(dtype)


def bytes_of(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def same_bits(codes, scales, want):
    got = bytes_of(codes)
    assert np.array_equal(got, want[0].reshape(got.shape)), f"{int((got != want[0].reshape(got.shape)).sum())} codes differ"
    s = scales.cpu().numpy()
    assert np.array_equal(np.isnan(s), np.isnan(want[1].reshape(s.shape)))
    keep = ~np.isnan(s)
    assert np.array_equal(s.view(np.uint32)[keep], want[1].reshape(s.shape).view(np.uint32)[keep]), "scales differ"


def edge_rows(dtype):
    """Groups of zeros, of the type's largest and smallest numbers, ties between codes, one large among small."""
    fi = torch.finfo(dtype)
    x = torch.zeros(9, 256)
    x[1] = fi.max
    x[2, ::2], x[2, 1::2] = fi.tiny, -fi.tiny
    x[3, 0] = fi.tiny * fi.eps  # the smallest subnormal
    x[4, :128] = torch.arange(128) * 0.125 - 8  # 448 / 7 = 64: exact quotients, ties among them
    x[4, 0] = 7.0
    x[5, 5] = -448.0
    x[5, 6:30] = torch.arange(24) * 2.0 ** -10  # codes' subnormals and their ties
    x[6] = -0.0
    x[7, 0], x[7, 1:] = 1.0, 1e-4
    x[8] = torch.linspace(-3, 3, 256)
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,k", [(1, 128), (1, 2048), (3, 384), (65, 1152), (130, 128), (7, 16384)])
def test_rows(m, k, dtype):
    dev = require_gpu()
    x = rows(m, k, dtype, 7 * m + k)
    say("quantize_fp8", m, k, dtype)
    codes, scales = w4.quantize_fp8(x.to(dev))
    assert codes.dtype == torch.float8_e4m3fn and codes.shape == (m, k) and scales.shape == (m, k // 128)
    same_bits(codes, scales, R.quantize_rows(x.float().numpy()))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_edges(dtype):
    dev = require_gpu()
    x = edge_rows(dtype)
    codes, scales = w4.quantize_fp8(x.to(dev))
    same_bits(codes, scales, R.quantize_rows(x.float().numpy()))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_not_finite(dtype):
    dev = require_gpu()
    x = rows(5, 384, dtype, 3)
    x[0, 5], x[1, 200], x[2, 383], x[3, 0:128] = float("nan"), float("inf"), -float("inf"), float("nan")
    codes, scales = w4.quantize_fp8(x.to(dev))
    same_bits(codes, scales, R.quantize_rows(x.float().numpy()))
    assert torch.isnan(scales).sum() == 4 and torch.isnan(codes.float()).sum() == 4 * 128


def test_rows_views():
    """Strided rows, rows at odd addresses, broadcast and permuted ones, more dimensions, none at all."""
    dev = require_gpu()
    base = rows(40, 1024, BF16, 11).to(dev)
    views = [base[:, :256], base[::3, 128:640], base[:, 4:260], base[:, 1:129], base.view(4, 10, 1024)[:, :, 512:],
             base.view(4, 10, 1024)[1:3, 2:5], base[:1].expand(6, 1024), base[:, :128].t().contiguous().t(), base.view(8, 5, 1024).transpose(0, 1),
             base[0], base[5:5], base.view(4, 10, 1024)[:, :0]]
    for x in views:
        codes, scales = w4.quantize_fp8(x)
        assert codes.shape == x.shape and scales.shape == (*x.shape[:-1], x.shape[-1] // 128)
        if x.numel():
            same_bits(codes, scales, R.quantize_rows(x.float().cpu().reshape(-1, x.shape[-1]).numpy()))


@pytest.mark.parametrize("act", ["swiglu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_rows_activated(act, dtype):
    """The activated value is within one step of dtype of the formula's; so are code times scale, plus half a code step."""
    dev = require_gpu()
    k = 640
    x = rows(33, 2 * k if act == "swiglu" else k, dtype, 5, 0.3)
    codes, scales = w4.quantize_fp8(x.to(dev), act=ACTS[act])
    want = R.activate(x, act)
    got = torch.from_numpy(R.decode(bytes_of(codes))).view(33, k // 128, 128) * scales.cpu().double().unsqueeze(-1)
    top = want.view(33, k // 128, 128).abs().amax(-1, keepdim=True)
    # scale: off by the largest value's step; code: half a step (2^-4 of the value, 2^-10 of the scale below), the value's own step
    step = torch.finfo(dtype).eps
    limit = want.view(33, -1, 128).abs() * (2.0 ** -4 + 2 * step) + top / 448 * 2.0 ** -10 + top * 2 * step * 2.0 ** -4
    assert ((got - want.view(33, -1, 128)).abs() <= limit * 1.01).all()


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("n,k", [(1, 128), (128, 256), (130, 384), (1000, 1024), (2049, 128)])
def test_blocks(n, k, dtype):
    dev = require_gpu()
    w = rows(n, k, dtype, n + k, 0.5)
    w[n // 2] *= 3
    if n > 128:
        w[:128, :128] = 0
    codes, scales = w4.quantize_fp8_weight(w.to(dev))
    same_bits(codes, scales, R.quantize_blocks(w.float().numpy()))
    wide = torch.zeros(n, k + 12, dtype=dtype)
    wide[:, 4:k + 4] = w
    codes, scales = w4.quantize_fp8_weight(wide.to(dev)[:, 4:k + 4])
    same_bits(codes, scales, R.quantize_blocks(w.float().numpy()))


def test_blocks_edges():
    dev = require_gpu()
    w = torch.zeros(300, 256)
    w[:128, :128] = 1e-44  # a scale of one subnormal step: quotients beyond 448 are clamped
    w[5, 200], w[130, 3], w[299, 255] = float("nan"), float("inf"), 3e38
    codes, scales = w4.quantize_fp8_weight(w.to(dev))
    same_bits(codes, scales, R.quantize_blocks(w.numpy()))


def layer(n, k, seed, dev):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(n, k, generator=g) * torch.exp(0.5 * torch.randn(n, 1, generator=g)) * k ** -0.5
    cw, sw = R.quantize_blocks(w.numpy())
    return cw, sw, torch.from_numpy(cw).to(dev).view(torch.float8_e4m3fn), torch.from_numpy(sw).to(dev)


def check_linear(m, n, k, dtype, bias, dev, seed=0, workspace=None):
    cw, sw, codes, scales = layer(n, k, seed + n, dev)
    x = rows(m, k, dtype, seed + m, 0.7)
    b = rows(1, n, dtype, seed + 1, 0.0)[0] if bias else None
    say("linear_fp8", m, n, k, dtype, bias)
    y = w4.linear_fp8(x.to(dev), codes, scales, None if b is None else b.to(dev), workspace=workspace)
    assert y.shape == (m, n) and y.dtype == dtype
    cx, sx = R.quantize_rows(x.float().numpy())
    want, tol = R.linear(cx, sx, cw, sw, b)
    R.within(y, want, tol, f"{m} x {n} x {k} {dtype}")


# one row to several tiles of each kernel, ragged rows and columns, one group to many, split or not
SIZES = [(1, 1, 128), (1, 16, 128), (1, 100, 256), (1, 2560, 2048), (2, 33, 640), (5, 130, 4096), (16, 64, 2048), (16, 300, 1152),
         (17, 40, 128), (17, 300, 1024), (31, 129, 384), (32, 128, 2048), (33, 256, 896), (50, 1000, 1024), (64, 64, 8192), (100, 77, 256),
         (128, 130, 640), (200, 500, 1280), (257, 300, 384), (300, 260, 2048), (520, 513, 128), (600, 130, 256)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear(m, n, k, dtype):
    check_linear(m, n, k, dtype, (m + n) % 2 == 0, require_gpu())


@pytest.mark.parametrize("act", ["swiglu", "gelu_tanh"])
@pytest.mark.parametrize("m,n,k,dtype", [(1, 130, 256, BF16), (1, 300, 2048, F16), (3, 200, 640, BF16), (4, 64, 2048, F16), (9, 100, 384, BF16),
                                         (40, 300, 1024, F16), (150, 129, 256, BF16), (300, 512, 640, F16)])
def test_linear_activated(m, n, k, dtype, act):
    """A fused activation is `quantize_fp8` with it and the product of those codes: the same codes whoever quantizes."""
    dev = require_gpu()
    cw, sw, codes, scales = layer(n, k, n + m, dev)
    x = rows(m, 2 * k if act == "swiglu" else k, dtype, m + k, 0.4).to(dev)
    bias = rows(1, n, dtype, 3, 0.0)[0]
    say("linear_fp8", m, n, k, dtype, act)
    y = w4.linear_fp8(x, codes, scales, bias.to(dev), act=ACTS[act])
    cx, sx = w4.quantize_fp8(x, act=ACTS[act])
    want, tol = R.linear(bytes_of(cx).reshape(m, k), sx.cpu().numpy(), cw, sw, bias)
    R.within(y, want, tol, f"{act} {m} x {n} x {k}")


@pytest.mark.parametrize("m,n,k", [(1, 100, 256), (2, 64, 8192), (16, 300, 640), (20, 130, 384), (130, 300, 640), (300, 200, 2048)])
@pytest.mark.parametrize("dtype", [None, BF16, F16])
def test_linear_of_codes(m, n, k, dtype):
    """x that is quantized already, in rows of a wider tensor; the same bits as the layer that quantizes for itself."""
    dev = require_gpu()
    cw, sw, codes, scales = layer(n, k, n, dev)
    x = rows(m, k, dtype or BF16, m, 0.5)
    cx, sx = w4.quantize_fp8(x.to(dev))
    wide = torch.zeros(m, k + 48, dtype=torch.uint8, device=dev)
    wide[:, 16:k + 16] = cx.view(torch.uint8)
    say("linear_fp8 of codes", m, n, k, dtype)
    y = w4.linear_fp8(wide.view(torch.float8_e4m3fn)[:, 16:k + 16], codes, scales, x_scales=sx, out_dtype=dtype)
    assert y.dtype == (dtype or BF16)
    want, tol = R.linear(bytes_of(cx).reshape(m, k), sx.cpu().numpy(), cw, sw)
    R.within(y, want, tol, f"codes {m} x {n} x {k}")
    assert torch.equal(y, w4.linear_fp8(x.to(dev), codes, scales)), "quantized in the call: other bits"


def test_linear_exact_integers():
    """Small integers with scales of powers of two: every product and sum is exact in FP32, in every kernel and split, so the
    output is the exact result rounded once."""
    dev = require_gpu()
    g = torch.Generator().manual_seed(5)
    for m, n, k in SIZES + [(3, 2048, 16384), (64, 256, 16384), (40, 2100, 1024)]:
        cx = torch.randint(-4, 5, (m, k), generator=g).float()
        cw = torch.randint(-3, 4, (n, k), generator=g).float()
        sx = 2.0 ** torch.randint(-2, 3, (m, k // 128), generator=g)
        sw = 2.0 ** torch.randint(-2, 3, (-(-n // 128), k // 128), generator=g)
        # sparse: sums of some hundreds in steps of 2^-4
        cx *= torch.rand(m, k, generator=g) < 8 / k
        want = torch.zeros(m, n, dtype=torch.float64)
        for i in range(k // 128):
            c = slice(128 * i, 128 * i + 128)
            want += (cx[:, c].double() @ cw[:, c].double().t()) * sx[:, i:i + 1].double() * sw[:, i].double().repeat_interleave(128)[:n]
        say("exact", m, n, k)
        y = w4.linear_fp8(cx.to(dev).to(torch.float8_e4m3fn), cw.to(dev).to(torch.float8_e4m3fn), sw.to(dev), x_scales=sx.to(dev), out_dtype=F16)
        assert torch.equal(y.cpu(), want.to(F16)), (m, n, k)


def test_linear_views_and_shapes():
    """Rows at odd addresses, broadcast or permuted, more dimensions, none, rows of weights that end inside a block."""
    dev = require_gpu()
    n, k = 200, 256
    cw, sw, codes, scales = layer(n, k, 9, dev)
    base = rows(24, 1024, BF16, 17).to(dev)
    for x in (base[:, :k], base[::2, 128:384], base[:, 4:260], base[:, 1:257], base.view(4, 6, 1024)[:, :, 256:512], base[:1, :k].expand(20, k),
              base.view(4, 6, 1024).transpose(0, 1)[..., :k], base[3, :k]):
        y = w4.linear_fp8(x, codes, scales)
        assert y.shape == (*x.shape[:-1], n)
        flat = x.reshape(-1, k)
        assert torch.equal(y.reshape(-1, n), w4.linear_fp8(flat.contiguous(), codes, scales))
        want, tol = R.linear(*R.quantize_rows(flat.float().cpu().numpy()), cw, sw)
        R.within(y.reshape(-1, n), want, tol, str(tuple(x.shape)))
    assert w4.linear_fp8(base[:0, :k], codes, scales).shape == (0, n)
    assert w4.linear_fp8(base[:, :k], codes[:0], scales[:0]).shape == (24, 0)


@pytest.mark.parametrize("m", [1, 3, 16, 40, 140, 300])
def test_linear_not_finite(m):
    """A NaN or an infinity in x makes its row NaN, one in W's block the columns of that block; the others are as without."""
    dev = require_gpu()
    n, k = 300, 384
    w = torch.randn(n, k, generator=torch.Generator().manual_seed(2))
    x = rows(m, k, BF16, m)
    clean = w4.linear_fp8(x.to(dev), *w4.quantize_fp8_weight(w.to(dev)))
    bad = x.clone()
    bad[m // 2, 200] = float("inf")
    y = w4.linear_fp8(bad.to(dev), *w4.quantize_fp8_weight(w.to(dev)))
    keep = torch.arange(m) != m // 2
    assert torch.isnan(y[m // 2]).all() and torch.equal(y[keep.to(dev)], clean[keep.to(dev)])
    w[130, 5] = float("nan")
    y = w4.linear_fp8(x.to(dev), *w4.quantize_fp8_weight(w.to(dev)))
    assert torch.isnan(y[:, 128:256]).all()
    assert torch.equal(y[:, :128], clean[:, :128]) and torch.equal(y[:, 256:], clean[:, 256:])


@pytest.mark.parametrize("m,n,k", [(1, 2560, 2048), (1, 64, 16384), (12, 64, 16384), (64, 256, 16384), (40, 300, 2048), (300, 512, 1024)])
def test_linear_streams_graphs_and_repeats(m, n, k):
    """Two runs, another stream, two graphs on one workspace, replays between eager calls: the same bits; the header stays zero."""
    dev = require_gpu()
    _, _, codes, scales = layer(n, k, 1, dev)
    x = rows(m, k, BF16, m).to(dev)
    say("streams and graphs", m, n, k)
    want = w4.linear_fp8(x, codes, scales)
    assert torch.equal(want, w4.linear_fp8(x, codes, scales))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = w4.linear_fp8(x, codes, scales)
    side.synchronize()
    assert torch.equal(got, want)
    need = w4.linear_fp8_workspace_bytes(m, n, k)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    torch.cuda.synchronize()
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(w4.linear_fp8(x, codes, scales, workspace=ws))
    for rep in range(4):
        out = outs[rep % 2]
        out.fill_(float("nan"))
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {rep}"
        assert torch.equal(w4.linear_fp8(x, codes, scales), want)
    assert not ws[:1 << 20].any(), "the workspace's header is not zero"
    if need:
        with pytest.raises(ValueError, match="workspace"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                w4.linear_fp8(x, codes, scales)


def test_quantize_in_a_graph():
    dev = require_gpu()
    x = rows(300, 1024, F16, 3).to(dev)
    want = w4.quantize_fp8(x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = w4.quantize_fp8(x)
    for _ in range(3):
        got[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(got[1], want[1])


def test_linear_shares_a_workspace():
    """One workspace serves this layer, the INT4 layer and the cache's operators in turn."""
    dev = require_gpu()
    _, _, codes, scales = layer(2048, 16384, 1, dev)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    x = rows(64, 16384, BF16, 3).to(dev)
    packed = w4.pack(*w4.quantize(torch.randn(2048, 16384, device=dev) * 0.02))
    a, b = w4.linear_fp8(x, codes, scales), w4.linear(x, packed, 2048)
    for m in (64, 1, 12):
        assert torch.equal(w4.linear_fp8(x[:m], codes, scales, workspace=ws), w4.linear_fp8(x[:m], codes, scales))
        assert torch.equal(w4.linear(x, packed, 2048, workspace=ws), b)
    assert torch.equal(w4.linear_fp8(x, codes, scales, workspace=ws), a)


def test_linear_far_rows():
    """Codes and outputs beyond 4 GiB of their tensors."""
    dev = require_gpu()
    n, k, m = 20480, 262144, 24  # 5 GiB of codes
    codes = torch.zeros(n, k, dtype=torch.uint8, device=dev)
    g = torch.Generator().manual_seed(1)
    w = torch.randn(130, k, generator=g)
    cw, sw = R.quantize_blocks(w.numpy())
    codes[-130:] = torch.from_numpy(cw).to(dev)
    scales = torch.zeros(n // 128, k // 128, device=dev)
    # the last 130 rows lie in the last two blocks of 128
    full = np.zeros((256, k), np.uint8)
    full[-130:] = cw
    two = np.repeat(np.float32([[0.5], [0.25]]), k // 128, 1)
    scales[-2:] = torch.from_numpy(two).to(dev)
    x = rows(m, k, BF16, 2, 0.2)
    for count in (1, m):
        y = w4.linear_fp8(x[:count].to(dev), codes.view(torch.float8_e4m3fn), scales)
        assert not y[:, :-256].any()
        cx, sx = R.quantize_rows(x[:count].float().numpy())
        some = np.r_[120:130, 250:256]
        a = torch.from_numpy(R.decode(cx) * np.repeat(sx.astype(np.float64), 128, 1))
        b = torch.from_numpy(R.decode(full[some]) * np.repeat(two.astype(np.float64)[some // 128], 128, 1))
        want, size = a @ b.t(), a.abs() @ b.abs().t()
        # products cut 2^-13 below the largest of eight: at most 7 x 2^-13 of the eight's sum of sizes; 2048 groups in FP32
        R.within(y[:, -256:].cpu()[:, some], want, size * (7 * 2.0 ** -13 + 2.0 ** -23 * (2048 + 19)), "far rows")


# x quantized by the workgroups themselves, by a launch of its own before the kernel of few rows and before tiles; tiles of
# few rows on a large layer
@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("m,n,k", [(1, 2560, 2048), (1, 131080, 512), (3, 17000, 1024), (8, 300, 2048), (2, 40, 16384), (5, 25000, 4096), (16, 33000, 1024),
                                   (40, 300, 2048), (300, 513, 1024)])
def test_linear_equals_linear_of_codes(m, n, k, act):
    dev = require_gpu()
    g = torch.Generator(device=dev).manual_seed(n + k)
    codes = torch.randint(0, 256, (n, k), dtype=torch.uint8, device=dev, generator=g)
    codes[(codes & 127) == 127] = 0x7E
    codes = codes.view(torch.float8_e4m3fn)
    scales = torch.rand(-(-n // 128), k // 128, device=dev, generator=g) * 2.0 ** -10
    x = rows(m, 2 * k if act == "swiglu" else k, F16, 7, 0.5).to(dev)
    say("linear of codes", m, n, k, act)
    cx, sx = w4.quantize_fp8(x, act=ACTS[act])
    y = w4.linear_fp8(x, codes, scales, act=ACTS[act])
    z = w4.linear_fp8(cx, codes, scales, x_scales=sx, out_dtype=F16)
    assert torch.equal(y, z)
    for block in {0, n // 256, (n - 1) // 128}:
        at = slice(128 * block, min(n, 128 * block + 128))
        want, tol = R.linear(bytes_of(cx), sx.cpu().numpy(), bytes_of(codes[at]), scales[block:block + 1].cpu().numpy())
        R.within(y[:, at], want, tol, f"{m} x {n} x {k} block {block}")


def test_rows_far_apart():
    """Rows of a view further apart than a kernel's strides reach are copied first."""
    dev = require_gpu()
    base = torch.zeros(3, (1 << 24) + 8, dtype=BF16, device=dev)
    x = base[:, :256]
    x.copy_(rows(3, 256, BF16, 3))
    same_bits(*w4.quantize_fp8(x), R.quantize_rows(x.float().cpu().numpy()))
    cw, sw, codes, scales = layer(200, 256, 4, dev)
    assert torch.equal(w4.linear_fp8(x, codes, scales), w4.linear_fp8(x.contiguous(), codes, scales))
    cx, sx = w4.quantize_fp8(x)
    far = torch.zeros(3, (1 << 22) + 16, dtype=torch.uint8, device=dev)
    far[:, :256] = cx.view(torch.uint8)
    y = w4.linear_fp8(far.view(torch.float8_e4m3fn)[:, :256], codes, scales, x_scales=sx)
    assert torch.equal(y, w4.linear_fp8(cx, codes, scales, x_scales=sx))
