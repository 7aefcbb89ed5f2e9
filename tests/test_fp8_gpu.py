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
