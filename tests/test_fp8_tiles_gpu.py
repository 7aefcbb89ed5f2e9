"""Every kernel of the 8-bit float layer (test_fp8_tiles_host lists sizes that reach them): exact integers bit for bit, normal
values against 64 bits, and the quantizer's kernel of many groups against the one of few."""
import numpy as np
import pytest
import torch

import weight_only_int4_rtn_amd as w4

from . import fp8_ref as R
from .gpu_util import require_gpu, say
from .test_fp8_gpu import ACTS, bytes_of, same_bits
from .test_fp8_tiles_host import SIZES

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def name(size):
    return "x".join(map(str, size))


@pytest.mark.parametrize("m,n,k", SIZES, ids=[name(s) for s in SIZES])
def test_exact_integers(dev, m, n, k):
    """Integers of up to 4 and 3 with scales of powers of two, eight values or so a row of x: every product and every sum is a
    multiple of 2^-4 below 2^15, exact in FP32 in any order, so each output is the exact result rounded once."""
    g = torch.Generator(device=dev).manual_seed(m + n + k)
    groups, blocks = k // 128, -(-n // 128)
    draw = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device=dev).float()  # noqa: E731
    x, w = draw(-4, 5, m, k), draw(-3, 4, n, k)
    x *= torch.rand(m, k, generator=g, device=dev) < 8 / k
    x[::5, -128:] = draw(-4, 5, 128)  # the last group in full, in every fifth row
    xs, ws = 2.0 ** draw(-2, 3, m, groups), 2.0 ** draw(-2, 3, blocks, groups)
    say("exact integers", m, n, k, w4.linear_fp8_tile(m, n, k))
    wide = torch.full((m, k + 16), 0x7F, dtype=torch.uint8, device=dev)  # rows further apart than they are long, NaN between
    wide[:, :k] = x.to(E4M3).view(torch.uint8)
    y = w4.linear_fp8(wide.view(E4M3)[:, :k], w.to(E4M3), ws, x_scales=xs, out_dtype=F16)
    want = (x * xs.repeat_interleave(128, 1)).double() @ (w * ws.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)).double().t()
    assert float(want.abs().max()) < 2 ** 15
    bad = (y != want.to(F16)).nonzero()
    assert not len(bad), f"{len(bad)} outputs differ, the first at {bad[0].tolist()}: {y[tuple(bad[0])]} for {want[tuple(bad[0])]}"


@pytest.mark.parametrize("m,n,k", SIZES, ids=[name(s) for s in SIZES])
def test_values(dev, m, n, k):
    """Normal values, quantized in the call, biased, in rows of y of odd length; some rows and columns against 64 bits.

    Within a group eight neighbouring products at a time are cut 2^-13 below the largest of them, at most 7 x 2^-13 of the
    sum of their sizes; k / 128 groups and 19 more additions and products in FP32 (fp8_ref.linear)."""
    g = torch.Generator(device=dev).manual_seed(m + 3 * n + k)
    x = (torch.randn(m, k, generator=g, device=dev) * torch.exp(0.5 * torch.randn(k, generator=g, device=dev))).to(BF16)
    codes, scales = w4.quantize_fp8_weight(torch.randn(n, k, generator=g, device=dev) * k ** -0.5)
    bias = torch.randn(n, generator=g, device=dev).to(BF16)
    say("values", m, n, k, w4.linear_fp8_tile(m, n, k))
    y = w4.linear_fp8(x, codes, scales, bias)
    cx, sx = w4.quantize_fp8(x)
    assert torch.equal(y, w4.linear_fp8(cx, codes, scales, bias, x_scales=sx))
    pick = lambda size: sorted({i for i in (0, 1, 15, 16, 63, 64, 127, 128, 255, 256, size // 2, size - 17, size - 2, size - 1) if 0 <= i < size})  # noqa: E731
    r, c = pick(m), pick(n)
    a = torch.from_numpy(R.decode(bytes_of(cx[r])) * np.repeat(sx[r].cpu().numpy().astype(np.float64), 128, 1))
    b = torch.from_numpy(R.decode(bytes_of(codes[c])) * np.repeat(scales.cpu().numpy().astype(np.float64)[np.array(c) // 128], 128, 1))
    add = bias.cpu().double()[c]
    want, size = a @ b.t() + add, a.abs() @ b.abs().t()
    tol = size * (7 * 2.0 ** -13 + 2.0 ** -23 * (k // 128 + 19)) + 2.0 ** -23 * (want.abs() + add.abs())
    R.within(y.cpu()[r][:, c], want, tol, name((m, n, k)))


# groups from 600000 on go through a kernel of their own; counts that are no multiple of what a workgroup takes
MANY = [(4799, 16000), (4801, 16000), (4807, 16000), (38, 2080768), (600011, 128)]


@pytest.mark.parametrize("act", ["none", "swiglu", "gelu_tanh"])
@pytest.mark.parametrize("m,k", MANY)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_many_groups(dev, m, k, act, dtype):
    """The whole at once and rows in pieces of few groups: the same bits; the first and last rows as the formula has them."""
    g = torch.Generator(device=dev).manual_seed(m + k)
    width = 2 * k if act == "swiglu" else k
    x = torch.empty(m, width, dtype=dtype, device=dev)
    for i in range(0, m, 4096):
        x[i:i + 4096] = torch.randn(min(4096, m - i), width, generator=g, device=dev)
    x[m // 2, 5], x[m // 3, -1] = float("nan"), float("inf")
    say("many groups", m, k, act, dtype)
    codes, scales = w4.quantize_fp8(x, act=ACTS[act])
    step = 300000 // (k // 128)
    for i in range(0, m, step):
        c, s = w4.quantize_fp8(x[i:i + step], act=ACTS[act])
        assert torch.equal(c.view(torch.uint8), codes[i:i + step].view(torch.uint8)), f"codes of rows from {i} on"
        assert torch.equal(s.nan_to_num(-1.0), scales[i:i + step].nan_to_num(-1.0)), f"scales of rows from {i} on"
    if act == "none":
        for at in (slice(0, 2), slice(m // 2, m // 2 + 1), slice(m - 2, m)):
            same_bits(codes[at, -4096:], scales[at, -32:], R.quantize_rows(x[at, -4096:].float().cpu().numpy()))


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_on_many_groups(dev, act):
    """Scales group by group, from the kernel of many groups: the product is that of the codes with their scales by row."""
    m, n, k = 4807, 130, 16000
    g = torch.Generator(device=dev).manual_seed(4)
    x = torch.randn(m, 2 * k if act == "swiglu" else k, generator=g, device=dev).to(BF16)
    codes, scales = w4.quantize_fp8_weight(torch.randn(n, k, generator=g, device=dev))
    say("linear on many groups", act)
    cx, sx = w4.quantize_fp8(x, act=ACTS[act])
    assert torch.equal(w4.linear_fp8(x, codes, scales, act=ACTS[act]), w4.linear_fp8(cx, codes, scales, x_scales=sx))
