"""Scales at the ends of what the 8-bit float layer takes: both scales' product in FP32's normal range, each far outside of the
other's."""
import pytest
import torch

import weight_only_int4_rtn_amd as w4

from .gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(1, 300, 512), (12, 64, 16384), (40, 2101, 1024), (130, 12301, 384), (520, 8197, 384), (1025, 12301, 1152)])
@pytest.mark.parametrize("a,b", [(100, -90), (-100, 90), (60, 40), (-55, -55), (110, 0), (0, 110), (-110, 0)])
def test_powers_of_two_pass_through(m, n, k, a, b):
    """x 2^a and W 2^b: codes stay, scales and outputs are those of x and W times a power of two, bit for bit, as long as the
    largest output (below 2^12) and the smallest product of two scales (above 2^-17: normal values, 448 a scale) stay normal."""
    dev = require_gpu()
    g = torch.Generator(device=dev).manual_seed(m + k)
    x = torch.randn(m, k, generator=g, device=dev).to(torch.bfloat16)
    codes, scales = w4.quantize_fp8_weight(torch.randn(n, k, generator=g, device=dev))
    say("powers of two", m, n, k, a, b, w4.linear_fp8_tile(m, n, k))
    y = w4.linear_fp8(x, codes, scales).double()
    assert float(y.abs().max()) < 2.0 ** 12 and float(scales.min()) * float(w4.quantize_fp8(x)[1].min()) > 2.0 ** -17
    got = w4.linear_fp8((x.double() * 2.0 ** a).to(torch.bfloat16), codes, (scales.double() * 2.0 ** b).float()).double()
    # below bf16's normal numbers its steps are 2^-133
    want = y * 2.0 ** (a + b)
    assert ((got == want) | ((got - want).abs() <= 2.0 ** -134)).all()
