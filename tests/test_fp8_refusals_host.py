"""Calls of the 8-bit float layer that need no launch (no GPU): inputs that autograd would record, and empty ones."""
import pytest
import torch

import weight_only_int4_rtn_amd as w4


def test_codes_that_autograd_would_record_are_refused():
    x, codes, scales = torch.zeros(3, 256, dtype=torch.bfloat16), torch.zeros(130, 256).to(torch.float8_e4m3fn), torch.zeros(2, 2)
    kept = codes.clone().requires_grad_()
    with pytest.raises(ValueError, match="inference only"):
        w4.linear_fp8(x, kept, scales)
    with pytest.raises(ValueError, match="inference only"):
        w4.linear_fp8(codes[:3].clone().requires_grad_(), codes, scales, x_scales=torch.zeros(3, 2))
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):  # a parameter under no_grad passes, up to its device
        w4.linear_fp8(x, torch.nn.Parameter(codes), scales)


@pytest.mark.parametrize("m,n", [(0, 300), (0, 0), (100, 0)])
def test_empty_codes_have_no_scales(m, n):
    """The C entry point on codes of no rows, or weights of none: nothing to do, whatever the addresses are."""
    from weight_only_int4_rtn_amd import _binding as B
    from weight_only_int4_rtn_amd import _fp8
    assert _fp8._lib().fp8_linear(None, _fp8.E4M3, None, 0, m, 512, 512, None, None, n, None, None, B.BF16, n, None, 0, None) == B.OK
