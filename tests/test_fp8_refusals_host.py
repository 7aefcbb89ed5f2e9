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
