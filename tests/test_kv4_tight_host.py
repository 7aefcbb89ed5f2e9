"""The error bound of tests/kv4_tight.py, on the CPU: it accepts weights rounded to
f16 relative to a row's largest weight and rejects outputs that are damaged."""
import pytest
import torch

from tests import kv4_ref as ref
from tests import kv4_tight as tight

CASES = [(1200, 1, 64, 2, 1), (700, 2, 128, 4, 3), (300, 1, 256, 2, 5)]  # tokens, kv heads, channels, heads, queries


def inputs(case, ratio, blocks=1.0):
    n, hk, d, h, nq = case
    x, q = tight.outlier_inputs(n, hk, d, h, nq, ratio, [n // 3], torch.bfloat16, n + d, blocks)
    values = ref.quantized(x.float().numpy(), min(d, 128))
    return q, values[:, 0], values[:, 1], n


def to_largest_weight(p, vs):
    return (p.unsqueeze(-1) * vs).amax((1, 2)).view(-1, 1) / 32


def to_largest_scale(p, vs):
    return (p.amax(1) * vs.max()).view(-1, 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("ratio", [1.0, 2.0 ** 12, 2.0 ** 20])
def test_bound_accepts_and_rejects(case, ratio, dtype):
    q, k, v, n = inputs(case, ratio)
    scale = case[2] ** -0.5
    want, tol = tight.attention(q, k, v, n, True, 0, scale)
    ref.within(want.to(dtype), want, tol, "the value itself")
    ref.within(tight.model(q, k, v, n, True, 0, scale, to_largest_weight).to(dtype), want, tol, "weights by the largest weight")
    for what, damaged in (("ordinary tokens dropped", v * (abs(v) > 50 if ratio > 1 else 0)), ("half the tokens dropped", v.copy())):
        if what.startswith("half"):
            damaged[::2] = 0
        with pytest.raises(AssertionError, match=what):
            ref.within(tight.attention(q, k, damaged, n, True, 0, scale)[0].to(dtype), want, tol, what)
    if ratio > 2.0 ** 16:
        with pytest.raises(AssertionError, match="largest scale"):
            ref.within(tight.model(q, k, v, n, True, 0, scale, to_largest_scale).to(dtype), want, tol, "weights by the largest scale")


def test_bound_of_blocks_apart():
    """Blocks of one head whose scales are far apart: the smaller one's weights are as exact."""
    q, k, v, n = inputs(CASES[2], 1.0, blocks=2.0 ** -16)
    want, tol = tight.attention(q, k, v, n, True, 0, 1 / 16)
    ref.within(tight.model(q, k, v, n, True, 0, 1 / 16, to_largest_weight).to(torch.bfloat16), want, tol, "blocks")
    with pytest.raises(AssertionError, match="largest scale"):
        ref.within(tight.model(q, k, v, n, True, 0, 1 / 16, to_largest_scale).to(torch.bfloat16), want, tol, "largest scale")
