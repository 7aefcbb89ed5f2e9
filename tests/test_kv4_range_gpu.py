"""Attention over the 4-bit cache with queries as large and as small as bf16 holds."""
import pytest
import torch

from tests import kv4_tight as tight
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def w4():
    import weight_only_int4_rtn_amd as m
    return m


@pytest.mark.parametrize("tokens,form", [(1, "decode"), (40, "chunk"), (600, "rows")], ids=["decode", "chunk", "rows"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("size", [3.3e38, 2.5e38, 1e-30])
def test_sizes_of_queries(dev, size, d, tokens, form):
    """Keys and the scale bring the logits back to ordinary size."""
    say("queries of size", size, d, form)
    n, hk, heads, page = 700, 2, 16, 32
    g = torch.Generator().manual_seed(d)
    x = torch.randn(n, 2, hk, d, generator=g)
    x[:, 0] *= 2.0 ** -20 if size > 1 else 2.0 ** 40
    q = torch.rand(tokens, heads, d, generator=g) * 2 - 1
    q[:, :, 5] = 1.0
    q = (q.double() * size).to(torch.bfloat16)
    assert torch.isfinite(q.float()).all()
    x = x.to(torch.bfloat16)
    scale = 2.0 ** 20 / size / d ** 0.5 if size > 1 else 2.0 ** -40 / size / d ** 0.5
    r = tight.Request(w4(), dev, x, page, seed=1)
    r.check(q, r.attend(q, causal=False, scale=scale), causal=False, scale=scale)
