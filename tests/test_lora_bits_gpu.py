"""How many bits of x A^T reach the second product: rank components of unlike size that B brings back to one size,
beside a y that takes nearly all of the sum away, so that what is left shows the product's own error."""
import pytest
import torch

from tests import kv4_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def w4():
    import weight_only_int4_rtn_amd as m
    return m


# m, n, k, adapters, rank: one launch; tiles of 16; gathered tiles of 64; many rows (tiles of 64 in order)
SIZES = [(2, 200, 256, 2, 16), (20, 520, 512, 3, 16), (64, 300, 256, 9, 24), (1100, 16901, 64, 4, 16)]


@pytest.mark.parametrize("spread", [0, 10, 14], ids=lambda s: f"spread{s}")
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_rank_components_of_unlike_size(dev, size, dtype, spread):
    m, n, k, adapters, rank = size
    say("rank components", size, dtype, spread)
    lib = w4()
    g = torch.Generator().manual_seed(m + spread)
    fall = 2.0 ** -(torch.arange(rank) * spread / (rank - 1))
    x = (4 * torch.randn(m, k, generator=g)).to(dtype)
    a = (8 * torch.randn(adapters, rank, k, generator=g) * k ** -0.5 * fall.view(1, rank, 1)).to(dtype)
    b = (torch.randn(adapters, n, rank, generator=g) * 2.0 ** -spread / fall).to(dtype)
    index = torch.randint(0, adapters, (m,), generator=g, dtype=torch.int32)
    some = torch.arange(m) if m < 100 else torch.randperm(m, generator=g)[:40]  # rows that are looked at
    zero = torch.zeros(m, n, dtype=dtype)
    whole = torch.zeros(m, n, dtype=torch.float64)
    whole[some] = ref.lora(zero[some], x[some], a, b, index[some], None)[0]
    y = (-whole).to(dtype)
    want, tol = ref.lora(y[some], x[some], a, b, index[some], None)
    assert float(want.abs().mean()) < 2.0 ** (-8 if dtype == torch.bfloat16 else -11) * float(whole[some].abs().mean())
    out = lib.lora_add(*(t.to(dev) for t in (y, x, a, b, index))).cpu()
    ref.within(out[some], want, tol, str(size))


def test_components_near_the_largest_number(dev):
    """x A^T times its scale close to FP32's largest number, with B's column zero there: y comes back."""
    say("near the largest number")
    lib = w4()
    for dtype in (torch.bfloat16, torch.float16):
        x = torch.zeros(3, 8, dtype=dtype)
        x[:, 0] = 1.0
        a = torch.zeros(1, 8, 8, dtype=dtype)
        a[0, 0, 0] = 1.875
        a[0, 1, 0] = 1.0
        b = torch.zeros(1, 40, 8, dtype=dtype)
        y = torch.randn(3, 40, generator=torch.Generator().manual_seed(1)).to(dtype)
        index, scales = torch.zeros(3, dtype=torch.int32), torch.tensor([2.0 ** 127])  # 1.875 * 2^127 is 3.19e38
        out = lib.lora_add(*(t.to(dev) for t in (y, x, a, b, index)), scales=scales.to(dev))
        assert torch.equal(out.cpu(), y)
