"""Keys and values that are not numbers: a group of channels that holds one is stored as NaN, and nothing else is
touched by it."""
import numpy as np
import pytest
import torch

from tests import kv4_ref as ref
from tests import kv4_tight as tight
from tests.gpu_util import require_gpu, say
from tests.test_kv4_gpu import DT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def w4():
    import weight_only_int4_rtn_amd as m
    return m


@pytest.mark.parametrize("dts", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")], ids=["nan", "inf", "minus_inf"])
def test_a_group_with_no_number_is_stored_as_nan(dev, bad, d, dts):
    say("not a number", bad, d, dts)
    lib, hk, n, page, w = w4(), 2, 24, 16, min(d, 128)
    x = torch.randn(n, 1 + 2 * hk, d, generator=torch.Generator().manual_seed(d)).to(DT[dts])
    marks = [(3, 1, 0), (5, 2, d - 1), (8, 3, d // 2), (9, 4, 7), (16, 1, 33)]  # token, head (1, 2: keys; 3, 4: values), channel
    for t, h, c in marks:
        x[t, h, c] = bad
    x[20, 3] = bad  # a head of nothing else
    x[21, 2] = 0.0
    x[21, 2, 5] = bad
    pool = lib.kv4_pool(3, page, hk, d, device=dev)
    slots = torch.randperm(3 * page, generator=torch.Generator().manual_seed(1))[:n].to(dev)
    q = lib.kv4_append(x.view(n, -1).to(dev), pool, slots, d)
    assert torch.equal(q.cpu(), x[:, :1])
    k, v = (z.cpu() for z in lib.kv4_read(pool, slots, d, dtype=torch.float32))
    got = torch.cat((k, v), 1)
    broken = ~torch.isfinite(x[:, 1:].float()).unflatten(-1, (-1, w)).all(-1, keepdim=True).expand(n, 2 * hk, d // w, w).flatten(-2)
    assert torch.isnan(got[broken]).all() and int(broken.sum()) >= 7 * w
    clean = torch.where(broken, torch.zeros(()), x[:, 1:].float())
    want = torch.from_numpy(ref.quantized(clean.numpy(), w))
    assert torch.equal(got[~broken], want[~broken])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens", [1, 40, 600], ids=["decode", "chunk", "rows"])
def test_attention_over_nan_tokens(dev, tokens, d):
    """A key that is NaN makes every row that sees it NaN, a value its own channels; other rows and heads are as before."""
    say("attention over NaN", tokens, d)
    lib, n, hk, heads, page, w = w4(), 1300, 2, 8, 32, min(d, 128)
    g = torch.Generator().manual_seed(d)
    x = torch.randn(n, 2, hk, d, generator=g).to(torch.bfloat16)
    q = torch.randn(tokens, heads, d, generator=g).to(torch.bfloat16)
    first = n - tokens
    hurt = first + tokens // 2 if tokens > 1 else 400
    x[hurt, 0, 0, 3] = float("nan")                # key of the first head
    x[first // 2, 1, 1, d - 1] = float("inf")      # value of the second
    r = tight.Request(lib, dev, x, page, seed=3)
    out = r.attend(q).cpu()
    sees = torch.arange(first, n) >= hurt
    assert torch.isnan(out[sees][:, :4]).all()
    assert torch.isnan(out[:, 4:, d - w:]).all()
    r.k, r.v = np.nan_to_num(r.k, nan=0.0), np.nan_to_num(r.v, nan=0.0)
    want, tol = tight.attention(q, r.k, r.v, n, True, 0, d ** -0.5)
    ref.within(out[~sees][:, :4], want[~sees][:, :4], tol[~sees][:, :4], "rows before it")
    ref.within(out[:, 4:, :d - w], want[:, 4:, :d - w], tol[:, 4:, :d - w], "the other block")
