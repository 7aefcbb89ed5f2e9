"""Attention over the 4-bit cache where values of unlike size meet: tokens with large values that the softmax leaves
out, values that grow along the tokens, blocks of one head far apart in size.  The bound (tests/kv4_tight.py) follows
each token's share of its row."""
import pytest
import torch

from tests import kv4_tight as tight
from tests.gpu_util import require_gpu, say
from tests.test_kv4_gpu import DT

pytestmark = pytest.mark.gpu

FORMS = [(1, "decode"), (40, "chunk"), (600, "rows")]  # query tokens: one, tiles of 16 rows, tiles of 64 rows


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def w4():
    import weight_only_int4_rtn_amd as m
    return m


def tiles(tokens, heads, hk, d, n, page, causal=True):
    return w4().kv4_attention_tile_rows(tokens, 1, heads, hk, d, -(-n // page), page, ragged=tokens != 1, causal=causal)


def causal_for(at, n, tokens):
    """The outliers have to be seen by every query: no mask where they stand among the queries themselves."""
    return max(at) < n - tokens


@pytest.mark.parametrize("dts", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,form", FORMS, ids=[f[1] for f in FORMS])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("log_ratio", [10, 16])
def test_values_that_the_softmax_leaves_out(dev, log_ratio, where, tokens, form, d, dts):
    say("outliers without weight", log_ratio, where, form, d, dts)
    n, hk, heads, page = 1300, 2, 8, 32
    at = {"first": [0, 1], "middle": [n // 3, n // 3 + 40], "last": [n - 2]}[where]
    causal = causal_for(at, n, tokens)
    x, q = tight.outlier_inputs(n, hk, d, heads, tokens, 2.0 ** log_ratio, at, torch.bfloat16, n + d)
    r = tight.Request(w4(), dev, x, page, seed=d)
    assert tiles(tokens, heads, hk, d, n, page, causal) == (64 if form == "rows" else 16)
    q = q.to(DT[dts])
    r.check(q, r.attend(q, causal=causal), causal=causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,form", FORMS, ids=[f[1] for f in FORMS])
def test_values_far_above_the_rest_that_the_softmax_leaves_out(dev, tokens, form, d):
    """A ratio of 2^40, in bf16."""
    say("far outliers without weight", form, d)
    n, hk, heads, page = 1300, 2, 8, 32
    g = torch.Generator().manual_seed(5)
    x = torch.randn(n, 2, hk, d, generator=g)
    for t in (100, 611):
        x[t, 1] *= 2.0 ** 40
        x[t, 0] = 0.0
        x[t, 0, :, 0] = -512.0
    q = torch.randn(tokens, heads, d, generator=g)
    q[:, :, 0] = 2 * d ** 0.5  # logits of -1024 for those tokens, of 2 k[0] for the others
    x[:, 0, :, 0] = torch.where(x[:, 0, :, 0] < -100, x[:, 0, :, 0], x[:, 0, :, 0] * 0.1)
    x, q = x.to(torch.bfloat16), q.to(torch.bfloat16)
    r = tight.Request(w4(), dev, x, page, seed=d)
    causal = causal_for([611], n, tokens)
    r.check(q, r.attend(q, causal=causal), causal=causal)


@pytest.mark.parametrize("dts", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,form", FORMS, ids=[f[1] for f in FORMS])
@pytest.mark.parametrize("rising", [True, False])
def test_values_that_grow_or_shrink_along_the_tokens(dev, rising, tokens, form, d, dts):
    """Logits fall by as much as the values grow (and the other way round), so every part of the row counts."""
    say("slopes", rising, form, d, dts)
    n, hk, heads, page = 1300, 2, 8, 32
    g = torch.Generator().manual_seed(d + tokens)
    slope = torch.linspace(0, 12, n) if rising else torch.linspace(12, 0, n)   # base-2 exponent
    x = torch.randn(n, 2, hk, d, generator=g)
    x[:, 1] *= (2.0 ** (slope - 8)).view(n, 1, 1)
    x[:, 0] *= 0.1
    x[:, 0, :, 0] = -slope.view(n, 1) * 0.6931
    q = torch.randn(tokens, heads, d, generator=g)
    q[:, :, 0] = d ** 0.5
    x, q = x.to(DT[dts]), q.to(DT[dts])
    r = tight.Request(w4(), dev, x, page, seed=d)
    r.check(q, r.attend(q, causal=False), causal=False)


@pytest.mark.parametrize("dts", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,form", FORMS, ids=[f[1] for f in FORMS])
@pytest.mark.parametrize("log_blocks", [-16, 10])
def test_blocks_of_one_head_apart(dev, log_blocks, tokens, form, dts):
    say("blocks apart", log_blocks, form, dts)
    n, hk, heads, page, d = 900, 2, 16, 48, 256
    x, q = tight.outlier_inputs(n, hk, d, heads, tokens, 1.0, [n // 2], torch.bfloat16, 3, blocks=2.0 ** log_blocks)
    r = tight.Request(w4(), dev, x, page, seed=2)
    causal = causal_for([n // 2], n, tokens)
    q = q.to(torch.bfloat16 if log_blocks < -12 else DT[dts])
    r.check(q, r.attend(q, causal=causal), causal=causal)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,form", FORMS, ids=[f[1] for f in FORMS])
def test_tokens_without_values_take_the_weight(dev, tokens, form, d):
    """The largest logits stand on tokens whose values are all zero: the others' part of the row is small, not lost."""
    say("zero values with weight", form, d)
    n, hk, heads, page = 1300, 2, 8, 32
    g = torch.Generator().manual_seed(d + 9)
    x = torch.randn(n, 2, hk, d, generator=g)
    x[:3, 1] = 0.0
    x[:3, 0] = 0.0
    x[:3, 0, :, 0] = 32.0
    q = torch.randn(tokens, heads, d, generator=g)
    q[:, :, 0] = d ** 0.5
    x, q = x.to(torch.bfloat16), q.to(torch.bfloat16)
    r = tight.Request(w4(), dev, x, page, seed=d)
    out = r.attend(q)
    r.check(q, out)
    assert out.any(), "nothing left"
    # and nothing but zeros: a row of zeros
    x[:, 1] = 0.0
    r = tight.Request(w4(), dev, x, page, seed=d)
    assert not r.attend(q).any()


@pytest.mark.parametrize("tokens,form", FORMS, ids=[f[1] for f in FORMS])
def test_values_as_small_and_as_large_as_bf16_holds(dev, tokens, form):
    say("sizes of values", form)
    n, hk, heads, page, d = 700, 2, 16, 32, 128
    for size in (2.0 ** -70, 2.0 ** -30, 2.0 ** 30, 2.0 ** 90):
        g = torch.Generator().manual_seed(4)
        x = torch.randn(n, 2, hk, d, generator=g)
        x[:, 1] *= size
        q = torch.randn(tokens, heads, d, generator=g).to(torch.bfloat16)
        r = tight.Request(w4(), dev, x.to(torch.bfloat16), page, seed=1)
        r.check(q, r.attend(q), what=f"size {size:.1e}")
