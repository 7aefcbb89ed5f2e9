"""Attention over the 4-bit cache on tiles of 64 rows, a kernel of its own: every case asserts that it takes it.
Both types and all head widths, from no sharing to many query heads on one key head, masks that leave rows empty,
bad pages, unlike sizes of values and logits, strided inputs; and block tables wider than the requests."""
import numpy as np
import pytest
import torch

from tests import kv4_ref as ref
from tests import kv4_tight as tight
from tests.gpu_util import require_gpu, say
from tests.test_kv4_gpu import DT, Cache, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def w4():
    import weight_only_int4_rtn_amd as m
    return m


def tiles_of(cache, qs, heads, causal, window):
    return w4().kv4_attention_tile_rows(sum(qs) if qs else len(cache.k), len(cache.k), heads, cache.hk, cache.d, cache.table.shape[1],
                                        cache.page, ragged=qs is not None, causal=causal, window=window)


def check(cache, q, counts, kv_lens, causal, window, out, scale=None, what="", pages_there=None):
    row = 0
    for i, n in enumerate(counts):
        there = None if pages_there is None else pages_there[i][np.arange(kv_lens[i]) // cache.page]
        want, tol = tight.attention(q[row:row + n], cache.k[i][:kv_lens[i]], cache.v[i][:kv_lens[i]], kv_lens[i], causal, window,
                                    cache.d ** -0.5 if scale is None else scale, there)
        ref.within(out[row:row + n], want, tol, f"{what} request {i}")
        row += n


CASES = [
    # kv lengths, query lengths, heads, kv_heads, dim, page, causal, window
    ([900, 33, 1], [600, 33, 1], 16, 16, 64, 16, True, 0),          # no shared heads
    ([900, 330, 64], [300, 290, 3], 24, 24, 64, 32, True, 100),
    ([1200], [400], 12, 12, 128, 48, True, 0),
    ([600, 500], [290, 400], 8, 8, 256, 16, True, 0),
    ([1500, 20], [260, 1], 20, 4, 64, 80, True, 300),               # 5 heads share one: tiles start inside a query
    ([1111], [333], 14, 2, 128, 64, True, 0),                       # 7
    ([700, 650], [333, 40], 20, 1, 128, 32, False, 61),             # 20
    ([900], [330], 24, 1, 256, 64, True, 17),                       # 24
    ([800, 700], [800, 200], 6, 2, 64, 16, False, 0),               # 3
    ([200, 0, 300], [500, 40, 400], 16, 4, 64, 16, True, 0),        # more queries than tokens: rows that see nothing
    ([100, 64], [700, 400], 24, 6, 128, 128, True, 33),
    ([40, 300], [500, 200], 32, 2, 256, 32, True, 0),
    ([130], [900], 24, 2, 256, 32, False, 40),
]


@pytest.mark.parametrize("dts", ["bf16", "f16"])
@pytest.mark.parametrize("case", CASES, ids=[f"kv{'_'.join(map(str, c[0]))}-q{'_'.join(map(str, c[1]))}-h{c[2]}_{c[3]}-d{c[4]}-{'c' if c[6] else 'b'}{c[7]}" for c in CASES])
def test_row_tiles(dev, case, dts):
    kv, qs, h, hk, d, page, causal, window = case
    say("row tiles", case, dts)
    cache = Cache(dev, kv, hk, d, page, seed=sum(kv) + d)
    # room for more tokens than these requests have, as a server's table has; enough for this kernel
    wide = torch.full((len(kv), max(cache.table.shape[1], -(-2048 // page))), -1, dtype=torch.int32)
    wide[:, :cache.table.shape[1]] = cache.table
    cache.table = wide
    if window:
        # a short window keeps a call of this size on the other tiles: each request four times
        kv, qs = kv * 4, qs * 4
        cache.table, cache.k, cache.v = cache.table.repeat(4, 1), cache.k * 4, cache.v * 4
    assert tiles_of(cache, qs, h, causal, window) == 64
    q, counts, out = run_attention(dev, cache, qs, kv, h, causal, window, DT[dts])
    check(cache, q, counts, kv, causal, window, out, what=str(case))
    again = run_attention(dev, cache, qs, kv, h, causal, window, DT[dts])[2]
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "two runs differ"


@pytest.mark.parametrize("dts", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("spread,vsize,voutlier,qsize,scale", [
    (1.0, 1e-3, 0.0, 1.5, None),
    (1.0, 3e4, 0.0, 1.5, None),
    (1.0, 1.0, 3000.0, 1.5, None),
    (40.0, 1.0, 0.0, 30.0, None),
    (1.0, 1.0, 0.0, 1.5, -0.3),
    (1e-4, 1.0, 0.0, 1e-4, 1.0),
    (1.0, 1.0, 0.0, 1e4, 1e-4),
], ids=["small_v", "large_v", "outlier_v", "one_hot", "negative_scale", "flat", "large_q"])
def test_row_tiles_ranges(dev, spread, vsize, voutlier, qsize, scale, d, dts):
    say("row tiles, ranges", spread, vsize, voutlier, qsize, scale, d, dts)
    kv, qs = [333, 1200], [70, 300]
    cache = Cache(dev, kv, 4, d, 32, seed=9, spread=spread, vsize=vsize if dts == "bf16" or vsize < 1e4 else 3e3, voutlier=voutlier)
    assert tiles_of(cache, qs, 16, True, 0) == 64
    q, counts, out = run_attention(dev, cache, qs, kv, 16, True, 0, DT[dts], scale=scale, qsize=qsize)
    check(cache, q, counts, kv, True, 0, out, scale=scale)


@pytest.mark.parametrize("dts", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_row_tiles_pages_outside_the_pool(dev, d, dts):
    say("row tiles, bad pages", d, dts)
    kv, qs = [400, 950], [300, 333]
    cache = Cache(dev, kv, 4, d, 32, seed=3)
    there = [np.ones(64, bool), np.ones(64, bool)]
    for i, p, bad in ((0, 2, -1), (0, 7, cache.pool.shape[0]), (1, 0, 2 ** 31 - 1), (1, 2, -2 ** 31), (1, 29, -5)):
        cache.table[i, p] = bad
        there[i][p] = False
    assert tiles_of(cache, qs, 16, True, 0) == 64
    q, counts, out = run_attention(dev, cache, qs, kv, 16, True, 0, DT[dts])
    check(cache, q, counts, kv, True, 0, out, what="bad pages", pages_there=there)


def test_row_tiles_strided_queries_and_table(dev):
    lib = w4()
    say("row tiles, strided q and table, out given")
    kv, qs = [700, 400], [300, 333]
    cache = Cache(dev, kv, 4, 128, 16, seed=6)
    assert tiles_of(cache, qs, 16, True, 0) == 64
    q, counts, out = run_attention(dev, cache, qs, kv, 16, True, 0, torch.float16)
    check(cache, q, counts, kv, True, 0, out)
    n, w = sum(qs), 16 * 128
    wide = torch.full((n, w + 72), float("nan"), dtype=torch.float16, device=dev)
    wide[:, 8:8 + w] = q.view(n, w).to(dev)
    table = torch.full((2, cache.table.shape[1] + 5), 2 ** 30, dtype=torch.int32, device=dev)
    table[:, :cache.table.shape[1]] = cache.table.to(dev)
    given = torch.full((n, 16, 128), float("nan"), dtype=torch.float16, device=dev)
    got = lib.kv4_attention(wide[:, 8:8 + w].unflatten(1, (16, 128)), cache.pool, table[:, :cache.table.shape[1]],
                            torch.tensor(kv, dtype=torch.int32, device=dev),
                            cu_q=torch.tensor([0, qs[0], n], dtype=torch.int32, device=dev), out=given)
    assert got is given and torch.equal(got, out)


@pytest.mark.parametrize("room", [2048, 32768, 131072])
@pytest.mark.parametrize("qs", [None, [200, 2, 400]], ids=["decode", "chunks"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_tables_wider_than_the_requests(dev, d, qs, room):
    """A server's block table has room for its longest context; what lies beyond a request's pages is never followed."""
    say("wide tables", d, qs, room)
    kv = [1000, 3, 700]
    cache = Cache(dev, kv, 2, d, 16, seed=21 + d)
    wide = torch.full((3, room // 16), 2 ** 30, dtype=torch.int32)
    wide[:, :cache.table.shape[1]] = cache.table
    cache.table = wide
    assert tiles_of(cache, qs, 8, True, 0) == (16 if qs is None else 64)
    q, counts, out = run_attention(dev, cache, qs, kv, 8, True, 0, torch.bfloat16)
    check(cache, q, counts, kv, True, 0, out, what="wide table")
