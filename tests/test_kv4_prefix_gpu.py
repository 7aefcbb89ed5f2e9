"""Attention for requests on shared prefixes, against 64 bits with a tolerance
derived from the kernels' roundings (kv4_prefix_ref)."""
import numpy as np
import pytest
import torch

from tests import kv4_prefix_ref as pref
from tests import kv4_ref as ref
from tests.gpu_util import require_gpu, say
from tests.test_kv4_gpu import DT, Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def w4():
    import weight_only_int4_rtn_amd as m
    return m


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


class Batch:
    """Prefixes and requests on one pool: `first` holds where each group's requests begin (cu_groups)."""

    def __init__(self, dev, prefix, own, first, heads, hk, d, page, dtype, q_lens=None, seed=0, qsize=1.5, **spread):
        self.dev, self.prefix, self.own, self.first, self.q_lens = dev, list(prefix), list(own), list(first), q_lens
        self.cache = Cache(dev, self.prefix + self.own, hk, d, page, seed=seed + sum(prefix) + d, **spread)
        self.counts = q_lens or [1] * len(own)
        g = torch.Generator().manual_seed(seed + 5)
        self.q = (qsize * torch.randn(sum(self.counts), heads, d, generator=g)).to(dtype)
        self.scale = d ** -0.5
        self.one = first == [0, len(own)] and len(prefix) == 1

    def tables(self):
        t = self.cache.table
        return t[:len(self.prefix)].contiguous(), t[len(self.prefix):].contiguous()

    def args(self, prefix=None, own=None):
        a, b = self.tables()
        cu = None
        if self.q_lens:
            cu = ints([sum(self.counts[:i]) for i in range(len(self.counts) + 1)], self.dev)
        return ((self.q.to(self.dev), self.cache.pool, a.to(self.dev), ints(self.prefix if prefix is None else prefix, self.dev),
                 b.to(self.dev), ints(self.own if own is None else own, self.dev)),
                dict(cu_q=cu, cu_groups=None if self.one else ints(self.first, self.dev)))

    def takes(self, rows):
        """That a call runs on tiles of `rows` rows over the prefixes (0: together with the own tokens)."""
        a, b = self.tables()
        got = w4().kv4_prefix_attention_tile_rows(self.q.shape[0], len(self.own), len(self.prefix), self.q.shape[1], self.cache.hk,
                                                  self.cache.d, a.shape[1], b.shape[1], self.cache.page, ragged=self.q_lens is not None)
        assert got == rows, f"tiles of {got} rows, not {rows}"

    def run(self, causal=True, **kw):
        a, k = self.args(kw.pop("prefix", None), kw.pop("own", None))
        return w4().kv4_prefix_attention(*a, **k, causal=causal, **kw)

    def check(self, out, causal=True, prefix=None, own=None, there=None, what="", scale=None):
        prefix, own = prefix or self.prefix, own or self.own
        row, n = 0, len(self.prefix)
        for b, count in enumerate(self.counts):
            j = next((g for g in range(n) if self.first[g] <= b < self.first[g + 1]), None)
            p = 0 if j is None else prefix[j]
            k = np.concatenate(([] if j is None else [self.cache.k[j][:p]]) + [self.cache.k[n + b][:own[b]]])
            v = np.concatenate(([] if j is None else [self.cache.v[j][:p]]) + [self.cache.v[n + b][:own[b]]])
            page = self.cache.page
            a = None if there is None or j is None else there[j][np.arange(p) // page]
            c = None if there is None else there[n + b][np.arange(own[b]) // page]
            seen = pref.seen_tokens(p, own[b], count, causal, a, c)
            want, tol = pref.attention(self.q[row:row + count], k, v, seen, self.scale if scale is None else scale)
            ref.within(out[row:row + count], want, tol, f"{what} request {b}")
            row += count


CASES = [
    # prefixes, own lengths, cu_groups, query lengths (None: one each), heads, kv_heads, dim, page, causal, dtype
    ([1], [0], [0, 1], None, 1, 1, 64, 16, True, "bf16"),
    ([16], [1], [0, 1], None, 8, 1, 256, 16, True, "bf16"),
    ([0], [0, 5, 1], [0, 3], None, 4, 2, 128, 16, True, "f16"),              # no prefix; a request that sees nothing
    ([100], [0, 1, 15, 16, 17, 33, 200], [0, 7], None, 8, 2, 64, 16, True, "bf16"),
    ([800], [3, 60], [0, 2], None, 8, 1, 256, 16, True, "bf16"),
    ([4097], [1, 129, 300, 0, 31, 7, 64, 90], [0, 8], None, 16, 4, 128, 64, True, "bf16"),
    ([257], [40] * 40, [0, 40], None, 12, 4, 128, 48, True, "f16"),
    ([5000], list(range(20)), [0, 20], None, 7, 1, 64, 128, True, "bf16"),
    ([300, 0, 1, 47], [9, 1, 0, 30, 2, 2, 700], [0, 2, 4, 4, 7], None, 6, 2, 128, 16, True, "bf16"),  # a group of nobody
    ([130, 64], [5, 6, 7, 8, 9], [1, 2, 4], None, 4, 4, 64, 32, True, "f16"),   # requests of no group at both ends
    ([2000, 900, 33], [100, 3, 50] * 9, [0, 9, 20, 27], None, 32, 8, 128, 64, True, "bf16"),
    ([50], [20, 3, 1], [0, 3], [20, 3, 1], 4, 1, 64, 16, True, "bf16"),
    ([500], [80, 3, 200], [0, 3], [7, 3, 150], 6, 2, 128, 32, True, "f16"),
    ([500], [80, 3, 200], [0, 3], [7, 3, 150], 6, 2, 128, 32, False, "bf16"),
    ([90], [4, 0], [0, 2], [9, 2], 3, 1, 64, 16, True, "bf16"),                # more queries than tokens: the first see the prefix alone
    ([1200, 700], [150, 90, 1, 0, 260], [0, 3, 5], [140, 90, 1, 0, 33], 16, 16, 64, 32, True, "f16"),
    ([700, 20], [70, 300, 9], [0, 2, 3], [64, 200, 1], 8, 1, 256, 16, True, "bf16"),
    ([1500], [200, 400, 350], [0, 3], [200, 333, 350], 8, 2, 128, 64, True, "bf16"),
    ([900], [128] * 24, [0, 24], [16] * 24, 8, 8, 128, 16, False, "bf16"),
]


# Calls with something to share take two launches: over the prefixes on tiles of 16 rows or 64, then over the own tokens.
APART = [
    (16, [1000], [1, 30, 0, 200, 64] * 13, [0, 65], None, 8, 8, 64, 16, True, "bf16"),
    (16, [700, 0, 1500], [3, 1, 77] * 20, [0, 25, 30, 60], None, 16, 4, 64, 48, True, "f16"),
    (16, [2049], [5, 0, 129, 40] * 12, [2, 47], None, 16, 8, 128, 64, True, "bf16"),        # requests of no group at both ends
    (16, [900, 400], [1, 2, 300] * 14, [0, 20, 42], None, 24, 8, 128, 32, True, "f16"),
    (16, [1100], [17, 9, 0, 60] * 12, [0, 48], None, 8, 8, 256, 16, True, "bf16"),
    (16, [800, 1000], [30, 12, 9, 50] * 12, [0, 20, 48], [5, 12, 1, 8] * 12, 8, 8, 64, 16, True, "bf16"),
    (16, [1400], [20, 12, 9, 40] * 11, [0, 44], [5, 20, 1, 8] * 11, 8, 4, 256, 32, False, "f16"),
    (64, [1500, 900], [150, 90, 300, 40, 260, 17], [0, 3, 6], [140, 90, 280, 1, 233, 16], 32, 8, 64, 32, True, "f16"),
    (64, [2100], [200, 333, 350, 31], [0, 4], [180, 333, 290, 31], 16, 2, 128, 64, True, "bf16"),
    (64, [1700, 0, 60], [220, 333, 100, 7], [0, 2, 3, 4], [220, 300, 90, 9], 24, 8, 128, 16, False, "bf16"),
    (64, [1600], [270, 1, 300, 310], [0, 4], [260, 1, 300, 301], 24, 3, 256, 16, True, "f16"),
]


def name(c):
    cut = lambda v: "_".join(map(str, v[:5])) + ("x" * (len(v) > 5))  # noqa: E731
    return f"p{cut(c[0])}-o{cut(c[1])}-q{cut(c[3]) if c[3] else 1}-h{c[4]}_{c[5]}-d{c[6]}-{'c' if c[8] else 'b'}-{c[9]}"


@pytest.mark.parametrize("case", CASES, ids=[name(c) for c in CASES])
def test_prefix(dev, case):
    prefix, own, first, qs, h, hk, d, page, causal, dts = case
    say("prefix", case)
    b = Batch(dev, prefix, own, first, h, hk, d, page, DT[dts], qs)
    out = b.run(causal)
    assert out.shape == b.q.shape and out.dtype == DT[dts]
    b.check(out, causal, what=str(case))
    assert torch.equal(b.run(causal).view(torch.int16), out.view(torch.int16)), "two runs differ"


@pytest.mark.parametrize("case", APART, ids=[f"t{c[0]}-" + name(c[1:]) for c in APART])
def test_prefix_apart(dev, case):
    rows, prefix, own, first, qs, h, hk, d, page, causal, dts = case
    say("prefix apart", case)
    b = Batch(dev, prefix, own, first, h, hk, d, page, DT[dts], qs)
    b.takes(rows)
    out = b.run(causal)
    b.check(out, causal, what=str(case))
    assert torch.equal(b.run(causal).view(torch.int16), out.view(torch.int16)), "two runs differ"


@pytest.mark.parametrize("spread,vsize,voutlier,qsize,scale", [
    (1.0, 1e-3, 0.0, 1.5, None), (1.0, 3e4, 0.0, 1.5, None), (1.0, 1.0, 3000.0, 1.5, None), (40.0, 1.0, 0.0, 30.0, None),
    (1.0, 1.0, 0.0, 1.5, -0.3), (1e-4, 1.0, 0.0, 1e-4, 1.0), (1.0, 1.0, 0.0, 1e5, 1e-5),
], ids=["small_v", "large_v", "outlier_v", "one_hot", "negative_scale", "flat", "large_q"])
@pytest.mark.parametrize("rows,qs", [(0, None), (0, [70, 130, 1]), (16, None), (64, [300, 450, 256])], ids=["decode", "chunk", "apart16", "apart64"])
def test_prefix_ranges(dev, spread, vsize, voutlier, qsize, scale, rows, qs):
    say("prefix ranges", spread, vsize, voutlier, qsize, scale, qs)
    if rows == 0:
        b = Batch(dev, [600], [133, 200, 40], [0, 3], 8, 2, 128, 32, torch.bfloat16, qs, seed=3, qsize=qsize, spread=spread, vsize=vsize,
                  voutlier=voutlier)
    elif rows == 16:
        b = Batch(dev, [1000], [33, 60, 1, 0] * 9, [0, 36], 8, 8, 128, 32, torch.bfloat16, qs, seed=3, qsize=qsize, spread=spread,
                  vsize=vsize, voutlier=voutlier)
    else:
        b = Batch(dev, [1600], [300, 500, 260], [0, 3], 16, 4, 128, 32, torch.bfloat16, qs, seed=3, qsize=qsize, spread=spread,
                  vsize=vsize, voutlier=voutlier)
    b.takes(rows)
    b.check(b.run(scale=scale), scale=scale)


@pytest.mark.parametrize("rows,qs", [(16, None), (64, [300, 450, 20, 290])], ids=["apart16", "apart64"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefix_apart_bad_pages_and_lengths(dev, rows, qs, d):
    say("bad pages apart", rows, d)
    heads, own, first = (16, [300, 500, 20, 290], [0, 1, 4]) if qs else (8, [20, 33, 1, 64] * 16, [0, 20, 64])
    b = Batch(dev, [1500, 700], own, first, heads, 8, d, 32, torch.bfloat16, qs)
    b.takes(rows)
    n = 2 + len(own)
    there = [np.ones(64, bool) for _ in range(n)]
    for i, p, bad in ((0, 2, -1), (0, 40, b.cache.pool.shape[0]), (1, 0, 2 ** 31 - 1), (2, 0, -2 ** 31), (n - 1, 1, 10 ** 6)):
        b.cache.table[i, p] = bad
        there[i][p] = False
    b.check(b.run(), there=there, what="bad pages")
    short = [1100, 0]
    mine = own[:]
    mine[1] = 0 if qs is None else own[1]
    b.check(b.run(prefix=[1100, -5], own=mine), prefix=short, own=mine, there=there, what="lengths")


@pytest.mark.parametrize("qs", [None, [40, 9, 30]], ids=["decode", "chunk"])
def test_prefix_bad_pages_and_lengths(dev, qs):
    """Pages outside the pool are not seen, in the prefix or behind it; lengths beyond a table end there, negative ones are none."""
    say("bad pages", qs)
    b = Batch(dev, [400, 64], [95, 64, 40], [0, 1, 3], 4, 2, 64, 32, torch.float16, qs)
    there = [np.ones(64, bool) for _ in range(5)]
    for i, p, bad in ((0, 2, -1), (0, 9, b.cache.pool.shape[0]), (1, 0, 2 ** 31 - 1), (2, 1, -2 ** 31), (4, 0, 10 ** 6)):
        b.cache.table[i, p] = bad
        there[i][p] = False
    b.check(b.run(), there=there, what="bad pages")
    b = Batch(dev, [64, 50], [64, 33, 9], [0, 2, 3], 4, 2, 64, 16, torch.bfloat16)
    b.cache.table = b.cache.table[:, :4].contiguous()
    out = b.run(prefix=[10 ** 6, -3], own=[2 ** 31 - 1, -2 ** 31, 9])
    b.check(out, prefix=[64, 0], own=[64, 0, 9], what="lengths")


def test_prefix_requests_outside_the_batch(dev):
    """Groups that begin before the batch or end behind it take the requests that there are."""
    say("cu_groups beyond the batch")
    b = Batch(dev, [70, 40], [5, 6, 7], [-3, 1, 50], 4, 2, 64, 16, torch.bfloat16)
    b.check(b.run(), what="cu_groups beyond the batch")


def test_prefix_rows_behind_the_last_sequence_stay(dev):
    say("rows behind the last sequence")
    b = Batch(dev, [300], [20, 40], [0, 2], 4, 2, 128, 16, torch.bfloat16, [3, 5])
    args, kw = b.args()
    q = torch.cat((args[0], torch.full_like(args[0][:4], float("nan"))))
    out = torch.full_like(q, 7.0)
    got = w4().kv4_prefix_attention(q, *args[1:], **kw, out=out)
    assert got is out and (out[8:] == 7.0).all()
    b.check(out[:8], what="the others")


def test_prefix_strided_rows_and_tables(dev):
    lib = w4()
    say("strided q and tables")
    b = Batch(dev, [200, 77], [12, 300, 4], [0, 2, 3], 4, 2, 128, 16, torch.bfloat16)
    want = b.run()
    (q, pool, table, lens, own, own_lens), kw = b.args()
    wide = torch.full((3, 4 * 128 + 72), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 8:520] = q.view(3, 512)
    def spread(t):
        s = torch.full((t.shape[0], t.shape[1] + 5), 2 ** 30, dtype=torch.int32, device=dev)
        s[:, :t.shape[1]] = t
        return s[:, :t.shape[1]]
    got = lib.kv4_prefix_attention(wide[:, 8:520].unflatten(1, (4, 128)), pool, spread(table), lens, spread(own), own_lens, **kw)
    assert torch.equal(got, want)


def test_prefix_equals_attention_over_both(dev):
    """A request's prefix and own pages in one block table of kv4_attention: the same within two roundings of the output."""
    lib = w4()
    say("against kv4_attention")
    b = Batch(dev, [512], [30, 64, 1, 100], [0, 4], 8, 2, 128, 64, torch.float16)
    (q, pool, table, lens, own, own_lens), _ = b.args()
    whole = torch.cat((table[:, :8].expand(4, 8), own), 1).contiguous()
    a = lib.kv4_attention(q, pool, whole, own_lens + 512).double()
    c = b.run().double()
    assert ((a - c).abs() <= 2.0 ** -9 * a.abs() + 2.0 ** -9 * a.abs().amax()).all()


@pytest.mark.parametrize("rows,qs", [(0, None), (0, [40, 200, 8]), (16, None), (64, [300, 450, 256])], ids=["decode", "chunk", "apart16", "apart64"])
def test_prefix_on_another_stream_and_in_a_graph(dev, rows, qs):
    lib = w4()
    say("stream and graph", rows, qs)
    own = [100, 250, 9] if rows == 0 else [40, 33, 1] * 12 if rows == 16 else [300, 480, 260]
    changed = [99, 210, 8] if rows == 0 else [39, 0, 1] * 12 if rows == 16 else [300, 470, 256]
    heads = 16 if rows == 64 else 8
    b = Batch(dev, [3000], own, [0, len(own)], heads, 2 if rows == 0 else 8, 128, 32, torch.bfloat16, qs)
    b.takes(rows)
    want = b.run()
    args, kw = b.args()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = lib.kv4_prefix_attention(*args, **kw)
    side.synchronize()
    assert torch.equal(got, want)
    need = lib.kv4_prefix_attention_workspace_bytes(b.q.shape[0], len(own), 1, heads, b.cache.hk, 128, args[2].shape[1], args[4].shape[1], 32, ragged=qs is not None)
    ws, out = torch.zeros(need, dtype=torch.uint8, device=dev), torch.empty_like(args[0])
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for graph in graphs:  # two graphs that share a workspace, replayed one after the other
        with torch.cuda.graph(graph):
            lib.kv4_prefix_attention(*args, **kw, out=out, workspace=ws)
    for rep in range(4):
        out.fill_(float("nan"))
        graphs[rep % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {rep}"
        assert torch.equal(lib.kv4_prefix_attention(*args, **kw), want)
    # other lengths in the same graph: the plan does not depend on them
    args[3].copy_(ints([1700], dev))
    args[5].copy_(ints(changed, dev))
    graphs[0].replay()
    torch.cuda.synchronize()
    b.check(out, prefix=[1700], own=changed, what="replay with other lengths")
    assert not ws[:1 << 20].any(), "the workspace's header is not zero"


@pytest.mark.parametrize("rows", [0, 16, 64])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefix_nan_tokens(dev, d, rows):
    """A key of the prefix that is NaN makes every row of its group and heads NaN, an own one its request's; others stay."""
    say("NaN tokens", d)
    lib = w4()
    if rows == 0:
        b = Batch(dev, [200, 90], [40, 33, 20], [0, 2, 3], 4, 2, d, 16, torch.bfloat16)
    elif rows == 16:
        b = Batch(dev, [1500, 900], [40, 33, 20] * 20, [0, 2, 60], 8, 8, d, 16, torch.bfloat16)
    else:
        b = Batch(dev, [1500, 900], [300, 433, 320], [0, 2, 3], 32, 8, d, 16, torch.bfloat16, [300, 1, 300])
    b.takes(rows)
    hk = b.cache.hk
    x = torch.ones(1, 2 * hk, d, dtype=torch.bfloat16, device=dev)  # the other heads stay numbers
    x[:, 0] = x[:, hk] = float("nan")
    page = b.cache.page
    slot = int(b.cache.table[1, 50 // page]) * page + 50 % page          # the second group's prefix
    mine = int(b.cache.table[2 + 1, 7 // page]) * page + 7 % page        # request 1's own tokens
    for s in (slot, mine):
        lib.kv4_append(x.flatten(1), b.cache.pool, torch.tensor([s], device=dev), d)
    out, share, n = b.run().cpu(), b.q.shape[1] // hk, b.counts[0]
    assert torch.isnan(out[n:, :share]).all() and torch.isfinite(out[:, share:]).all() and torch.isfinite(out[:n]).all()
    b.counts = [n]
    b.check(out[:n], what="the first request")
