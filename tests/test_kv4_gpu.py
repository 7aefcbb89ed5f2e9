"""The 4-bit paged cache and attention over it, against plain implementations
(tests/kv4_ref.py): appended values bit for bit, attention within a tolerance
derived from the kernel's roundings."""
import numpy as np
import pytest
import torch

from tests import kv4_ref as ref
from tests.gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def w4():
    import weight_only_int4_rtn_amd as m
    return m


def f32(t):
    return t.detach().cpu().float().numpy()


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------

APPEND = [
    # tokens, heads, kv_heads, dim, page, rot, interleaved, dtype, extra columns of a row
    (1, 8, 1, 256, 16, 256, False, "bf16", 0),
    (1, 1, 1, 64, 16, 16, True, "f16", 0),
    (17, 3, 3, 64, 48, 64, False, "bf16", 8),
    (33, 0, 2, 128, 64, 64, False, "f16", 0),
    (130, 7, 1, 128, 4096, 128, True, "bf16", 24),
    (65, 16, 4, 256, 32, 0, False, "f16", 0),
    (300, 5, 5, 64, 16, 48, True, "bf16", 0),
    (41, 4, 2, 128, 80, 112, False, "f16", 40),
]


@pytest.mark.parametrize("case", APPEND, ids=[f"t{c[0]}_h{c[1]}_{c[2]}_d{c[3]}_p{c[4]}_r{c[5]}_{'i' if c[6] else 'h'}_{c[7]}" for c in APPEND])
def test_append_equals_fp32_steps(dev, case):
    t, h, hk, d, page, rot, inter, dts, extra = case
    lib, dt = w4(), DT[dts]
    say("append", case)
    g = torch.Generator().manual_seed(t * 31 + d)
    width = (h + 2 * hk) * d
    x = torch.randn(t, width, generator=g) * torch.exp(2 * torch.randn(t, 1, generator=g))
    x[t // 2, h * d:h * d + 16] = 0.0
    if t > 4:
        x[3] = 0.0       # zero groups
        x[4] *= 2.0 ** -14  # small ones
    x = x.to(dt)
    full = torch.full((t, width + extra), 7.0, dtype=dt)
    full[:, :width] = x
    qkv = full.to(dev)[:, :width]
    pages = -(-t // page) + 2
    pool = lib.kv4_pool(pages, page, hk, d, device=dev)
    pool.random_(0, 256)
    slots = torch.randperm(pages * page, generator=g)[:t]
    dropped = torch.rand(t, generator=g) < (0.2 if t > 1 else 0.0)
    given = torch.where(dropped, torch.tensor([-1, pages * page, 2 ** 40, -2 ** 40])[torch.arange(t) % 4], slots)
    others = torch.tensor(sorted(set(range(pages * page)) - set(slots[~dropped].tolist())))
    before = [z.cpu() for z in lib.kv4_read(pool, others.to(dev), d, dtype=torch.float32)]
    positions = table = None
    if rot:
        table = lib.rope_table(1000, rot, device=dev)
        positions = torch.randint(0, 1000, (t,), generator=g, dtype=torch.int32)
    q = lib.kv4_append(qkv, pool, given.to(dev), d, positions=None if positions is None else positions.to(dev), rope=table,
                       interleaved=inter)
    xs = f32(x).reshape(t, h + 2 * hk, d)
    if rot:
        xs[:, :h + hk] = ref.rotated(xs[:, :h + hk], table.cpu().numpy(), positions.numpy(), inter)
    assert torch.equal(q.cpu(), torch.from_numpy(xs[:, :h].copy()).to(dt))
    keep = ~dropped.numpy()
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        k, v = lib.kv4_read(pool, given.to(dev), d, dtype=dtype)
        for got, part in ((k, xs[:, h:h + hk]), (v, xs[:, h + hk:])):
            want = torch.from_numpy(np.where(keep[:, None, None], ref.quantized(part, min(d, 128)), np.float32(0)))
            assert torch.equal(got.cpu(), want.to(dtype)), (dtype, float((got.cpu().float() - want).abs().max()))
    after = [z.cpu() for z in lib.kv4_read(pool, others.to(dev), d, dtype=torch.float32)]
    assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(before, after)), "other tokens changed"


def test_append_position_outside_the_table(dev):
    lib = w4()
    say("positions outside the table")
    d, page = 64, 16
    pool = lib.kv4_pool(2, page, 1, d, device=dev)
    table = lib.rope_table(8, 64, device=dev)
    qkv = torch.ones(4, 3 * d, dtype=torch.bfloat16, device=dev)
    positions = torch.tensor([0, 8, -1, 7], dtype=torch.int32, device=dev)
    q = lib.kv4_append(qkv, pool, torch.arange(4, device=dev), d, positions=positions, rope=table)
    assert torch.isnan(q.float()).flatten(1).all(1).tolist() == [False, True, True, False]
    assert torch.isfinite(q[[0, 3]].float()).all()
    v = lib.kv4_read(pool, torch.arange(4, device=dev), d)[1]
    assert (v != 0).flatten(1).all(1).tolist() == [True, False, False, True]


def test_append_and_attention_past_32_bit_offsets(dev):
    lib = w4()
    say("a pool of more than 4 GiB")
    d, hk, page = 128, 8, 64
    region = page * d + 8 * page
    pages = (5 << 30) // (hk * region)
    pool = torch.empty(pages, hk, region, dtype=torch.uint8, device=dev)
    pool[-2:].zero_()
    g = torch.Generator().manual_seed(5)
    t = 100
    x = torch.randn(t, 2 * hk * d, generator=g).to(torch.bfloat16)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32)
    at = torch.arange(t)
    slots = table[0].long()[at // page] * page + at % page
    lib.kv4_append(x.to(dev), pool, slots.to(dev), d)
    xs = ref.quantized(f32(x).reshape(t, 2 * hk, d), 128)
    k, v = lib.kv4_read(pool, slots.to(dev), d, dtype=torch.float32)
    assert np.array_equal(k.cpu().numpy(), xs[:, :hk]) and np.array_equal(v.cpu().numpy(), xs[:, hk:])
    q = torch.randn(1, 2 * hk, d, generator=g).to(torch.bfloat16)
    out = lib.kv4_attention(q.to(dev), pool, table.to(dev), torch.tensor([t], dtype=torch.int32, device=dev))
    want, tol = ref.attention(q, xs[:, :hk], xs[:, hk:], t, 1, True, 0, d ** -0.5)
    ref.within(out, want, tol, "far pages")


def test_rope_table_scaling(dev):
    lib = w4()
    say("rope tables")
    i = np.arange(0, 64, 2) / 64
    far = 100000
    plain = lib.rope_table(far + 1, 64, base=10000.0, device=dev)[far].cpu().double().numpy()
    angle = far * 10000.0 ** -i
    assert np.abs(plain - np.concatenate((np.cos(angle), np.sin(angle)))).max() <= 2.0 ** -24 + 1e-9
    f = 10000.0 ** -i
    turns = 4096 * f / (2 * np.pi)
    keep = np.clip((turns - 1) / 31, 0, 1)
    angle = far * f * (keep + (1 - keep) / 8)
    got = lib.rope_table(far + 1, 64, factor=8.0, original_length=4096, magnitude=1.25, device=dev)[far].cpu().double().numpy()
    assert np.abs(got - 1.25 * np.concatenate((np.cos(angle), np.sin(angle)))).max() <= 1.25 * 2.0 ** -23 + 1e-9
    got = lib.rope_table(9, 32, factor=4.0, device=dev)[8].cpu()
    assert torch.equal(got, lib.rope_table(3, 32, device=dev)[2].cpu())


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------


class Cache:
    """A pool with `lens` tokens of each request on shuffled pages, everything else NaN or random."""

    def __init__(self, dev, lens, hk, d, page, seed, spread=1.0, vsize=1.0, voutlier=0.0):
        lib = w4()
        g = torch.Generator().manual_seed(seed)
        self.page, self.hk, self.d = page, hk, d
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        self.pool = torch.empty(pages, hk, lib.kv4_pool(1, page, hk, d, device="cpu").shape[2], dtype=torch.uint8)
        self.pool.random_(0, 256, generator=g)
        self.pool[:, :, page * d:] = 255  # scales of unwritten tokens: NaN
        self.pool = self.pool.to(dev)
        order = torch.randperm(pages, generator=g)
        self.table = torch.full((len(lens), max(need + [0]) + 1), -1, dtype=torch.int32)
        self.k, self.v = [], []
        at = 0
        for i, n in enumerate(lens):
            self.table[i, :need[i]] = order[at:at + need[i]].to(torch.int32)
            at += need[i]
            x = torch.randn(n, 2, hk, d, generator=g)
            x[:, 0] *= spread
            x[:, 1] *= vsize
            if voutlier and n > 3:
                x[n // 3, 1] *= voutlier
            x = x.to(torch.bfloat16)
            if n:
                tok = torch.arange(n)
                slots = self.table[i].long()[tok // page] * page + tok % page
                lib.kv4_append(x.reshape(n, -1).to(dev), self.pool, slots.to(dev), d)
            vals = ref.quantized(f32(x), min(d, 128)) if n else np.zeros((0, 2, hk, d), np.float32)
            self.k.append(vals[:, 0])
            self.v.append(vals[:, 1])


ATT = [
    # kv lengths, query lengths (None: one each without cu_q), heads, kv_heads, dim, page, causal, window, dtype
    ([1], None, 8, 1, 256, 16, True, 0, "bf16"),
    ([0, 1, 15, 16, 17, 31, 32, 33, 47, 48, 49], None, 4, 4, 64, 16, True, 0, "f16"),
    ([127, 128, 129, 255, 256, 257, 511], None, 6, 2, 128, 48, True, 0, "bf16"),
    ([1000, 3, 2500], None, 16, 1, 64, 32, True, 0, "bf16"),
    ([1000, 0, 700], None, 40, 2, 128, 64, True, 0, "f16"),       # 20 heads share one: two row tiles
    ([5000], None, 8, 1, 256, 128, True, 0, "bf16"),
    ([900, 64, 1], None, 8, 8, 128, 16, True, 100, "bf16"),
    ([900, 64, 1], None, 8, 2, 128, 4096, False, 33, "f16"),
    ([50], [50], 8, 1, 256, 16, False, 0, "bf16"),
    ([1074], [50], 8, 1, 256, 16, False, 0, "bf16"),
    ([65, 300, 1, 0, 33], [65, 7, 1, 0, 32], 6, 2, 64, 16, True, 0, "f16"),
    ([130, 513], [129, 200], 4, 4, 128, 64, True, 0, "bf16"),
    ([130, 513], [129, 200], 3, 1, 128, 64, True, 17, "f16"),
    ([700, 40], [333, 40], 4, 1, 256, 32, False, 61, "bf16"),
    ([10, 3], [20, 3], 5, 1, 64, 16, True, 0, "bf16"),            # more queries than tokens: the first see nothing
    ([1500, 20], [260, 1], 16, 1, 64, 80, True, 300, "bf16"),     # tiles of rows that start inside a query
]


def att_id(c):
    return f"kv{'_'.join(map(str, c[0]))}-q{'_'.join(map(str, c[1])) if c[1] else '1'}-h{c[2]}_{c[3]}-d{c[4]}-p{c[5]}-{'c' if c[6] else 'b'}{c[7]}-{c[8]}"


def run_attention(dev, cache, q_lens, kv_lens, heads, causal, window, dtype, scale=None, seed=0, qsize=1.5, **more):
    lib = w4()
    g = torch.Generator().manual_seed(seed + 77)
    counts = q_lens or [1] * len(kv_lens)
    q = (qsize * torch.randn(sum(counts), heads, cache.d, generator=g)).to(dtype)
    cu = None
    if q_lens:
        cu = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device=dev)
    out = lib.kv4_attention(q.to(dev), cache.pool, cache.table.to(dev), torch.tensor(kv_lens, dtype=torch.int32, device=dev),
                            cu_q=cu, causal=causal, window=window, scale=scale, **more)
    return q, counts, out


def check_attention(cache, q, counts, kv_lens, causal, window, out, scale=None, what="", pages_there=None):
    row = 0
    for i, n in enumerate(counts):
        there = None
        if pages_there is not None:
            there = pages_there[i][np.arange(kv_lens[i]) // cache.page]
        want, tol = ref.attention(q[row:row + n], cache.k[i][:kv_lens[i]], cache.v[i][:kv_lens[i]], kv_lens[i], n, causal, window,
                                  cache.d ** -0.5 if scale is None else scale, there)
        ref.within(out[row:row + n], want, tol, f"{what} request {i}")
        row += n


@pytest.mark.parametrize("case", ATT, ids=[att_id(c) for c in ATT])
def test_attention(dev, case):
    kv, qs, h, hk, d, page, causal, window, dts = case
    say("attention", case)
    cache = Cache(dev, kv, hk, d, page, seed=sum(kv) + d)
    q, counts, out = run_attention(dev, cache, qs, kv, h, causal, window, DT[dts])
    check_attention(cache, q, counts, kv, causal, window, out, what=str(case))
    again = run_attention(dev, cache, qs, kv, h, causal, window, DT[dts])[2]
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "two runs differ"


@pytest.mark.parametrize("spread,vsize,voutlier,qsize,scale", [
    (1.0, 1e-3, 0.0, 1.5, None),     # small values: probabilities times scales below f16's normals without the reference
    (1.0, 3e4, 0.0, 1.5, None),      # large ones
    (1.0, 1.0, 3000.0, 1.5, None),   # one token's values far above the rest
    (40.0, 1.0, 0.0, 30.0, None),    # logits in the hundreds: one-hot rows
    (1.0, 1.0, 0.0, 1.5, -0.3),      # any scale
    (1e-4, 1.0, 0.0, 1e-4, 1.0),     # flat rows, queries below f16's normals
    (1.0, 1.0, 0.0, 1e5, 1e-5),      # queries above f16's range
], ids=["small_v", "large_v", "outlier_v", "one_hot", "negative_scale", "flat", "large_q"])
@pytest.mark.parametrize("qs", [None, [70, 130]], ids=["decode", "chunk"])
def test_attention_ranges(dev, spread, vsize, voutlier, qsize, scale, qs):
    say("attention ranges", spread, vsize, voutlier, qsize, scale, qs)
    kv = [333, 1200]
    cache = Cache(dev, kv, 2, 128, 32, seed=9, spread=spread, vsize=vsize, voutlier=voutlier)
    q, counts, out = run_attention(dev, cache, qs, kv, 8, True, 0, torch.bfloat16, scale=scale, qsize=qsize)
    check_attention(cache, q, counts, kv, True, 0, out, scale=scale)


@pytest.mark.parametrize("qs", [None, [90, 5]], ids=["decode", "chunk"])
def test_attention_pages_outside_the_pool_are_not_seen(dev, qs):
    say("bad pages", qs)
    kv = [400, 95]
    cache = Cache(dev, kv, 2, 64, 32, seed=3)
    there = [np.ones(64, bool), np.ones(64, bool)]
    for i, p, bad in ((0, 2, -1), (0, 7, cache.pool.shape[0]), (1, 0, 2 ** 31 - 1), (1, 2, -2 ** 31)):
        cache.table[i, p] = bad
        there[i][p] = False
    q, counts, out = run_attention(dev, cache, qs, kv, 4, True, 0, torch.float16)
    check_attention(cache, q, counts, kv, True, 0, out, what="bad pages", pages_there=there)


def test_attention_lengths_beyond_the_table(dev):
    say("lengths beyond the table, and below zero")
    kv = [64, 40]
    cache = Cache(dev, kv, 1, 64, 16, seed=4)
    cache.table = cache.table[:, :4].contiguous()
    q, counts, out = run_attention(dev, cache, None, [1000, -5], 2, True, 0, torch.bfloat16)
    check_attention(cache, q[:1], [1], [64], False, 0, out[:1])
    assert not out[1].any()


def test_attention_strided_rows_and_tables(dev):
    lib = w4()
    say("strided q and table, out given")
    kv = [77, 300, 12]
    cache = Cache(dev, kv, 2, 128, 16, seed=6)
    q, counts, out = run_attention(dev, cache, None, kv, 4, True, 0, torch.bfloat16)
    wide = torch.full((3, 4 * 128 + 72), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, 8:8 + 512] = q.view(3, 512).to(dev)
    table = torch.full((3, cache.table.shape[1] + 5), 2 ** 30, dtype=torch.int32, device=dev)
    table[:, :cache.table.shape[1]] = cache.table.to(dev)
    given = torch.full((3, 4, 128), float("nan"), dtype=torch.bfloat16, device=dev)
    got = lib.kv4_attention(wide[:, 8:520].unflatten(1, (4, 128)), cache.pool, table[:, :cache.table.shape[1]],
                            torch.tensor(kv, dtype=torch.int32, device=dev), out=given)
    assert got is given and torch.equal(got, out)


def test_attention_no_query_tokens(dev):
    lib = w4()
    say("no tokens")
    pool = lib.kv4_pool(1, 16, 1, 64, device=dev)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    out = lib.kv4_attention(torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=dev), pool, z(2, 1), z(2), cu_q=z(3))
    assert out.shape == (0, 2, 64)
    q = lib.kv4_append(torch.zeros(0, 4 * 64, dtype=torch.bfloat16, device=dev), pool, torch.zeros(0, dtype=torch.int64, device=dev), 64)
    assert q.shape == (0, 2, 64)


@pytest.mark.parametrize("qs", [None, [40, 200]], ids=["decode", "chunk"])
def test_attention_on_another_stream_and_in_a_graph(dev, qs):
    lib = w4()
    say("stream and graph", qs)
    kv = [3000, 1500]
    cache = Cache(dev, kv, 2, 128, 32, seed=8)
    q, counts, want = run_attention(dev, cache, qs, kv, 8, True, 0, torch.bfloat16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    qd, table, lens = q.to(dev), cache.table.to(dev), torch.tensor(kv, dtype=torch.int32, device=dev)
    cu = None if qs is None else torch.tensor([0, qs[0], sum(qs)], dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = lib.kv4_attention(qd, cache.pool, table, lens, cu_q=cu)
    side.synchronize()
    assert torch.equal(got, want)
    need = lib.kv4_attention_workspace_bytes(q.shape[0], 2, 8, 2, 128, table.shape[1], 32, ragged=qs is not None)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
    out = torch.empty_like(qd)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lib.kv4_attention(qd, cache.pool, table, lens, cu_q=cu, out=out, workspace=ws)
    for rep in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {rep}"
        assert torch.equal(lib.kv4_attention(qd, cache.pool, table, lens, cu_q=cu), want)
    # other lengths in the same graph: the plan does not depend on them
    lens.copy_(torch.tensor([1100, 1499], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check_attention(cache, q, counts, [1100, 1499], True, 0, out, what="replay with other lengths")
    assert not ws[:min(need, 1 << 20)].any(), "the workspace's header is not zero"


def test_attention_of_rows_of_256_channels_in_a_graph(dev):
    """Row tiles of 256 channels need more than 64 KB of LDS, which is asked for per launch: under capture too."""
    lib = w4()
    say("row tiles of 256 channels in a graph")
    kv, qs = [700, 900], [600, 450]
    cache = Cache(dev, kv, 1, 256, 16, seed=12)
    q, counts, want = run_attention(dev, cache, qs, kv, 8, True, 0, torch.bfloat16)
    check_attention(cache, q, counts, kv, True, 0, want, what="eager")
    qd, table, lens = q.to(dev), cache.table.to(dev), torch.tensor(kv, dtype=torch.int32, device=dev)
    cu = torch.tensor([0, qs[0], sum(qs)], dtype=torch.int32, device=dev)
    need = lib.kv4_attention_workspace_bytes(q.shape[0], 2, 8, 1, 256, table.shape[1], 16, ragged=True)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=dev)
    out = torch.empty_like(qd)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lib.kv4_attention(qd, cache.pool, table, lens, cu_q=cu, out=out, workspace=ws)
    for rep in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {rep}"


@pytest.mark.parametrize("d,hk,share", [(64, 8, 8), (128, 4, 16), (256, 2, 16)], ids=["d64", "d128", "d256"])
def test_attention_row_tiles(dev, d, hk, share):
    """Tiles of 64 rows: prompts whole and in pieces, with windows, without a mask, on bad pages, split and unsplit (rows
    and tokens enough that every call takes them)."""
    say("row tiles", d, hk, share)
    for kv, qs, causal, window, page in (([700, 33, 1300], [700, 33, 140], True, 0, 48), ([900, 1000], [333, 500], True, 130, 16),
                                         ([2500], [190], False, 0, 64), ([1200, 640], [320, 640], False, 77, 32)):
        cache = Cache(dev, kv, hk, d, page, seed=sum(kv) + d + window)
        there = [np.ones(cache.table.shape[1], bool) for _ in kv]
        cache.table[0, 3] = -7
        there[0][3] = False
        q, counts, out = run_attention(dev, cache, qs, kv, share * hk, causal, window, torch.bfloat16)
        check_attention(cache, q, counts, kv, causal, window, out, what=f"{kv} {qs}", pages_there=there)
        again = run_attention(dev, cache, qs, kv, share * hk, causal, window, torch.bfloat16)[2]
        assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "two runs differ"
