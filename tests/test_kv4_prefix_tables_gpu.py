"""Attention on shared prefixes whose block tables have room, as those of captured steps do: the same answers, and parts
that follow the lengths and not the table's width."""
import pytest
import torch

from tests.gpu_util import require_gpu, say
from tests.test_kv4_prefix_gpu import Batch, ints, w4

pytestmark = pytest.mark.gpu

HEADER = 1 << 20  # bytes of a workspace that are zero before and after a call


@pytest.fixture(scope="module")
def dev():
    return require_gpu()


def wider(table, width):
    """The table in rows of `width` pages; what lies behind its own is not in use (garbage)."""
    out = torch.full((table.shape[0], width), 2 ** 30, dtype=torch.int32, device=table.device)
    out[:, :table.shape[1]] = table
    return out


# route (rows of a prefix tile, 0: one launch), prefixes, own lengths, cu_groups, query lengths, heads, kv_heads, dim, page
SHAPES = [
    (0, [800], [3, 60], [0, 2], None, 8, 1, 256, 16),
    (0, [900, 300], [20, 9, 33], [0, 1, 3], [1, 9, 4], 4, 2, 64, 16),
    (16, [3000], [5, 0, 40, 17] * 15, [0, 60], None, 8, 8, 64, 16),
    (16, [1300, 2000, 0], [5, 0, 40, 17] * 12, [0, 20, 45, 48], None, 16, 8, 128, 32),
    (64, [1600], [300, 500, 260], [0, 3], [300, 450, 256], 16, 4, 128, 32),
]


def call(b, times, own_times=1):
    """A call on tables `times` as wide: (output, words of the workspace behind its header that it wrote, rows of a tile)."""
    lib = w4()
    args, kw = b.args()
    q, pool, table, lens, own, own_lens = args
    table, own = wider(table, times * table.shape[1]), wider(own, own_times * own.shape[1])
    sizes = (q.shape[0], own.shape[0], table.shape[0], q.shape[1], b.cache.hk, b.cache.d, table.shape[1], own.shape[1], b.cache.page)
    need = lib.kv4_prefix_attention_workspace_bytes(*sizes, ragged=b.q_lens is not None)
    ws = torch.full((max(need, HEADER),), 255, dtype=torch.uint8, device=b.dev)
    ws[:HEADER] = 0
    out = lib.kv4_prefix_attention(q, pool, table, lens, own, own_lens, **kw, workspace=ws)
    assert not ws[:HEADER].any()
    wrote = int((ws[HEADER:need].view(torch.int32) != -1).sum()) if need > HEADER else 0
    return out, wrote, lib.kv4_prefix_attention_tile_rows(*sizes, ragged=b.q_lens is not None)


@pytest.mark.parametrize("shape", SHAPES, ids=[f"t{s[0]}-d{s[7]}-{len(s[1])}x{len(s[2])}" for s in SHAPES])
def test_tables_with_room(dev, shape):
    rows, prefix, own, first, qs, heads, hk, d, page = shape
    b = Batch(dev, prefix, own, first, heads, hk, d, page, torch.bfloat16, qs)
    say("tables with room", shape)
    out, exact, route = call(b, 1)
    assert route == rows and exact > 0, "the case is cut into parts"
    b.check(out, what="exact")
    for times, own_times in ((4, 1), (8, 1), (8, 4)):
        out, wrote, route = call(b, times, own_times)
        assert route == rows
        # what parts leave in the workspace grows with their number (own tokens of a second launch are cut by their table)
        if own_times == 1 or rows == 0:
            assert wrote >= exact, f"{wrote} words of parts in a table {times} times as wide, {exact} in the exact one"
        b.check(out, what=f"{times} times as wide")


def test_parts_in_one_graph_follow_lengths(dev):
    """One graph on a table of 16384 tokens, replayed for prefixes from none to all of it."""
    lib = w4()
    b = Batch(dev, [16000], [20, 3, 50] * 8, [0, 24], 8, 8, 64, 16, torch.bfloat16)
    say("one graph, many lengths")
    b.takes(16)
    args, kw = b.args()
    out = torch.empty_like(args[0])
    need = lib.kv4_prefix_attention_workspace_bytes(24, 24, 1, 8, 8, 64, args[2].shape[1], args[4].shape[1], 16)
    ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    lib.kv4_prefix_attention(*args, **kw, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        lib.kv4_prefix_attention(*args, **kw, out=out, workspace=ws)
    for n in (16000, 0, 1, 127, 128, 129, 700, 5001, 16000):
        args[3].copy_(ints([n], dev))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        b.check(out, prefix=[n], what=f"prefix of {n}")
        assert torch.equal(out, lib.kv4_prefix_attention(*args, **kw))


# route, requests of each group, heads, kv_heads, dim, table width of a prefix in pages of 16 (so wide that tall tiles come into question)
GROUPS = [
    (0, [1] * 40, 32, 8, 64, 1400), (0, [1] * 24, 16, 2, 256, 4200),
    (16, [2] * 20, 32, 8, 128, 1300), (16, [1, 2, 3, 0, 4] * 6, 32, 8, 64, 1000), (16, [8] * 6, 16, 8, 256, 2100),
    (64, [12] * 5, 32, 4, 128, 900), (64, [60, 1, 1, 40], 16, 4, 64, 1000),
]


@pytest.mark.parametrize("rows,each,heads,hk,d,width", GROUPS, ids=[f"t{c[0]}-{len(c[1])}x{max(c[1])}-d{c[4]}" for c in GROUPS])
def test_many_groups(dev, rows, each, heads, hk, d, width):
    """Groups of one request, of few and of many, on long tables."""
    n, batch = len(each), sum(each)
    b = Batch(dev, [(97 * i + 61) % 400 for i in range(n)], [(31 * i) % 70 for i in range(batch)], [sum(each[:i]) for i in range(n + 1)],
              heads, hk, d, 16, torch.float16)
    say("many groups", rows, each, heads, hk, d)
    out, _, route = call(b, -(-width // b.cache.table.shape[1]))
    assert route == rows
    b.check(out, what="many groups")
