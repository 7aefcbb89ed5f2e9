"""Which kernels attention on shared prefixes takes (no GPU): tiles of 64 rows only where groups fill them, one launch where
requests share little."""
import pytest

import weight_only_int4_rtn_amd as w4


def route(groups, each, heads, kv_heads, dim, tokens, own=64, page=64, q=1):
    """Rows of a prefix tile, 0 for one launch: `groups` of `each` requests with q query tokens on tables of `tokens`."""
    batch = groups * each
    return w4.kv4_prefix_attention_tile_rows(batch * q, batch, groups, heads, kv_heads, dim, -(-tokens // page), -(-own // page), page,
                                             ragged=q > 1)


@pytest.mark.parametrize("groups,each,heads,kv_heads,tokens,rows", [
    (64, 2, 32, 8, 8192, 16), (64, 2, 32, 8, 16384, 16), (64, 4, 32, 8, 16384, 16), (64, 8, 32, 8, 16384, 16),  # 8, 16, 32 rows a group
    (16, 16, 16, 16, 25600, 16), (64, 3, 64, 8, 32768, 16),
    (64, 16, 32, 8, 8192, 64), (16, 12, 32, 4, 6656, 64), (4, 48, 32, 8, 32768, 64), (1, 64, 32, 8, 16384, 64),  # 64 rows and more
])
def test_tall_tiles_need_groups_that_fill_them(groups, each, heads, kv_heads, tokens, rows):
    assert route(groups, each, heads, kv_heads, 128, tokens) == rows


@pytest.mark.parametrize("tokens", [64, 8192, 16384, 131072])
@pytest.mark.parametrize("groups,dim", [(1, 64), (64, 128), (256, 256)])
def test_one_request_a_group_takes_one_launch(groups, dim, tokens):
    assert route(groups, 1, 32, 8, dim, tokens) == 0


# measured both ways (the comment in plan_kv4_prefix): requests, heads, key heads, dim, tokens of the prefix, whether one launch was faster
MEASURED = [
    (8, 8, 1, 64, 1000, True), (8, 16, 16, 64, 1000, True), (8, 16, 16, 64, 4000, False), (32, 32, 8, 64, 1000, True), (64, 32, 8, 64, 1000, False),
    (20, 16, 2, 64, 12000, True), (4, 32, 8, 128, 1000, True), (150, 16, 2, 128, 1000, True), (4, 8, 8, 128, 8000, True), (32, 8, 8, 128, 1000, False),
    (64, 32, 8, 128, 1000, True), (64, 8, 1, 128, 16000, True), (2, 8, 1, 256, 800, True), (64, 8, 1, 256, 8000, True), (40, 16, 4, 256, 2500, False),
    (64, 4, 4, 256, 2000, False),
]


@pytest.mark.parametrize("requests,heads,kv_heads,dim,tokens,one", MEASURED)
def test_the_faster_of_one_launch_and_two(requests, heads, kv_heads, dim, tokens, one):
    assert (route(1, requests, heads, kv_heads, dim, tokens) == 0) == one
