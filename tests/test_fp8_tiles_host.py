"""That the sizes of test_fp8_tiles_gpu reach every kernel of the 8-bit float layer, cut along k and whole (no GPU), and what
the call that tells says of sizes that there are none of."""
import weight_only_int4_rtn_amd as w4

# rows, columns, k: each tile shape with a ragged end in both directions, one group to 128 (more than the 64 whose scales a lane
# holds at a time), fewer groups than a ring has buffers, uneven parts of k
SIZES = [
    (1, 40, 2048), (3, 2100, 16384), (16, 300, 8192), (9, 8197, 384),
    (17, 101, 128), (33, 130, 256), (129, 257, 512), (50, 130, 1152), (2300, 257, 256), (33, 100, 8192), (130, 2101, 4096), (520, 301, 8192),
    (65, 12301, 128), (65, 12301, 256), (1025, 1003, 640), (300, 6301, 8192), (3900, 257, 4096), (33, 2101, 16384), (300, 1301, 8192), (385, 516, 4096),
    (129, 12301, 128), (200, 8197, 256), (130, 12301, 384), (130, 12301, 640), (2050, 8195, 640), (65, 6301, 4096), (700, 1003, 8192), (2050, 257, 16384),
    (520, 8197, 384), (4000, 1301, 512), (700, 6301, 4096), (129, 6301, 8192), (1025, 1301, 16384), (200, 8197, 16384),
    (1025, 12301, 1152), (2050, 4101, 2048), (4000, 2101, 4096), (131, 12301, 16384), (700, 6301, 16384), (2050, 4101, 16384),
]
TILES = [(16, 16), (32, 128), (64, 128), (128, 128), (128, 256), (256, 256)]


def test_sizes_reach_every_kernel():
    reached = {(rows, columns, splits > 1) for rows, columns, splits in (w4.linear_fp8_tile(*size) for size in SIZES)}
    missing = [(*tile, cut) for tile in TILES for cut in (False, True) if (*tile, cut) not in reached]
    assert not missing, f"no size of the list takes (rows, columns, cut along k): {missing}"


def test_ragged_both_ways():
    """Each shape has a size whose last tile is ragged along rows and columns, with more than one tile of rows if it has many."""
    for tile in TILES:
        sizes = [s for s in SIZES if w4.linear_fp8_tile(*s)[:2] == tile]
        assert any(s[0] % tile[0] and s[1] % tile[1] for s in sizes), tile
        assert tile[0] == 16 or any(s[0] > tile[0] and s[0] % tile[0] and s[1] > tile[1] for s in sizes), tile


def test_no_such_sizes():
    for size in ((0, 100, 256), (10, 0, 256), (10, 10, 200), (-1, 10, 128), (10, -5, 128), (10, 10, 0), (1 << 25, 10, 128), (10, 10, 1 << 23)):
        assert w4.linear_fp8_tile(*size) == (0, 0, 0), size
    from weight_only_int4_rtn_amd import _fp8
    assert _fp8._lib().fp8_linear_tile(100, 100, 256, None, None) == w4.linear_fp8_tile(100, 100, 256)[0]
