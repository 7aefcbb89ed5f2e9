"""The 8-bit float layer's choice of tile and parts at sizes where every choice was measured (no GPU)."""
import pytest

import weight_only_int4_rtn_amd as w4

# rows of x, columns of y, k -> tiles and parts that were within 6 % of the best measured
NEAR_BEST = {
    (17, 2560, 2048): [(32, 128, 1), (32, 128, 2), (32, 128, 3), (32, 128, 4), (64, 128, 1), (64, 128, 3), (64, 128, 4)],
    (64, 2048, 16384): [(32, 128, 8), (64, 128, 10), (64, 128, 12), (64, 128, 16), (128, 128, 16)],
    (128, 255, 1920): [(32, 128, 2), (32, 128, 3), (32, 128, 4), (32, 128, 5)],
    (512, 2048, 16384): [(128, 128, 4), (128, 128, 6), (128, 256, 6), (128, 256, 8)],
    (512, 23345, 15872): [(256, 256, 1)],
    (1024, 2048, 16384): [(128, 128, 2), (128, 256, 3), (128, 256, 4)],
    (1024, 2560, 2048): [(128, 128, 1)],
    (1500, 27594, 512): [(128, 128, 1)],
    (3000, 13038, 256): [(128, 128, 1)],
    (4096, 32768, 2048): [(256, 256, 1)],
}


@pytest.mark.parametrize("size", NEAR_BEST, ids=["x".join(map(str, s)) for s in NEAR_BEST])
def test_plan_is_near_the_best(size):
    assert w4.linear_fp8_tile(*size) in NEAR_BEST[size]


@pytest.mark.parametrize("m,n,k", [(1, 64, 16384), (12, 64, 16384), (1, 16, 131072), (3, 2048, 16384)])
def test_few_rows_leave_one_vector_a_lane_and_part(m, n, k):
    """Parts of the kernel for few rows meet in 64 vectors of 16 bytes a tile and part, behind the header."""
    rows, columns, splits = w4.linear_fp8_tile(m, n, k)
    assert (rows, columns) == (16, 16) and splits > 1
    assert w4.linear_fp8_workspace_bytes(m, n, k, codes=True) == (1 << 20) + -(-n // 16) * splits * 64 * 16
