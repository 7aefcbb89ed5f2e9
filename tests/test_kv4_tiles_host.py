"""Which kernel a call of kv4_attention takes (kv4_attention_tile_rows), from sizes alone."""
import weight_only_int4_rtn_amd as w4

f = w4.kv4_attention_tile_rows


def test_decoding_takes_tiles_of_16():
    for heads, kv_heads, dim, batch in ((8, 1, 256, 1), (32, 8, 128, 64), (16, 16, 64, 500)):
        assert f(batch, batch, heads, kv_heads, dim, 8192, 16) == 16


def test_prompts_take_tiles_of_64():
    assert f(4096, 1, 32, 8, 128, 64, 64, ragged=True) == 64
    assert f(2000, 12, 16, 16, 64, 94, 32, ragged=True, window=1024) == 64
    assert f(50, 1, 8, 1, 256, 67, 16, ragged=True, causal=False) == 16


def test_invalid_sizes():
    for bad in ((0, 0, 8, 1, 256, 4, 16), (4, 3, 8, 1, 256, 4, 16), (4, 4, 8, 3, 256, 4, 16), (4, 4, 8, 1, 96, 4, 16),
                (4, 4, 8, 1, 64, 0, 16), (4, 4, 8, 1, 64, 4, 24)):
        assert f(*bad) == 0
