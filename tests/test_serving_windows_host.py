"""Windows longer than any cache: the workspace asked for, the check against it
and the launch agree on them (no GPU: every call here returns before a launch)."""
import pytest

import weight_only_int4_rtn_amd as w4
from weight_only_int4_rtn_amd import _binding as B
from weight_only_int4_rtn_amd import _serving as S

A, GB = 1 << 20, 1 << 30
WINDOWS = [1 << 17, (1 << 17) - 16, 1 << 28, 1 << 31, 1 << 61, 1 << 62, (1 << 63) - 65, (1 << 63) - 1]
SHAPES = [(1, 1, False), (7, 7, False), (512, 1, True), (3000, 5, True)]


def attend(window, causal, tokens, batch, ragged, ws, ws_bytes):
    """8192 pages of 16 tokens a request, 8 query heads on one key head of 128 channels, fake addresses."""
    return S._lib().kv4_attention(A, B.BF16, tokens, 8 * 128, 8, 1, 128, A + GB, 8192, 16, A + 2 * GB, 8192, 8192, A + 3 * GB,
                                  A + 6 * GB if ragged else None, batch, int(causal), window, 0.1, A + 4 * GB, 8 * 128, ws,
                                  ws_bytes, None)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tokens,batch,ragged", SHAPES)
@pytest.mark.parametrize("window", WINDOWS)
def test_a_window_beyond_the_cache_is_none(window, tokens, batch, ragged, causal):
    need = w4.kv4_attention_workspace_bytes(tokens, batch, 8, 1, 128, 8192, 16, ragged=ragged, causal=causal)
    assert need > 1 << 20
    assert w4.kv4_attention_workspace_bytes(tokens, batch, 8, 1, 128, 8192, 16, ragged=ragged, causal=causal, window=window) == need
    assert attend(window, causal, tokens, batch, ragged, None, 0) == B.EWORKSPACE
    assert attend(window, causal, tokens, batch, ragged, A + 5 * GB, need - 1) == B.EWORKSPACE


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("tokens,batch,ragged", SHAPES)
def test_a_shorter_window_needs_no_more(tokens, batch, ragged, causal):
    last = 0
    for window in (1, 64, 1000, 30000, 1 << 16, 1 << 17, 1 << 40):
        need = w4.kv4_attention_workspace_bytes(tokens, batch, 8, 1, 128, 8192, 16, ragged=ragged, causal=causal, window=window)
        assert need <= w4.kv4_attention_workspace_bytes(tokens, batch, 8, 1, 128, 8192, 16, ragged=ragged, causal=causal)
        last = need
    assert last > 1 << 20
