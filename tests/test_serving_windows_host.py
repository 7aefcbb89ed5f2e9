"""Windows longer than any cache: the workspace asked for, the check against it
and the launch agree on them (no GPU: every call here returns before a launch)."""
import pytest
import torch

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


@pytest.mark.parametrize("window", [1 << 63, 1 << 64, (1 << 64) + 5, 1 << 200])
def test_a_window_past_64_bits_does_not_wrap(window, monkeypatch):
    """In ctypes 2^64 + 5 is 5: the binding hands the library the longest window instead."""
    f = w4.kv4_attention_workspace_bytes
    assert f(1, 1, 8, 1, 128, 8192, 16, window=window) == f(1, 1, 8, 1, 128, 8192, 16)
    pool = w4.kv4_pool(2, 16, 2, 64, device="cpu")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    given = []

    class Library:
        def kv4_attention(self, *args):
            given.append(args)
            return B.OK

    monkeypatch.setattr(S, "_lib", lambda: Library())
    monkeypatch.setattr(S, "_attention_need", lambda *sizes: 0)
    monkeypatch.setattr(S, "_device_index", lambda *tensors: 0)
    monkeypatch.setattr(S, "_raw_stream", lambda index: 0)
    S._attention_plan.cache_clear()
    try:
        w4.kv4_attention(torch.zeros(3, 4, 64, dtype=torch.bfloat16), pool, i32(3, 2), i32(3), window=window)
    finally:
        S._attention_plan.cache_clear()
    assert given[0][17] == (1 << 63) - 1


def test_a_window_is_a_whole_number():
    for bad in (-1, 1.5, None):
        with pytest.raises(ValueError, match="window"):
            w4.kv4_attention_workspace_bytes(1, 1, 8, 1, 128, 8192, 16, window=bad)
