"""Refusals of the serving operators, from metadata alone (no GPU: every call
here returns before a launch), and their sizes."""
import ctypes

import pytest
import torch

import weight_only_int4_rtn_amd as w4
from weight_only_int4_rtn_amd import _binding as B
from weight_only_int4_rtn_amd import _serving as S

A = 1 << 20  # a 16-byte aligned fake device address (never dereferenced)
GB = 1 << 30


@pytest.fixture(scope="module")
def lib():
    return S._lib()


def test_pool_bytes(lib):
    assert lib.kv4_pool_bytes(1, 16, 1, 64) == 16 * 64 + 8 * 16
    assert lib.kv4_pool_bytes(10, 64, 8, 128) == 10 * 8 * (64 * 128 + 8 * 64)
    assert lib.kv4_pool_bytes(3, 48, 2, 256) == 3 * 2 * (48 * 256 + 16 * 48)
    for bad in ((0, 16, 1, 64), (1, 8, 1, 64), (1, 24, 1, 64), (1, 4112, 1, 64), (1, 16, 0, 64), (1, 16, 1025, 64),
                (1, 16, 1, 96), (1, 16, 1, 512), (-1, 16, 1, 64), (1 << 31, 16, 1, 64)):
        assert lib.kv4_pool_bytes(*bad) == 0, bad
    pool = w4.kv4_pool(3, 48, 2, 256, device="cpu")
    assert pool.numel() == lib.kv4_pool_bytes(3, 48, 2, 256) and w4.kv4_page_size(pool, 256) == 48
    with pytest.raises(ValueError, match="no such cache"):
        w4.kv4_pool(3, 40, 2, 256, device="cpu")
    for dim in (64, 128, 96):
        with pytest.raises(ValueError):
            w4.kv4_page_size(pool[:, :, :-16].contiguous(), dim)


def append(lib, **kw):
    d = dict(qkv=A, dtype=B.BF16, tokens=4, ld=6 * 128, heads=4, kv_heads=1, dim=128, rope=A + GB, rope_len=100, rot=128,
             inter=0, positions=A + 2 * GB, slots=A + 3 * GB, pool=A + 4 * GB, pages=2, page=16, q_out=A + 5 * GB)
    d.update(kw)
    return lib.kv4_append(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0), B.OK),
    (dict(tokens=0, qkv=None, slots=None, pool=None, q_out=None), B.OK),
    (dict(dtype=B.F32), B.EUNSUPPORTED), (dict(dtype=9), B.EUNSUPPORTED),
    (dict(tokens=-1), B.EINVAL), (dict(tokens=(1 << 24) + 1), B.EINVAL),
    (dict(ld=6 * 128 - 8), B.EINVAL), (dict(ld=6 * 128 + 4), B.EINVAL), (dict(ld=(1 << 24) + 8), B.EINVAL),
    (dict(heads=-1), B.EINVAL), (dict(kv_heads=0), B.EINVAL), (dict(dim=96), B.EINVAL),
    (dict(rope=None), B.EINVAL), (dict(positions=None), B.EINVAL),
    (dict(rot=0), B.EINVAL), (dict(rot=24), B.EINVAL), (dict(rot=144), B.EINVAL), (dict(rope_len=0), B.EINVAL),
    (dict(page=24), B.EINVAL), (dict(pages=0), B.EINVAL),
    (dict(qkv=None), B.EINVAL), (dict(slots=None), B.EINVAL), (dict(pool=None), B.EINVAL), (dict(q_out=None), B.EINVAL),
    (dict(qkv=A + 8), B.EINVAL), (dict(slots=A + 4), B.EINVAL), (dict(pool=A + 4 * GB + 8), B.EINVAL),
    (dict(q_out=A + 2), B.EINVAL), (dict(rope=A + GB + 2), B.EINVAL),
    (dict(q_out=A + 16), B.EINVAL), (dict(pool=A), B.EINVAL), (dict(q_out=A + 4 * GB), B.EINVAL),
    (dict(slots=A + 4 * GB + 8), B.EINVAL), (dict(positions=A + 5 * GB), B.EINVAL),
])
def test_append_status(lib, kw, status):
    assert append(lib, **kw) == status


def test_read_status(lib):
    def read(**kw):
        d = dict(pool=A, pages=2, page=16, kv_heads=1, dim=128, slots=A + GB, tokens=4, dtype=B.BF16, k=A + 2 * GB, v=A + 3 * GB)
        d.update(kw)
        return lib.kv4_read(*d.values(), None)
    assert read(tokens=0) == B.OK
    assert read(dtype=7) == B.EUNSUPPORTED
    for kw in (dict(tokens=-1), dict(dim=32), dict(page=0), dict(pool=None), dict(slots=None), dict(k=None), dict(v=None),
               dict(k=A + 2), dict(slots=A + 4), dict(v=A + 2 * GB), dict(k=A + 16), dict(v=A + GB - 16)):
        assert read(**kw) == B.EINVAL, kw


def attend(lib, **kw):
    d = dict(q=A, dtype=B.F16, tokens=4, ldq=512, heads=4, kv_heads=1, dim=128, pool=A + GB, pages=8, page=16, table=A + 2 * GB,
             width=4, ldt=4, lens=A + 3 * GB, cu=None, batch=4, causal=1, window=0, scale=0.1, out=A + 4 * GB, ldo=512,
             ws=A + 5 * GB, ws_bytes=GB)
    d.update(kw)
    return lib.kv4_attention(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0, batch=0), B.OK), (dict(tokens=0, cu=A + 6 * GB), B.OK),
    (dict(dtype=B.F32), B.EUNSUPPORTED),
    (dict(tokens=3), B.EINVAL), (dict(batch=0, cu=A + 6 * GB), B.EINVAL), (dict(tokens=-1, batch=-1), B.EINVAL),
    (dict(heads=0), B.EINVAL), (dict(heads=3, kv_heads=2), B.EINVAL), (dict(heads=1028), B.EINVAL),
    (dict(ldq=504), B.EINVAL), (dict(ldq=516), B.EINVAL), (dict(ldo=508), B.EINVAL), (dict(ldt=3), B.EINVAL),
    (dict(dim=80), B.EINVAL), (dict(page=17), B.EINVAL), (dict(pages=0), B.EINVAL),
    (dict(width=0), B.EINVAL), (dict(width=1 << 24, ldt=1 << 24), B.EINVAL),
    (dict(window=-1), B.EINVAL), (dict(scale=float("nan")), B.EINVAL), (dict(scale=float("inf")), B.EINVAL),
    (dict(q=None), B.EINVAL), (dict(pool=None), B.EINVAL), (dict(table=None), B.EINVAL), (dict(lens=None), B.EINVAL),
    (dict(out=None), B.EINVAL), (dict(q=A + 8), B.EINVAL), (dict(out=A + 4 * GB + 8), B.EINVAL), (dict(table=A + 2), B.EINVAL),
    (dict(out=A), B.EINVAL), (dict(out=A + GB + 64), B.EINVAL), (dict(out=A + 2 * GB), B.EINVAL), (dict(out=A + 3 * GB), B.EINVAL),
    (dict(width=4000, ldt=4000, ws=None), B.EWORKSPACE), (dict(width=4000, ldt=4000, ws_bytes=1 << 20), B.EWORKSPACE),
    (dict(width=4000, ldt=4000, ws=A + 5 * GB + 4), B.EINVAL), (dict(width=4000, ldt=4000, ws=A + 4 * GB), B.EINVAL),
    (dict(width=4000, ldt=4000, ws=A), B.EINVAL), (dict(width=4000, ldt=4000, ws=A + GB), B.EINVAL),
])
def test_attention_status(lib, kw, status):
    assert attend(lib, **kw) == status


def test_attention_workspace(lib):
    f = w4.kv4_attention_workspace_bytes
    assert f(0, 0, 4, 1, 128, 10, 16) == 0
    assert f(4, 4, 4, 3, 128, 10, 16) == 0 and f(4, 3, 4, 1, 128, 10, 16) == 0 and f(4, 4, 4, 1, 100, 10, 16) == 0
    assert f(1, 1, 8, 1, 128, 1, 16) == 0  # a single split
    # long caches split; the header (1 MiB) comes first; nothing but sizes goes in
    assert f(1, 1, 8, 1, 128, 8192, 16) > 1 << 20
    assert f(1, 1, 8, 1, 128, 8192, 16, window=64) < f(1, 1, 8, 1, 128, 8192, 16)


def lora(lib, **kw):
    d = dict(x=A, dtype=B.BF16, m=4, k=256, ldx=256, a=A + GB, b=A + 2 * GB, adapters=2, rank=16, n=100, index=A + 3 * GB,
             scales=A + 4 * GB, y=A + 5 * GB, ldy=100, out=A + 6 * GB, ldo=100, ws=A + 7 * GB, ws_bytes=GB)
    d.update(kw)
    return lib.lora_add(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=0), B.OK), (dict(n=0, ldy=0, ldo=0), B.OK), (dict(m=0, x=None, a=None, b=None, index=None, y=None, out=None), B.OK),
    (dict(dtype=B.F32), B.EUNSUPPORTED),
    (dict(m=-1), B.EINVAL), (dict(k=0), B.EINVAL), (dict(k=252), B.EINVAL), (dict(ldx=248), B.EINVAL), (dict(ldx=260), B.EINVAL),
    (dict(ldy=99), B.EINVAL), (dict(ldo=99), B.EINVAL), (dict(adapters=0), B.EINVAL), (dict(rank=0), B.EINVAL),
    (dict(rank=12), B.EINVAL), (dict(rank=136), B.EINVAL),
    (dict(x=None), B.EINVAL), (dict(a=None), B.EINVAL), (dict(b=None), B.EINVAL), (dict(index=None), B.EINVAL),
    (dict(y=None), B.EINVAL), (dict(out=None), B.EINVAL), (dict(x=A + 8), B.EINVAL), (dict(a=A + GB + 8), B.EINVAL),
    (dict(b=A + 2 * GB + 2), B.EINVAL), (dict(y=A + 5 * GB + 1), B.EINVAL), (dict(index=A + 2), B.EINVAL),
    (dict(out=A + 5 * GB + 2), B.EINVAL), (dict(out=A + 5 * GB, ldo=104), B.EINVAL), (dict(out=A), B.EINVAL),
    (dict(out=A + GB), B.EINVAL), (dict(out=A + 2 * GB), B.EINVAL), (dict(out=A + 3 * GB), B.EINVAL), (dict(out=A + 4 * GB), B.EINVAL),
    (dict(ws=None), B.EWORKSPACE), (dict(ws_bytes=1 << 20), B.EWORKSPACE), (dict(ws=A + 7 * GB + 4), B.EINVAL),
    (dict(ws=A + 6 * GB), B.EINVAL), (dict(ws=A), B.EINVAL), (dict(ws=A + 5 * GB), B.EINVAL),
])
def test_lora_status(lib, kw, status):
    assert lora(lib, **kw) == status


def test_lora_workspace(lib):
    f = w4.lora_add_workspace_bytes
    assert f(4, 100, 256, 2, 16) >= (1 << 20) + 4 * 16 * 4
    for bad in ((0, 100, 256, 2, 16), (4, 0, 256, 2, 16), (4, 100, 250, 2, 16), (4, 100, 256, 0, 16), (4, 100, 256, 2, 12),
                (4, 100, 256, 2, 136)):
        assert f(*bad) == 0


def test_size_limits(lib):
    """Sizes whose launches or offsets would not fit are refused, the largest that do are not."""
    assert lib.kv4_pool_bytes(1 << 21, 64, 8, 128) == (1 << 21) * 8 * 64 * 136  # 136 GiB
    assert lib.kv4_pool_bytes(1 << 22, 64, 8, 128) == 0                         # 272 GiB
    assert append(lib, tokens=0) == B.OK and append(lib, tokens=(1 << 23) + 1) == B.EINVAL
    big = dict(table=A + 2 * GB, width=4, ldt=4, cu=A + 6 * GB)
    assert attend(lib, tokens=1 << 25, heads=4, **big) == B.EINVAL   # 2^27 rows
    assert attend(lib, tokens=4, batch=(1 << 20) + 1, **big) == B.EINVAL
    f = w4.kv4_attention_workspace_bytes
    assert f(1 << 20, 1, 64, 8, 128, 1 << 16, 16, ragged=True) == 0  # fits, in one part
    assert f((1 << 20) + 1, 1, 64, 8, 128, 1 << 16, 16, ragged=True) == 0


# the binding's own checks come before the library and the device: CPU tensors reach them


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_append_refuses():
    pool = w4.kv4_pool(2, 16, 1, 64, device="cpu")
    slots, pos, rope = t(4, dtype=torch.int64), t(4, dtype=torch.int32), t(10, 64, dtype=torch.float32)
    good = dict(qkv=t(4, 4 * 64), pool=pool, slots=slots, head_dim=64, positions=pos, rope=rope)
    for kw, why in ((dict(qkv=t(4, 256, dtype=torch.float32)), "bfloat16 or float16"), (dict(qkv=t(4, 248)), "do not hold"),
                    (dict(qkv=t(4, 64)), "do not hold"), (dict(qkv=t(256, 4).t()), "contiguous rows"),
                    (dict(qkv=t(4, 260)[:, :256]), "multiple of 8"), (dict(slots=pos), "slots"),
                    (dict(slots=t(5, dtype=torch.int64)), "slots"), (dict(slots=t(8, dtype=torch.int64)[::2]), "contiguous"),
                    (dict(positions=None), "positions"), (dict(positions=slots), "positions"), (dict(rope=t(10, 64)), "float32"),
                    (dict(rope=t(10, 24, dtype=torch.float32)), "multiple of 16"), (dict(rope=t(10, 80, dtype=torch.float32)), "head_dim"),
                    (dict(head_dim=128), "channels"), (dict(pool=pool[:, :, :100]), "contiguous"),
                    (dict(qkv=t(4, 256).requires_grad_()), "inference only"), ({}, "GPU")):
        with pytest.raises(ValueError, match=why):
            w4.kv4_append(**{**good, **kw})
    with pytest.raises(ValueError, match="GPU"):
        w4.kv4_read(pool, slots, 64)
    with pytest.raises(ValueError, match="1-D"):
        w4.kv4_read(pool, t(2, 2, dtype=torch.int64), 64)
    for args in ((0, 64), (10, 0), (10, 24), (10, 64, 0.0), (10, 64, 1e4, 0.5), (10, 64, 1e4, 2.0, 100, 4.0, 2.0)):
        with pytest.raises(ValueError):
            w4.rope_table(*args, device="cpu")


def test_binding_attention_refuses():
    pool = w4.kv4_pool(2, 16, 2, 64, device="cpu")
    i32 = lambda *s: t(*s, dtype=torch.int32)  # noqa: E731
    good = dict(q=t(3, 4, 64), pool=pool, block_table=i32(3, 2), kv_lens=i32(3))
    for kw, why in ((dict(q=t(3, 256)), "heads"), (dict(q=t(3, 4, 64, dtype=torch.float32)), "bfloat16 or float16"),
                    (dict(q=t(4, 3, 64).transpose(0, 1)), "contiguous tokens"), (dict(q=t(3, 3, 64)), "share"),
                    (dict(q=t(3, 4, 128)), "channels"), (dict(block_table=t(3, 2, dtype=torch.int64)), "block_table"),
                    (dict(block_table=i32(3, 0)), "block_table"), (dict(kv_lens=i32(2)), "kv_lens"), (dict(cu_q=i32(3)), "cu_q"),
                    (dict(q=t(4, 4, 64)), "pass cu_q"), (dict(window=-1), "window"), (dict(q=t(3, 4, 64).requires_grad_()), "inference"),
                    (dict(block_table=i32(0, 2), kv_lens=i32(0), cu_q=i32(1)), "without a request"), ({}, "GPU")):
        with pytest.raises(ValueError, match=why):
            w4.kv4_attention(**{**good, **kw})


def test_binding_lora_refuses():
    good = dict(y=t(5, 40), x=t(5, 64), a=t(2, 8, 64), b=t(2, 40, 8), index=t(5, dtype=torch.int32))
    for kw, why in ((dict(x=t(5, 64, dtype=torch.float32)), "bfloat16 or float16"), (dict(y=t(5, 40, dtype=torch.float16)), "one dtype"),
                    (dict(a=t(2, 12, 64), b=t(2, 40, 12)), "multiple of 8"), (dict(a=t(2, 136, 64), b=t(2, 40, 136)), "at most 128"),
                    (dict(b=t(2, 40, 16)), "are not"), (dict(b=t(3, 40, 8)), "are not"), (dict(a=t(2, 64, 8).transpose(1, 2)), "contiguous"),
                    (dict(x=t(5, 56)), "needed"), (dict(y=t(4, 40)), "needed"), (dict(index=t(5, dtype=torch.int64)), "index"),
                    (dict(index=t(4, dtype=torch.int32)), "index"), (dict(scales=t(2)), "scales"), (dict(y=t(40, 5).t()), "contiguous rows"),
                    (dict(x=t(5, 64).requires_grad_()), "inference"), ({}, "GPU")):
        with pytest.raises(ValueError, match=why):
            w4.lora_add(**{**good, **kw})


def test_captured_calls_need_an_explicit_workspace(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(ValueError, match="workspace"):
        S._workspace(None, 100, "cuda", 0)
    assert S._workspace(None, 0, "cuda", 0) == (None, 0)
