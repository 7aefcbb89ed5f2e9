"""Refusals of the 8-bit float layer and of attention on shared prefixes, from
metadata alone (no GPU: every call here returns before a launch), and their sizes;
the tests' own e4m3 against torch's."""
import numpy as np
import pytest
import torch

import weight_only_int4_rtn_amd as w4
from weight_only_int4_rtn_amd import _binding as B
from weight_only_int4_rtn_amd import _fp8 as F
from weight_only_int4_rtn_amd import _serving as S

from . import fp8_ref as R
from . import kv4_prefix_ref as pref
from . import kv4_ref as ref

A = 1 << 20  # a 16-byte aligned fake device address (never dereferenced)
GB = 1 << 30
E4M3 = F.E4M3


@pytest.fixture(scope="module")
def lib():
    S._lib()
    return F._lib()


# ---------------------------------------------------------------------------
# the oracles
# ---------------------------------------------------------------------------


def test_e4m3_is_the_format():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    got = R.decode(codes)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])
    assert R.decode([0x7E])[0] == 448 and R.decode([0x01])[0] == 2.0 ** -9
    x = torch.cat((torch.randn(100000) * 100, torch.randn(100000) * 0.01, torch.arange(-3584, 3585) / 8, torch.arange(-64, 65) * 2.0 ** -12))
    x = x.clamp(-448, 448)
    assert np.array_equal(R.encode(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_quantizer_by_hand():
    x = np.zeros((1, 256), np.float32)
    x[0, :4] = 7.0, -3.5, 0.0625, 0.01  # s = 1/64: 448, -224, 4, 0.64 (halfway steps of 1/16: 0.625)
    c, s = R.quantize_rows(x)
    assert s[0, 0] == np.float32(7) / np.float32(448) and s[0, 1] == 0
    assert R.decode(c[0, :4]).tolist() == [448.0, -224.0, 4.0, 0.625] and not c[0, 4:].any()
    x[0, 130] = np.inf
    c, s = R.quantize_rows(x)
    assert np.isnan(s[0, 1]) and (c[0, 128:] == 0x7F).all() and c[0, 0] == 0x7E


def test_linear_oracle_is_a_product():
    g = torch.Generator().manual_seed(1)
    cx, sx = R.quantize_rows(torch.randn(5, 256, generator=g).numpy())
    cw, sw = R.quantize_blocks(torch.randn(140, 256, generator=g).numpy())
    y, tol = R.linear(cx, sx, cw, sw, torch.ones(140))
    a = torch.from_numpy(R.decode(cx)) * torch.from_numpy(sx).double().repeat_interleave(128, 1)
    b = torch.from_numpy(R.decode(cw)) * torch.from_numpy(sw).double().repeat_interleave(128, 0)[:140].repeat_interleave(128, 1)
    assert torch.allclose(y, a @ b.t() + 1, rtol=1e-12, atol=1e-12) and (tol > 0).all() and (tol < 0.05 * (a.abs() @ b.abs().t())).all()


def test_prefix_oracle_is_attention_over_both():
    g = torch.Generator().manual_seed(2)
    q, k, v = torch.randn(3, 4, 64, generator=g), torch.randn(30, 2, 64, generator=g), torch.randn(30, 2, 64, generator=g)
    for causal in (True, False):
        want = ref.attention(q, k, v, 30, 3, causal, 0, 0.125)[0]
        got = pref.attention(q, k, v, pref.seen_tokens(20, 10, 3, causal), 0.125)[0]
        assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)
    assert pref.seen_tokens(2, 1, 3, True).tolist() == [[True, True, False], [True, True, False], [True, True, True]]


# ---------------------------------------------------------------------------
# the C boundary
# ---------------------------------------------------------------------------


def rows(lib, **kw):
    d = dict(x=A, dtype=B.BF16, act=0, m=4, k=256, ldx=256, codes=A + GB, scales=A + 2 * GB)
    d.update(kw)
    return lib.quantize_fp8_rows(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=0), B.OK), (dict(m=0, x=None, codes=None, scales=None), B.OK),
    (dict(dtype=B.F32), B.EUNSUPPORTED), (dict(dtype=E4M3), B.EUNSUPPORTED), (dict(dtype=9), B.EUNSUPPORTED), (dict(act=3), B.EUNSUPPORTED),
    (dict(m=-1), B.EINVAL), (dict(m=(1 << 24) + 1), B.EINVAL), (dict(k=0), B.EINVAL), (dict(k=200, ldx=200), B.EINVAL),
    (dict(k=-128), B.EINVAL), (dict(k=(1 << 22) + 128, ldx=1 << 23), B.EINVAL), (dict(m=1 << 24, k=1 << 22, ldx=1 << 22), B.EINVAL),
    (dict(ldx=248), B.EINVAL), (dict(ldx=260), B.EINVAL), (dict(ldx=(1 << 24) + 8), B.EINVAL), (dict(act=1), B.EINVAL),
    (dict(x=None), B.EINVAL), (dict(codes=None), B.EINVAL), (dict(scales=None), B.EINVAL),
    (dict(x=A + 8), B.EINVAL), (dict(codes=A + GB + 8), B.EINVAL), (dict(scales=A + 2), B.EINVAL),
    (dict(codes=A), B.EINVAL), (dict(scales=A + 1024), B.EINVAL), (dict(scales=A + GB + 1020), B.EINVAL),
])
def test_rows_status(lib, kw, status):
    assert rows(lib, **kw) == status


def test_blocks_status(lib):
    def blocks(**kw):
        d = dict(w=A, dtype=B.F32, n=300, k=256, ldw=256, codes=A + GB, scales=A + 2 * GB)
        d.update(kw)
        return lib.quantize_fp8_blocks(*d.values(), None)
    assert blocks(n=0) == B.OK
    assert blocks(dtype=E4M3) == B.EUNSUPPORTED and blocks(dtype=-1) == B.EUNSUPPORTED
    for kw in (dict(n=-1), dict(k=100), dict(ldw=128), dict(ldw=258), dict(w=None), dict(w=A + 4), dict(codes=None), dict(scales=None),
               dict(codes=A + 1024), dict(scales=A + GB)):
        assert blocks(**kw) == B.EINVAL, kw


def linear(lib, **kw):
    d = dict(x=A, x_dtype=B.BF16, xs=None, act=0, m=100, k=512, ldx=512, w=A + GB, ws=A + 2 * GB, n=300, bias=A + 3 * GB, y=A + 4 * GB,
             y_dtype=B.BF16, ldy=300, work=A + 5 * GB, bytes=GB)
    d.update(kw)
    return lib.fp8_linear(*d.values(), None)


CODES = dict(x_dtype=E4M3, xs=A + 6 * GB)


@pytest.mark.parametrize("kw,status", [
    (dict(m=0), B.OK), (dict(n=0, ldy=0), B.OK), (dict(m=0, x=None, w=None, ws=None, y=None, work=None), B.OK),
    (dict(x_dtype=B.F32), B.EUNSUPPORTED), (dict(y_dtype=B.F16), B.EUNSUPPORTED), (dict(y_dtype=B.F32), B.EUNSUPPORTED),
    (dict(y_dtype=E4M3), B.EUNSUPPORTED), (dict(act=7), B.EUNSUPPORTED), (dict(CODES, act=2), B.EUNSUPPORTED),
    (dict(xs=A + 6 * GB), B.EINVAL), (dict(x_dtype=E4M3), B.EINVAL),
    (dict(m=-1), B.EINVAL), (dict(n=-1), B.EINVAL), (dict(n=(1 << 24) + 1, ldy=1 << 25), B.EINVAL), (dict(k=500), B.EINVAL), (dict(k=0), B.EINVAL),
    (dict(ldx=504), B.EINVAL), (dict(ldx=516), B.EINVAL), (dict(act=1), B.EINVAL), (dict(ldy=299), B.EINVAL), (dict(ldy=(1 << 24) + 1), B.EINVAL),
    (dict(CODES, ldx=520), B.EINVAL), (dict(CODES, ldx=(1 << 22) + 16), B.EINVAL),
    (dict(x=None), B.EINVAL), (dict(w=None), B.EINVAL), (dict(ws=None), B.EINVAL), (dict(y=None), B.EINVAL),
    (dict(x=A + 8), B.EINVAL), (dict(w=A + GB + 8), B.EINVAL), (dict(ws=A + 2), B.EINVAL), (dict(bias=A + 1), B.EINVAL), (dict(y=A + 1), B.EINVAL),
    (dict(CODES, xs=A + 2), B.EINVAL),
    (dict(y=A), B.EINVAL), (dict(y=A + GB), B.EINVAL), (dict(y=A + 2 * GB), B.EINVAL), (dict(y=A + 3 * GB), B.EINVAL), (dict(CODES, y=A + 6 * GB), B.EINVAL),
    (dict(work=None), B.EWORKSPACE), (dict(bytes=100), B.EWORKSPACE), (dict(work=A + 5 * GB + 8), B.EINVAL),
    (dict(work=A), B.EINVAL), (dict(work=A + GB), B.EINVAL), (dict(work=A + 2 * GB), B.EINVAL), (dict(work=A + 4 * GB), B.EINVAL),
])
def test_linear_status(lib, kw, status):
    assert linear(lib, **kw) == status


def test_linear_workspace(lib):
    f = w4.linear_fp8_workspace_bytes
    assert f(0, 100, 256) == 0 and f(10, 0, 256) == 0 and f(10, 10, 200) == 0 and f(-1, 10, 128) == 0
    assert f(1, 2560, 2048) == 0 and f(1, 2560, 2048, codes=True) == 0   # one row: quantized in the kernel
    assert f(4096, 32768, 2048, codes=True) == 0                          # unsplit
    assert f(4096, 32768, 2048) == (1 << 20) + 4096 * 2048 + 4096 * 16 * 4
    assert f(64, 2048, 16384, codes=True) > 1 << 20                       # split along k
    assert lib.fp8_linear_workspace_bytes(B.F32, 64, 2048, 16384) == 0


def prefix(lib, **kw):
    d = dict(q=A, dtype=B.F16, tokens=4, ldq=512, heads=4, kv_heads=1, dim=128, pool=A + GB, pages=8, page=16, ptable=A + 2 * GB, pwidth=400,
             ldp=400, plens=A + 3 * GB, cug=None, groups=1, table=A + 4 * GB, width=4, ldt=4, lens=A + 5 * GB, cu=None, batch=4, causal=1,
             scale=0.1, out=A + 6 * GB, ldo=512, ws=A + 7 * GB, ws_bytes=GB)
    d.update(kw)
    return lib.kv4_prefix_attention(*d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=0, batch=0), B.OK), (dict(tokens=0, cu=A + 8 * GB), B.OK), (dict(dtype=B.F32), B.EUNSUPPORTED), (dict(dtype=E4M3), B.EUNSUPPORTED),
    (dict(tokens=3), B.EINVAL), (dict(batch=0, cu=A + 8 * GB), B.EINVAL), (dict(heads=3, kv_heads=2), B.EINVAL), (dict(dim=80), B.EINVAL),
    (dict(page=17), B.EINVAL), (dict(pages=0), B.EINVAL), (dict(width=0), B.EINVAL), (dict(pwidth=0), B.EINVAL), (dict(groups=0), B.EINVAL),
    (dict(groups=2), B.EINVAL), (dict(pwidth=1 << 24, ldp=1 << 24), B.EINVAL), (dict(pwidth=1 << 62, ldp=1 << 62), B.EINVAL),
    (dict(groups=(1 << 20) + 1, cug=A + 8 * GB), B.EINVAL), (dict(ldq=504), B.EINVAL), (dict(ldo=516), B.EINVAL), (dict(ldt=3), B.EINVAL),
    (dict(ldp=399), B.EINVAL), (dict(scale=float("nan")), B.EINVAL), (dict(q=None), B.EINVAL), (dict(pool=None), B.EINVAL),
    (dict(ptable=None), B.EINVAL), (dict(plens=None), B.EINVAL), (dict(table=None), B.EINVAL), (dict(lens=None), B.EINVAL), (dict(out=None), B.EINVAL),
    (dict(q=A + 8), B.EINVAL), (dict(out=A + 6 * GB + 8), B.EINVAL), (dict(ptable=A + 2), B.EINVAL), (dict(plens=A + 1), B.EINVAL),
    (dict(cug=A + 2, groups=1), B.EINVAL), (dict(out=A), B.EINVAL), (dict(out=A + GB), B.EINVAL), (dict(out=A + 2 * GB), B.EINVAL),
    (dict(out=A + 3 * GB), B.EINVAL), (dict(out=A + 4 * GB), B.EINVAL), (dict(out=A + 5 * GB), B.EINVAL),
    (dict(ws=None), B.EWORKSPACE), (dict(ws_bytes=1 << 20), B.EWORKSPACE), (dict(ws=A + 7 * GB + 8), B.EINVAL), (dict(ws=A), B.EINVAL),
    (dict(ws=A + GB), B.EINVAL), (dict(ws=A + 6 * GB), B.EINVAL),
])
def test_prefix_status(lib, kw, status):
    assert prefix(lib, **kw) == status


def test_prefix_workspace(lib):
    f = w4.kv4_prefix_attention_workspace_bytes
    assert f(0, 0, 1, 4, 1, 128, 10, 10, 16) == 0 and f(4, 4, 1, 4, 3, 128, 10, 10, 16) == 0 and f(4, 4, 0, 4, 1, 128, 10, 10, 16) == 0
    assert f(4, 3, 1, 4, 1, 128, 10, 10, 16) == 0 and f(4, 4, 1, 4, 1, 128, 0, 10, 16) == 0
    rows = w4.kv4_prefix_attention_tile_rows
    # little to share: one launch, which needs nothing for one part
    assert rows(4, 4, 1, 4, 1, 128, 1, 1, 16) == 0 and f(4, 4, 1, 4, 1, 128, 1, 1, 16) == 0
    assert rows(4, 4, 1, 4, 1, 128, 400, 1, 16) == 0 and f(4, 4, 1, 4, 1, 128, 400, 1, 16) > 1 << 20
    # apart: at least a row of sums and two statistics of each query and head
    assert rows(64, 64, 1, 32, 8, 128, 128, 4, 64) == 16 and rows(192, 192, 4, 32, 8, 128, 256, 8, 128) == 64
    assert f(64, 64, 1, 32, 8, 128, 128, 4, 64) >= (1 << 20) + 64 * 32 * 130 * 4
    assert rows(4, 3, 1, 4, 1, 128, 10, 10, 16) == 0 and rows(0, 0, 1, 4, 1, 128, 10, 10, 16) == 0


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------


def test_binding_refusals():
    bf = torch.bfloat16
    x, codes, scales = torch.zeros(3, 256, dtype=bf), torch.zeros(130, 256, dtype=torch.float8_e4m3fn), torch.zeros(2, 2)
    for call in (lambda: w4.quantize_fp8(x), lambda: w4.quantize_fp8_weight(torch.zeros(4, 128)), lambda: w4.linear_fp8(x, codes, scales)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for bad in (x[:, :200], torch.zeros(3, 0, dtype=bf), x.float(), x.view(torch.int16)):
        with pytest.raises(ValueError):
            w4.quantize_fp8(bad)
    with pytest.raises(ValueError):
        w4.quantize_fp8(torch.zeros(3, 129 * 2, dtype=bf), act=w4.Act.SWIGLU)
    for bad in (torch.zeros(3, 100), torch.zeros(128), torch.zeros(3, 128, dtype=torch.float64)):
        with pytest.raises(ValueError):
            w4.quantize_fp8_weight(bad)
    xs = torch.zeros(3, 2)
    for args, kw in (((x, codes.view(torch.uint8), scales), {}), ((x, codes[:, :128], scales), {}), ((x, codes, scales[:1]), {}),
                     ((x, codes, scales.double()), {}), ((x, codes, scales.t()), {}), ((x, codes, scales), dict(bias=torch.zeros(130))),
                     ((x, codes, scales), dict(bias=torch.zeros(129, dtype=bf))), ((x, codes, scales), dict(x_scales=xs)),
                     ((x, codes, scales), dict(out_dtype=torch.float16)), ((codes[:3], codes, scales), {}),
                     ((codes[:3], codes, scales), dict(x_scales=xs[:2])), ((codes[:3], codes, scales), dict(x_scales=xs, out_dtype=torch.float32)),
                     ((codes[:3], codes, scales), dict(x_scales=xs, act=w4.Act.GELU_TANH)), ((x, codes, scales), dict(act=w4.Act.SWIGLU)),
                     ((x, codes[:, ::2], scales), {})):
        with pytest.raises(ValueError):
            w4.linear_fp8(*args, **kw)
    for t in (x.clone().requires_grad_(),):
        with pytest.raises(ValueError, match="inference only"):
            w4.linear_fp8(t, codes, scales)
        with pytest.raises(ValueError, match="inference only"):
            w4.quantize_fp8(t)


def test_prefix_binding_refusals():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool = w4.kv4_pool(4, 16, 2, 64, device="cpu")
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    good = dict(prefix_table=i32(1, 2), prefix_lens=i32(1), block_table=i32(3, 2), kv_lens=i32(3))
    with pytest.raises(ValueError, match="GPU"):
        w4.kv4_prefix_attention(q, pool, **good)
    for kw in (dict(prefix_table=i32(2)), dict(prefix_table=i32(1, 0)), dict(prefix_table=i32(1, 2).long()), dict(prefix_lens=i32(2)),
               dict(prefix_lens=i32(1).long()), dict(prefix_table=i32(2, 2), prefix_lens=i32(2)), dict(cu_groups=i32(3)), dict(cu_groups=i32(2).long()),
               dict(kv_lens=i32(2)), dict(block_table=i32(2, 2)), dict(out=torch.zeros(3, 4, 64)), dict(cu_q=i32(3))):
        with pytest.raises(ValueError):
            w4.kv4_prefix_attention(q, pool, **{**good, **kw})
    with pytest.raises(ValueError, match="inference only"):
        w4.kv4_prefix_attention(q.clone().requires_grad_(), pool, **good)
