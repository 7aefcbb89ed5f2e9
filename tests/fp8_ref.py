"""Plain implementations of the 8-bit float layer for the tests: e4m3 written
from its definition, the quantizer as FP32 steps in numpy, products in 64 bits
on the host.  Nothing here uses the library."""
from __future__ import annotations

import math

import numpy as np
import torch


def decode(codes) -> np.ndarray:
    """Values (float64) of e4m3 bytes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN."""
    b = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, f = (b >> 3) & 15, b & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e.astype(np.float64) - 10))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b >> 7, -v, v)


_POSITIVE = decode(np.arange(127))  # 0 .. 448, rising


def encode(v) -> np.ndarray:
    """e4m3 bytes of the values nearest to v (|v| <= 448; ties to the even code), found by search."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def _quantize(blocks: np.ndarray, axes) -> tuple[np.ndarray, np.ndarray]:
    x = blocks.astype(np.float32)
    with np.errstate(all="ignore"):
        top = np.abs(x).max(axes, keepdims=True)  # NaN where there is one
        s = (top / np.float32(448)).astype(np.float32)
        bad = ~np.isfinite(top)
        s = np.where(bad, np.float32(np.nan), s)
        z = np.where(s == 0, np.float32(0), np.clip((x / s).astype(np.float32), -448, 448))
        codes = np.where(bad, 0x7F, encode(np.where(np.isnan(z), 0, z)))
        codes = np.where(s == 0, 0, codes)
    return codes.astype(np.uint8), s


def quantize_rows(x) -> tuple[np.ndarray, np.ndarray]:
    """x [m, k] float32 -> codes [m, k] uint8, scales [m, k / 128] float32."""
    x = np.asarray(x, dtype=np.float32)
    m, k = x.shape
    c, s = _quantize(x.reshape(m, k // 128, 128), 2)
    return c.reshape(m, k), s.reshape(m, k // 128)


def quantize_blocks(w) -> tuple[np.ndarray, np.ndarray]:
    """w [n, k] float32 -> codes [n, k] uint8, scales [ceil(n / 128), k / 128] float32."""
    w = np.asarray(w, dtype=np.float32)
    n, k = w.shape
    nb = -(-n // 128)
    pad = np.zeros((nb * 128, k), np.float32)
    pad[:n] = w
    c, s = _quantize(pad.reshape(nb, 128, k // 128, 128), (1, 3))
    return c.reshape(nb * 128, k)[:n], s.reshape(nb, k // 128)


def activate(x: torch.Tensor, act: str) -> torch.Tensor:
    """The activation in 64 bits, before its rounding to x's dtype."""
    v = x.double()
    if act == "swiglu":
        up, gate = v.chunk(2, -1)
        return up * gate * torch.sigmoid(gate)
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def linear(cx, sx, cw, sw, bias=None):
    """(y, tol) in 64 bits from codes (uint8) and scales; tol apart from the output's own rounding.

    The kernel's arithmetic, per group of 128 columns: of eight neighbouring products all are cut 2^-13 below the
    largest one's exponent (7 of them lose less than that times the largest each); the sixteen sums and the groups are
    added in FP32 (a step of 2^-23 an addition, whichever way it is cut), after three FP32 multiplications."""
    a, b = torch.from_numpy(decode(cx)), torch.from_numpy(decode(cw))
    m, k = a.shape
    n, groups = b.shape[0], k // 128
    sx = torch.as_tensor(np.asarray(sx), dtype=torch.float64)
    sw = torch.as_tensor(np.asarray(sw), dtype=torch.float64).repeat_interleave(128, 0)[:n]
    y, cut, size = (torch.zeros(m, n, dtype=torch.float64) for _ in range(3))
    for g in range(groups):
        p, q = a[:, 128 * g:128 * g + 128], b[:, 128 * g:128 * g + 128]
        f = sx[:, g:g + 1] * sw[:, g]
        y += f * (p @ q.t())
        size += f.abs() * (p.abs() @ q.abs().t())
        for e in range(0, 128, 8):
            big = torch.zeros(m, n, dtype=torch.float64)
            for j in range(e, e + 8):
                big = torch.maximum(big, torch.outer(p[:, j].abs(), q[:, j].abs()))
            cut += f.abs() * big
    tol = cut * 7 * 2.0 ** -13 + size * 2.0 ** -23 * (16 + groups + 3)
    if bias is not None:
        y = y + bias.double()
        tol = tol + 2.0 ** -23 * (y.abs() + bias.double().abs())
    return y, tol


def within(got: torch.Tensor, want: torch.Tensor, tol: torch.Tensor, what: str):
    """|got - want| within tol plus half a step of got's type (relative, and the subnormals'); NaN where want is NaN."""
    got_ = got.detach().cpu().double()
    want = want.reshape(got_.shape)
    tol = tol.reshape(got_.shape)
    step = torch.finfo(got.dtype).eps / 2
    limit = tol + step * (want.abs() + tol) + torch.finfo(got.dtype).tiny * step * 2
    bad = ~(((got_ - want).abs() <= limit) | (got_.isnan() & want.isnan()))
    if bad.any():
        at = bad.nonzero()[:4].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond tolerance, first {at}: got {got_[bad][:4].tolist()}, "
                             f"want {want[bad][:4].tolist()}, tol {limit[bad][:4].tolist()}")
