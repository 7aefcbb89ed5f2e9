"""Plain implementations of the 4-bit cache's operators for the tests: the
quantizer and the rotation as FP32 steps in numpy, attention and adapters in
64 bits on the host.  Nothing here uses the library."""
from __future__ import annotations

import numpy as np
import torch


def quantized(x: np.ndarray, width: int) -> np.ndarray:
    """x [..., d] float32 -> the values its 4-bit codes stand for (float32: code * scale)."""
    g = x.astype(np.float32).reshape(*x.shape[:-1], -1, width)
    s = (np.abs(g).max(-1, keepdims=True) / np.float32(7)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s == 0, np.float32(0), np.clip(np.rint((g / s).astype(np.float32)), -8, 7))
    return (q.astype(np.float32) * s).astype(np.float32).reshape(x.shape)


def rotated(x: np.ndarray, table: np.ndarray, positions: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [t, h, d] float32 turned by table rows [cos | sin] at positions, every operation one FP32 step."""
    rot = table.shape[1]
    half = rot // 2
    row = table[positions][:, None]
    c, s = row[..., :half], row[..., half:]
    out = x.astype(np.float32).copy()
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    a, b = x[..., at[0]].astype(np.float32), x[..., at[1]].astype(np.float32)
    out[..., at[0]] = a * c - b * s
    out[..., at[1]] = b * c + a * s
    return out


def attention(q, k, v, kv_len, q_len, causal, window, scale, seen_page=None):
    """One request in 64 bits: q [n, h, d], k, v [m, hk, d] -> (out [n, h, d], tol [n, h, d] apart from the output's
    own rounding).  seen_page [m]: tokens whose page exists."""
    q, k, v = (torch.as_tensor(x).double() for x in (q, k, v))
    n, h, d = q.shape
    m, hk = k.shape[0], k.shape[1]
    out, tol = torch.zeros(n, h, d, dtype=torch.float64), torch.zeros(n, h, d, dtype=torch.float64)
    if m == 0:
        return out, tol
    pos = kv_len - q_len + torch.arange(n).view(-1, 1)
    tok = torch.arange(m).view(1, -1)
    seen = (tok < kv_len).expand(n, m).clone()
    if causal:
        seen &= tok <= pos
    if window:
        seen &= pos - tok < window
        if not causal:
            seen &= tok - pos < window
    if seen_page is not None:
        seen &= torch.as_tensor(seen_page).view(1, -1)
    share = h // hk
    for i in range(h):
        kk, vv = k[:, i // share], v[:, i // share]
        z = (q[:, i] @ kk.t()) * scale
        z = z.masked_fill(~seen, -torch.inf)
        p = torch.softmax(z, 1).nan_to_num(0.0)
        vv = torch.where(seen.any(0).view(-1, 1), vv, 0.0)
        kk = torch.where(seen.any(0).view(-1, 1), kk, 0.0)
        out[:, i] = p @ vv
        # Error of the kernel's arithmetic.  A probability times a value scale is rounded to f16: 2^-11 of each
        # (half a step), or 2^-25 of the largest value scale where it is subnormal (relative to the row's largest
        # probability).  Sums run in FP32 over codes offset by 24 (at most 31 in size).  A logit is off by an FP32
        # sum of up to 31 |q| ks terms and a few roundings of itself.
        ksmax, vsmax = kk.abs().max() / 7, vv.abs().max() / 7
        dz = 2.0 ** -22 * (31 * q[:, i].abs().sum(1) * ksmax * abs(scale) + 4 * z.masked_fill(~seen, 0).abs().amax(1) + 4)
        count, pmax = seen.sum(1), p.amax(1)
        tol[:, i] = ((p @ vv.abs()) * (2.0 ** -11 + 2.0 ** -18 + dz).view(-1, 1)
                     + (vsmax * count * 2.0 ** -24 * (14 * pmax + 2)).view(-1, 1))
    return out, tol


def lora(y, x, a, b, index, scales):
    """(out, tol) in 64 bits: y + scale (x A^T) B^T per row."""
    y, x, a, b = (t.double() for t in (y, x, a, b))
    out, tol = y.clone(), torch.zeros_like(y)
    for i, l in enumerate(index.tolist()):
        if 0 <= l < a.shape[0]:
            f = 1.0 if scales is None else float(scales[l])
            t = a[l] @ x[i]
            out[i] += f * (b[l] @ t)
            # FP32 sums over k (products exact in FP32 up to their rounding) and over the rank; t enters with 16 bits
            size = a[l].abs() @ x[i].abs()
            tol[i] = abs(f) * (b[l].abs() @ (size * (2.0 ** -24 * (8 + x.shape[1] / 32)) + t.abs() * (2.0 ** -16 + 2.0 ** -20)))
            tol[i] += 2.0 ** -22 * (out[i].abs() + y[i].abs())
    return out, tol


def within(got: torch.Tensor, want: torch.Tensor, tol: torch.Tensor, what: str):
    """|got - want| within tol plus half a step of got's type (relative, and the subnormals')."""
    got_ = got.detach().cpu().double()
    step = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).tiny * step * 2
    limit = tol + step * (want.abs() + tol) + tiny
    bad = ~((got_ - want).abs() <= limit)
    if bad.any():
        at = bad.nonzero()[:4].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond tolerance, first {at}: got "
                             f"{got_[bad][:4].tolist()}, want {want[bad][:4].tolist()}, tol {limit[bad][:4].tolist()}")
