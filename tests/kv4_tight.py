"""Attention over the 4-bit cache in 64 bits with an error bound that follows each
token's own share of the row: a token that the softmax leaves out adds nothing to
it, however large its values.  Nothing here uses the library.

The bound, for out = sum_t P[t] v[t] with v[t] = vs[t] c[t], codes |c| <= 7:

  weights    P vs enters the second product as f16: 2^-11 of each (half a step), or,
             for one more than 2^19 below the row's largest, 2^-30 of the largest
             (f16's smallest step is 2^-24 and the largest weight is kept at 2^5 or
             more); a weight's error reaches the output times its code
  sums       FP32 sums of codes offset by 24 (at most 31 in size), four waves by 32
             tokens at a time, and the parts' join: 2^-24 of 31 P vs for each of at
             most 8 + n / 64 additions that matter
  logits     off by dz, so each P by 2 dz relatively (its own and the sum's): FP32
             sums of up to 31 |q| ks terms and a few roundings of the logit itself
  the rest   exponential, sum of P, quotient: 2^-18 + n 2^-28"""
from __future__ import annotations

import numpy as np
import torch

from tests import kv4_ref as ref


def scales_of(v: torch.Tensor, width: int) -> torch.Tensor:
    """The scale each value was quantized with, [..., d] (the largest code of a group is 7)."""
    g = v.unflatten(-1, (-1, width))
    return (g.abs().amax(-1, keepdim=True) / 7).expand_as(g).flatten(-2)


def seen_by(n, m, kv_len, causal, window, seen_page=None):
    pos = kv_len - n + torch.arange(n).view(-1, 1)
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
    return seen


def probabilities(q, k, seen, scale):
    """One head: q [n, d], k [m, d] in 64 bits -> (softmax [n, m], logits)."""
    z = ((q @ k.t()) * scale).masked_fill(~seen, -torch.inf)
    return torch.softmax(z, 1).nan_to_num(0.0), z


def attention(q, k, v, kv_len, causal, window, scale, seen_page=None):
    """One request: q [n, h, d], k, v [m, hk, d] (quantized values) -> (out, tol) [n, h, d] apart from the output's own
    rounding."""
    q, k, v = (torch.as_tensor(x).double() for x in (q, k, v))
    n, h, d = q.shape
    m, hk = k.shape[0], k.shape[1]
    out, tol = torch.zeros(n, h, d, dtype=torch.float64), torch.zeros(n, h, d, dtype=torch.float64)
    if m == 0 or n == 0:
        return out, tol
    width = min(d, 128)
    seen = seen_by(n, m, kv_len, causal, window, seen_page)
    for i in range(h):
        kk, vv = k[:, i // (h // hk)], v[:, i // (h // hk)]
        p, z = probabilities(q[:, i], kk, seen, scale)
        out[:, i] = p @ vv
        ks, vs = scales_of(kk, width), scales_of(vv, width)
        # the logit's sums: per token sum_c |q| ks, and its own size
        dz = 2.0 ** -22 * (31 * abs(scale) * (q[:, i].abs() @ ks.t()) + 4 * z.abs() + 4).masked_fill(~seen, 0).amax(1)
        size = p @ vs                                            # sum of P vs, per channel's block
        top = torch.stack([(p * vs[:, b]).amax(1) for b in range(0, d, width)]).amax(0)
        low = torch.stack([((p * vs[:, b] < top.view(-1, 1) * 2.0 ** -19) & seen).sum(1) for b in range(0, d, width)], 1)
        low = low.repeat_interleave(width, 1).double()
        tol[:, i] = ((p @ vv.abs()) * (2.0 ** -11 + 2 * dz + 2.0 ** -18 + m * 2.0 ** -28).view(-1, 1)
                     + size * 31 * 2.0 ** -24 * (8 + m / 64) + 7 * 2.0 ** -30 * low * top.view(-1, 1))
    return out, tol


def as_f16(w: torch.Tensor) -> torch.Tensor:
    return w.to(torch.float16).double()


def model(q, k, v, kv_len, causal, window, scale, reference):
    """The same with weights P vs rounded to f16 relative to `reference(p, vs)` [n, 1] per row (vs [m, blocks])."""
    q, k, v = (torch.as_tensor(x).double() for x in (q, k, v))
    n, h, d = q.shape
    width = min(d, 128)
    seen = seen_by(n, k.shape[0], kv_len, causal, window)
    out = torch.zeros(n, h, d, dtype=torch.float64)
    for i in range(h):
        kk, vv = k[:, i // (h // k.shape[1])], v[:, i // (h // k.shape[1])]
        p, _ = probabilities(q[:, i], kk, seen, scale)
        vs = scales_of(vv, width)
        codes = torch.where(vs > 0, vv / vs, 0.0)
        r = reference(p, vs[:, ::width])
        for b in range(0, d, width):
            out[:, i, b:b + width] = (as_f16(p * vs[:, b] / r) * r) @ codes[:, b:b + width]
    return out


class Request:
    """One request's tokens in a cache of its own pages, in shuffled order among pages of NaN."""

    def __init__(self, lib, dev, x, page, seed=0, extra_columns=0):
        """x [n, 2, kv_heads, d] in a 16-bit type: keys, values."""
        n, _, hk, d = x.shape
        g = torch.Generator().manual_seed(seed)
        need = -(-n // page)
        self.pool = torch.full((need + 2, hk, lib.kv4_pool(1, page, hk, d, device="cpu").shape[2]), 255, dtype=torch.uint8).to(dev)
        self.table = torch.full((1, need + extra_columns), -1, dtype=torch.int32)
        self.table[0, :need] = torch.randperm(need + 2, generator=g)[:need].to(torch.int32)
        at = torch.arange(n)
        self.slots = (self.table[0].long()[at // page] * page + at % page).to(dev)
        lib.kv4_append(x.reshape(n, -1).to(dev), self.pool, self.slots, d)
        values = ref.quantized(x.float().numpy(), min(d, 128))
        self.k, self.v = values[:, 0], values[:, 1]
        self.n, self.d, self.page, self.dev, self.lib = n, d, page, dev, lib

    def attend(self, q, causal=True, window=0, scale=None, ragged=None, kv_len=None):
        """q [tokens, heads, d] of the request's last tokens."""
        ragged = q.shape[0] != 1 if ragged is None else ragged
        cu = torch.tensor([0, q.shape[0]], dtype=torch.int32, device=self.dev) if ragged else None
        lens = torch.tensor([self.n if kv_len is None else kv_len], dtype=torch.int32, device=self.dev)
        return self.lib.kv4_attention(q.to(self.dev), self.pool, self.table.to(self.dev), lens, cu_q=cu, causal=causal,
                                      window=window, scale=scale)

    def check(self, q, out, causal=True, window=0, scale=None, what="", kv_len=None):
        m = self.n if kv_len is None else kv_len
        want, tol = attention(q, self.k[:m], self.v[:m], m, causal, window, self.d ** -0.5 if scale is None else scale)
        ref.within(out, want, tol, what)


def outlier_inputs(n, hk, d, heads, tokens, ratio, at, dtype, seed, blocks=1.0):
    """Keys, values and queries in which the tokens `at` have values `ratio` times the others' and logits some 60 below
    them; `blocks`: what the second block's values (channels from 128 on) are multiplied by."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, 2, hk, d, generator=g)
    for t in at:
        x[t, 1] *= ratio
        x[t, 0] = 0.0
        x[t, 0, :, 0] = -64.0
    x[:, 1, :, 128:] *= blocks
    q = torch.randn(tokens, heads, d, generator=g)
    q[:, :, 0] = d ** 0.5  # a logit of -64 for those tokens, of this token's own k[0] for the others
    return x.to(dtype), q.to(dtype)


def as_numpy(t):
    return np.asarray(t.detach().cpu().float())
