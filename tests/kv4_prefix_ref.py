"""Attention over a shared prefix and own tokens in 64 bits, with a tolerance
from the kernels' roundings.  Nothing here uses the library."""
from __future__ import annotations

import torch


def attention(q, k, v, seen, scale):
    """One request: q [n, h, d], k, v [m, hk, d], seen [n, m] -> (out [n, h, d], tol [n, h, d] apart from the output's own
    rounding).

    A probability times a value scale is rounded to f16: 2^-11 of each (half a step), or 2^-25 of the largest value scale
    where it is subnormal, relative to the largest probability of its part (prefix or own tokens), so at most the row's.
    Sums run in FP32 over codes offset by 24 (at most 31 in size); a logit is off by an FP32 sum of up to 31 |q| ks terms
    and a few roundings of itself; joining the two parts takes two exponentials, four products and two sums in FP32,
    each off by 2^-22 at most."""
    q, k, v = (torch.as_tensor(x).double() for x in (q, k, v))
    n, h, d = q.shape
    m, hk = k.shape[0], k.shape[1]
    out, tol = torch.zeros(n, h, d, dtype=torch.float64), torch.zeros(n, h, d, dtype=torch.float64)
    if m == 0:
        return out, tol
    share = h // hk
    some = seen.any(0).view(-1, 1)
    for i in range(h):
        kk, vv = (torch.where(some, x[:, i // share], 0.0) for x in (k, v))
        z = ((q[:, i] @ kk.t()) * scale).masked_fill(~seen, -torch.inf)
        p = torch.softmax(z, 1).nan_to_num(0.0)
        out[:, i] = p @ vv
        ksmax, vsmax = kk.abs().max() / 7, vv.abs().max() / 7
        dz = 2.0 ** -22 * (31 * q[:, i].abs().sum(1) * ksmax * abs(scale) + 4 * z.masked_fill(~seen, 0).abs().amax(1) + 4)
        count, pmax = seen.sum(1), p.amax(1)
        tol[:, i] = ((p @ vv.abs()) * (2.0 ** -11 + 2.0 ** -18 + 8 * 2.0 ** -22 + dz).view(-1, 1)
                     + (vsmax * count * 2.0 ** -24 * (14 * pmax + 2)).view(-1, 1))
    return out, tol


def seen_tokens(prefix, own, queries, causal, prefix_there=None, own_there=None):
    """[queries, prefix + own]: all of the prefix, and the own tokens up to each query's (causal) or all of them."""
    left = torch.ones(queries, prefix, dtype=torch.bool)
    right = torch.ones(queries, own, dtype=torch.bool)
    if causal:
        right = torch.arange(own).view(1, -1) <= (own - queries + torch.arange(queries)).view(-1, 1)
    if prefix_there is not None:
        left = left & torch.as_tensor(prefix_there).view(1, -1)
    if own_there is not None:
        right = right & torch.as_tensor(own_there).view(1, -1)
    return torch.cat((left, right), 1)
