"""What is measured of the operators for many requests at once.

A server that decodes a large batch leaves the range where 4-bit weights save
time (the products become bound by arithmetic, not by the weights' bytes), and
its requests often begin with the same text.  For it stand beside the INT4
layer and the 4-bit cache:

  quantise   rows to 8-bit floats (e4m3), one FP32 scale per row and group of
             128 columns
  linear     y = x W^T (+ bias) on 8-bit floats: W with one FP32 scale per block
             of 128 x 128, x quantised as above (or codes already), the input
             activation of an FFN's second projection fused
  prefix     attention over the paged 4-bit cache for requests that share a long
             prefix: the prefix's tokens are met once for all of a group, then
             each request's own

run() computes them in their plain form with elementary torch operations, or,
where `own` is true, with the framework's kernels.

Quantization: s = fl32(max|x| / 448), the code is fl32(x / s) rounded to the
nearest e4m3 value, ties to even; a group of zeros has s = 0 and codes 0.

The cache is the one of perf/operators.py: uint8 [pages, kv heads, region]; with
P tokens a page, D channels, W = min(D, 128) and NB = D / W a region holds

  bytes [0, PD/2)         codes of keys: 16-token chunk c and block b at
                          (c NB + b) 8W; in it the token t and quarter kq own
                          W/8 bytes at (16 kq + t) W/8: word s holds channels
                          W b + 32 s + 8 kq + j, nibble j/2 for even j and
                          4 + j/2 for odd j
  bytes [PD/2, PD)        codes of values, in the same chunks; the lane l (0..15)
                          and quarter kq own W/8 bytes at (16 kq + l) W/8: word
                          2 h + a holds tokens 4 kq + 2 a (low half) and
                          4 kq + 2 a + 1 (high half), nibble i of a half being
                          channel W b + (W/16) l + 4 h + i
  then FP32 scales        of keys [NB][P], of values [NB][P]

with codes u = q + 8, q in [-7, 7].
"""
import math
import random

import torch

own = False

BF16, F16 = "bf16", "f16"
LARGEST = 4096 * 2048 * 32768  # products of the largest listed linear


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decoding token before the qkv projection
        dict(name="quantise 1 row", op="quantise", dtype=BF16, rows=1, k=2048, pad=0),
        # a mixed batch, the rows a part of wider ones
        dict(name="quantise 777 rows", op="quantise", dtype=F16, rows=777, k=4096, pad=64),
        # the activated input of a long prompt's down projection
        dict(name="quantise 8192 rows", op="quantise", dtype=BF16, rows=8192, k=16384, pad=0),
        # one decoding token on the gate and up projection
        dict(name="linear 1 row", op="linear", dtype=BF16, rows=1, n=32768, k=2048, bias=False, act="none", codes=False),
        # a decoding batch on the down projection, SwiGLU fused into its input
        dict(name="linear 64 rows swiglu", op="linear", dtype=BF16, rows=64, n=2048, k=16384, bias=False, act="swiglu", codes=False),
        # prompt pieces beside decoding rows, odd sizes, biased
        dict(name="linear 333 rows", op="linear", dtype=F16, rows=333, n=4100, k=4096, bias=True, act="none", codes=False),
        # rows that arrive quantised (from another rank, say)
        dict(name="linear 1024 rows of codes", op="linear", dtype=BF16, rows=1024, n=2560, k=2048, bias=False, act="none", codes=True),
        # a long prompt on the gate and up projection
        dict(name="linear 4096 rows", op="linear", dtype=BF16, rows=4096, n=32768, k=2048, bias=False, act="none", codes=False),
        # two requests on one prompt of images and instructions
        dict(name="prefix 2 on 800", op="prefix", dtype=BF16, groups=1, batch=2, heads=8, kv_heads=1, dim=256, page=16, q_min=1,
             q_max=1, prefix_min=800, prefix_max=800, own_min=1, own_max=60, causal=True, lens=0),
        # a decoding batch on one system prompt
        dict(name="prefix 64 on 8192", op="prefix", dtype=BF16, groups=1, batch=64, heads=32, kv_heads=8, dim=128, page=64, q_min=1,
             q_max=1, prefix_min=8192, prefix_max=8192, own_min=0, own_max=512, causal=True, lens=1),
        # several documents with many questions each
        dict(name="prefix 4 x 48 on 32768", op="prefix", dtype=BF16, groups=4, batch=192, heads=32, kv_heads=8, dim=128, page=128,
             q_min=1, q_max=1, prefix_min=20000, prefix_max=32768, own_min=1, own_max=1000, causal=True, lens=2),
        # questions of many tokens beside decoding rows, no shared heads
        dict(name="prefix pieces 24 on 3000", op="prefix", dtype=F16, groups=2, batch=24, heads=16, kv_heads=16, dim=64, page=32,
             q_min=1, q_max=150, prefix_min=1000, prefix_max=3000, own_min=0, own_max=400, causal=True, lens=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice([BF16, F16])
    op = rng.choice(["quantise", "linear", "linear", "prefix", "prefix"])
    if op == "quantise":
        k = 128 * _log(rng, 1, 128)
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, min(32768, 8192 * 16384 // k)), k=k, pad=rng.choice([0, 0, 8, 128]))
    if op == "linear":
        rows, n, k = _log(rng, 1, 4096), _log(rng, 100, 32768), 128 * _log(rng, 1, 128)
        while rows * n * k > LARGEST:
            rows, n, k = rows // 2 + 1, n // 2 + 50, 128 * (k // 256 + 1)
        codes = rng.random() < 0.2
        return dict(op=op, dtype=dtype, rows=rows, n=n, k=k, bias=rng.random() < 0.4,
                    act="none" if codes else rng.choice(["none", "none", "swiglu", "gelu_tanh"]), codes=codes)
    dim, kv_heads = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
    groups = _log(rng, 1, 4)
    pieces = rng.random() < 0.4
    batch = groups + (_log(rng, 1, 24) if pieces else _log(rng, 1, 190))
    # the plain form's scores of one group fit
    most = _log(rng, 300, 4000 if pieces else max(600, min(32768, (1 << 28) // (batch * heads), (1 << 24) // (kv_heads * dim // 64))))
    own_max = _log(rng, 1, 400 if pieces else 1000)
    return dict(op=op, dtype=dtype, groups=groups, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim,
                page=rng.choice([16, 32, 48, 64, 128]), q_min=1, q_max=rng.choice([7, 40, 150]) if pieces else 1,
                prefix_min=rng.choice([0, most // 2, most]), prefix_max=most, own_min=rng.choice([0, 1, own_max]), own_max=own_max,
                causal=rng.random() < 0.8, lens=rng.randint(0, 1 << 30))


def _lengths(case):
    """Prefix lengths, the first request of each group, query and own lengths of each request, the same for every seed."""
    r = random.Random(case["lens"])
    prefix = [r.randint(case["prefix_min"], case["prefix_max"]) for _ in range(case["groups"])]
    cuts = sorted(r.sample(range(1, case["batch"]), case["groups"] - 1))
    first = [0, *cuts, case["batch"]]
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["batch"])]
    mine = [r.randint(case["own_min"], case["own_max"]) for _ in range(case["batch"])]
    if case["q_max"] > 1:  # query tokens are in the cache themselves
        mine = [max(a, b) for a, b in zip(q, mine)]
    return prefix, first, q, mine


# ---------------------------------------------------------------------------
# the cache's layout, whole pages at a time
# ---------------------------------------------------------------------------


def _geometry(dim):
    w = min(dim, 128)
    return w, dim // w


def _fill(data, page, dim, gen, spread):
    """Quantized normal keys and values in every token of the cache."""
    pages, hk, _ = data.shape
    w, nb = _geometry(dim)
    c = page // 16
    some = max(1, (1 << 27) // (hk * page * dim))
    for p in range(0, pages, some):
        d = data[p:p + some]
        n = d.shape[0]
        for which in (0, 1):
            x = torch.randn(n, hk, page, nb, w, generator=gen, device=data.device)
            x *= spread[which].view(hk, 1, nb, w)
            s = x.abs().amax(-1) / 7.0
            u = (torch.round(x / s.unsqueeze(-1)).clamp_(-7, 7) + 8.0).to(torch.uint8)
            if which == 0:
                u = u.view(n, hk, c, 16, nb, w // 32, 4, 2, 2, 2).permute(0, 1, 2, 4, 6, 3, 5, 9, 7, 8)
            else:
                u = u.view(n, hk, c, 4, 2, 2, nb, 16, w // 64, 2, 2).permute(0, 1, 2, 6, 3, 7, 8, 4, 5, 9, 10)
            b = (u[..., 0] | (u[..., 1] << 4)).reshape(n, hk, page * dim // 2)
            d[:, :, which * page * dim // 2:(which + 1) * page * dim // 2] = b
            at = page * dim + which * 4 * page * nb
            d[:, :, at:at + 4 * page * nb] = s.permute(0, 1, 3, 2).contiguous().view(torch.uint8).view(n, hk, 4 * nb * page)


def _values(d, page, dim):
    """Keys and values [pages, heads, page, dim] in 32 bits of whole pages."""
    n, hk, _ = d.shape
    w, nb = _geometry(dim)
    c = page // 16
    got = []
    for which in (0, 1):
        b = d[:, :, which * page * dim // 2:(which + 1) * page * dim // 2]
        u = torch.stack((b & 15, b >> 4), -1)
        if which == 0:
            u = u.view(n, hk, c, nb, 4, 16, w // 32, 2, 2, 2).permute(0, 1, 2, 5, 3, 6, 4, 8, 9, 7)
        else:
            u = u.view(n, hk, c, nb, 4, 16, w // 64, 2, 2, 2, 2).permute(0, 1, 2, 4, 7, 8, 3, 5, 6, 9, 10)
        at = page * dim + which * 4 * page * nb
        s = d[:, :, at:at + 4 * page * nb].contiguous().view(torch.float32).view(n, hk, nb, page).transpose(2, 3)
        got.append((u.reshape(n, hk, page, nb, w).float() - 8.0).mul_(s.unsqueeze(-1)).view(n, hk, page, dim))
    return got


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _weight(n, k, gen, dev):
    """Codes [n, k] and scales [blocks of 128 rows, blocks of 128 columns] of normal weights."""
    rows, cols = -(-n // 128), k // 128
    w = torch.randn(rows * 128, k, generator=gen, device=dev) * k ** -0.5
    w[n:] = 0
    blocks = w.view(rows, 128, cols, 128)
    s = blocks.abs().amax((1, 3)) / 448.0
    codes = (blocks / s.view(rows, 1, cols, 1)).view(rows * 128, k)[:n].to(torch.float8_e4m3fn)
    return codes.contiguous(), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 29)
    dt = _dtype(case)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    if case["op"] in ("quantise", "linear"):
        m, k = case["rows"], case["k"]
        # channels of unlike size, some of them large, as hidden states have
        size = torch.exp(0.5 * randn(k))
        size[torch.rand(k, generator=g, device=dev) < 0.01] *= 20
    if case["op"] == "quantise":
        x = (randn(m, k + case["pad"]) * torch.nn.functional.pad(size, (0, case["pad"]), value=1.0)).to(dt)
        return dict(case=case, x=x[:, :k])
    if case["op"] == "linear":
        n = case["n"]
        codes, scales = _weight(n, k, g, dev)
        bias = (0.1 * randn(n)).to(dt) if case["bias"] else None
        x, x_scales = randn(m, k) * size, None
        if case["act"] == "swiglu":
            x = torch.cat((x, randn(m, k)), 1)
        if case["codes"]:
            groups = x.view(m, k // 128, 128)
            x_scales = groups.abs().amax(-1) / 448.0
            x = (groups / x_scales.unsqueeze(-1)).view(m, k).to(torch.float8_e4m3fn)
        else:
            x = x.to(dt)
        return dict(case=case, x=x, x_scales=x_scales, codes=codes, scales=scales, bias=bias)
    prefix, first, q_lens, mine = _lengths(case)
    d, page, hk = case["dim"], case["page"], case["kv_heads"]
    lens = prefix + mine
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 1
    pool = torch.empty(pages, hk, page * d + 8 * page * (d // min(d, 128)), dtype=torch.uint8, device=dev)
    # keys with channels of unlike size, as keys have
    spread = (torch.exp(0.5 * randn(hk, d)), torch.exp(0.2 * randn(hk, d)))
    _fill(pool, page, d, g, spread)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    tables, at = [], 0
    for part in (used[:len(prefix)], used[len(prefix):]):
        table = torch.full((len(part), max(max(part), 1)), -1, dtype=torch.int32, device=dev)
        for i, n in enumerate(part):
            table[i, :n] = order[at:at + n]
            at += n
        tables.append(table)
    # what lies behind a sequence's last token was never written
    scales = pool[:, :, page * d:].view(torch.float32).view(pages, hk, -1, page)
    for table, part in zip(tables, (prefix, mine)):
        for i, n in enumerate(part):
            if n % page:
                scales[int(table[i, n // page]), :, :, n % page:] = float("nan")
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    cu = [sum(q_lens[:i]) for i in range(len(q_lens) + 1)]
    return dict(case=case, q=(1.5 * randn(cu[-1], case["heads"], d)).to(dt), pool=pool, prefix_table=tables[0], prefix_lens=ints(prefix),
                table=tables[1], kv_lens=ints(mine), cu_q=ints(cu) if case["q_max"] > 1 else None,
                cu_groups=ints(first) if case["groups"] > 1 else None)


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------


def run(state):
    case = state["case"]
    if own:
        import weight_only_int4_rtn_amd as w4
        if case["op"] == "quantise":
            codes, scales = w4.quantize_fp8(state["x"])
            return {"codes": codes, "scales": scales}
        if case["op"] == "linear":
            act = {"none": w4.Act.NONE, "swiglu": w4.Act.SWIGLU, "gelu_tanh": w4.Act.GELU_TANH}[case["act"]]
            return w4.linear_fp8(state["x"], state["codes"], state["scales"], bias=state["bias"], act=act, x_scales=state["x_scales"],
                                 out_dtype=_dtype(case))
        return w4.kv4_prefix_attention(state["q"], state["pool"], state["prefix_table"], state["prefix_lens"], state["table"],
                                       state["kv_lens"], cu_q=state["cu_q"], cu_groups=state["cu_groups"], causal=case["causal"])
    return {"quantise": _plain_quantise, "linear": _plain_linear, "prefix": _plain_prefix}[case["op"]](state)


def _quantised(x):
    """e4m3 codes and scales of rows x, the quotients in 64 bits, then rounded: ties decide codes."""
    groups = x.unflatten(-1, (-1, 128))
    s = (groups.abs().amax(-1).double() / 448.0).float()
    z = (groups.double() / s.double().unsqueeze(-1)).float()
    z = torch.where((s == 0).unsqueeze(-1), 0.0, z.clamp(-448, 448))
    return z.flatten(-2).to(torch.float8_e4m3fn), s


def _plain_quantise(state):
    codes, scales = _quantised(state["x"].float())
    return {"codes": codes, "scales": scales}


def _plain_linear(state):
    case, x, s = state["case"], state["x"], state["x_scales"]
    if not case["codes"]:
        v = x.float()
        if case["act"] == "swiglu":
            up, gate = v.chunk(2, 1)
            v = up * (gate / (1.0 + torch.exp(-gate)))
        elif case["act"] == "gelu_tanh":
            v = v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
        x, s = _quantised(v.to(x.dtype).float())
    a = (x.float().unflatten(1, (-1, 128)) * s.unsqueeze(-1)).flatten(1)
    codes, n = state["codes"], case["n"]
    b = codes.float().unflatten(1, (-1, 128)) * state["scales"].repeat_interleave(128, 0)[:n].unsqueeze(-1)
    y = a @ b.flatten(1).t()
    if state["bias"] is not None:
        y = y + state["bias"].float()
    return y.to(_dtype(case))


def _plain_prefix(state):
    case, q, pool = state["case"], state["q"], state["pool"]
    prefix, first, q_lens, mine = _lengths(case)
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    share = case["heads"] // hk
    out = torch.empty_like(q)
    at = 0
    for j, n in enumerate(prefix):
        count = first[j + 1] - first[j]
        counts = torch.tensor(q_lens[first[j]:first[j + 1]], device=q.device)
        lens = state["kv_lens"][first[j]:first[j + 1]]
        rows = int(sum(q_lens[first[j]:first[j + 1]]))
        most = max(q_lens[first[j]:first[j + 1]])
        x = q[at:at + rows].float() / math.sqrt(d)
        # the prefix, one product for all of the group's rows
        k, v = _values(pool[state["prefix_table"][j].clamp(min=0).long()], page, d)
        k, v = (t.transpose(0, 1).reshape(hk, -1, d)[:, :n] for t in (k, v))
        xs = x.view(rows, hk, share, d).permute(1, 2, 0, 3).reshape(hk, share * rows, d)
        near = (xs @ k.transpose(1, 2)).view(hk, share, rows, n)
        # own tokens, padded to the longest request's rows
        own_k, own_v = _values(pool[state["table"][first[j]:first[j + 1]].clamp(min=0).long().flatten()], page, d)
        own_k, own_v = (t.view(count, -1, hk, page, d).transpose(1, 2).reshape(count, hk, -1, d) for t in (own_k, own_v))
        tokens = torch.arange(own_k.shape[2], device=q.device)
        inside = tokens < lens.view(-1, 1)
        own_v = torch.where(inside.view(count, 1, -1, 1), own_v, 0.0)
        slot = torch.arange(most, device=q.device)
        real = slot < counts.view(-1, 1)
        begin = torch.cumsum(counts, 0) - counts
        padded = x[(begin.view(-1, 1) + slot).clamp(max=rows - 1)].view(count, most, hk, share, d).permute(0, 2, 3, 1, 4)
        far = (padded.reshape(count, hk, share * most, d) @ own_k.transpose(2, 3)).view(count, hk, share, most, -1)
        seen = inside.view(count, 1, -1).expand(count, most, -1)
        if case["causal"]:
            seen = seen & (tokens <= (lens.view(-1, 1) - counts.view(-1, 1) + slot).unsqueeze(-1))
        far = torch.where(seen.view(count, 1, 1, most, -1), far, float("-inf"))
        far = far.permute(0, 3, 1, 2, 4)[real]  # [rows, hk, share, tokens]
        near = near.permute(2, 0, 1, 3)
        top = far.amax(-1, keepdim=True)
        if n:
            top = torch.maximum(top, near.amax(-1, keepdim=True))
        top = torch.where(torch.isinf(top), 0.0, top)
        near, far = torch.exp(near - top), torch.exp(far - top)
        total = near.sum(-1, keepdim=True) + far.sum(-1, keepdim=True)
        o = (near.permute(1, 2, 0, 3).reshape(hk, share * rows, n) @ v).view(hk, share, rows, d).permute(2, 0, 1, 3)
        wide = torch.zeros(count, most, hk, share, far.shape[-1], device=q.device)
        wide[real] = far
        wide = wide.permute(0, 2, 3, 1, 4).reshape(count, hk, share * most, -1) @ own_v
        o = o + wide.view(count, hk, share, most, d).permute(0, 3, 1, 2, 4)[real]
        out[at:at + rows] = torch.where(total > 0, o / total, 0.0).reshape(rows, hk * share, d).to(q.dtype)
        at += rows
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    if case["op"] == "quantise":
        m, k = case["rows"], case["k"]
        return {"bytes": m * (3 * k + 4 * (k // 128)), "flops": 3 * m * k}
    if case["op"] == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        x = m * (k + 4 * (k // 128)) if case["codes"] else 2 * m * k * (2 if case["act"] == "swiglu" else 1)
        return {"bytes": x + n * k + 4 * -(-n // 128) * (k // 128) + 2 * m * n + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    prefix, first, q_lens, mine = _lengths(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    pairs = 0
    for j, n in enumerate(prefix):
        for c, m in zip(q_lens[first[j]:first[j + 1]], mine[first[j]:first[j + 1]]):
            pairs += c * n + (sum(max(0, m - c + i + 1) for i in range(c)) if case["causal"] else c * m)
    token = hk * (d + 8 * (d // min(d, 128)))
    return {"bytes": (sum(prefix) + sum(mine)) * token + 4 * sum(q_lens) * hq * d, "flops": 4 * pairs * hq * d}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    state = prepare(case, seed)
    return {"quantise": _exact_quantise, "linear": _exact_linear, "prefix": _exact_prefix}[case["op"]](state)


def _nearest_e4m3(z):
    """The nearest value of e4m3 (3 bits behind the point, exponents from -6, at most 448), ties to even, of 64-bit z."""
    _, e = torch.frexp(z)
    exponent = torch.clamp(e.long() - 1, min=-6) - 3
    step = ((exponent + 1023) << 52).view(torch.float64)  # 2^exponent, exactly
    return (torch.round(z / step) * step).clamp(-448.0, 448.0)


def _exact_rows(v):
    """Codes' values and scales of rows v (64 bits) with the definition's two roundings to 32 bits, the scale's and the quotient's."""
    part = v.unflatten(-1, (v.shape[-1] // 128, 128))
    s = (part.abs().amax(-1, keepdim=True) / 448.0).float().double()
    quotient = torch.where(s > 0, part / torch.where(s > 0, s, 1.0), 0.0).float().double()
    return _nearest_e4m3(quotient), s


def _exact_quantise(state):
    codes, s = _exact_rows(state["x"].double())
    return {"codes": codes.flatten(-2), "scales": s.squeeze(-1)}


def _exact_linear(state):
    case, x = state["case"], state["x"]
    if case["codes"]:
        a = x.double().unflatten(-1, (-1, 128)) * state["x_scales"].double().unsqueeze(-1)
    else:
        v = x.double()
        if case["act"] == "swiglu":
            v = v[:, :case["k"]] * v[:, case["k"]:] * torch.sigmoid(v[:, case["k"]:])
        elif case["act"] == "gelu_tanh":
            v = 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
        codes, s = _exact_rows(v.to(x.dtype).double())
        a = codes * s
    a = a.flatten(-2)
    y = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device=x.device)
    for i in range(0, case["n"], 128):
        w = state["codes"][i:i + 128].double().unflatten(-1, (-1, 128)) * state["scales"][i // 128].double().view(1, -1, 1)
        y[:, i:i + 128] = a @ w.flatten(-2).t()
    return y if state["bias"] is None else y + state["bias"].double()


def _exact_prefix(state):
    case = state["case"]
    prefix, first, q_lens, mine = _lengths(case)
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    if work(case)["flops"] > 3e12:
        return None
    share, w = hq // hk, min(d, 128)
    dev = state["q"].device
    flat = state["pool"]
    ch = torch.arange(d, device=dev)
    cb, cw = ch // w, ch % w

    def side(table, n, head, which):
        """Values of one head's n tokens, byte by byte from the layout."""
        tok = torch.arange(n, device=dev)
        pg, t = table[tok // page].long().view(-1, 1), (tok % page).view(-1, 1)
        c, i = t // 16, t % 16
        if which == 0:
            word = (16 * (cw % 32 // 8) + i) * (w // 32) + cw // 32
            j = cw % 8
            nibble = j // 2 + 4 * (j % 2) + 0 * word
        else:
            lane, r = cw // (w // 16), cw % (w // 16)
            word = (16 * (i // 4) + lane) * (w // 32) + 2 * (r // 4) + i % 4 // 2
            nibble = 4 * (i % 2) + r % 4
        byte = which * page * d // 2 + (c * (d // w) + cb) * 8 * w + 4 * word + nibble // 2
        code = ((flat[pg, head, byte].int() >> (4 * (nibble % 2))) & 15).double() - 8.0
        at = page * d + 4 * (which * page * (d // w) + cb * page + t)
        scale = torch.stack([flat[pg, head, at + b] for b in range(4)], -1).view(torch.float32).squeeze(-1).double()
        return code * scale

    out = torch.zeros(sum(q_lens), hq, d, dtype=torch.float64, device=dev)
    for head in range(hk):
        begin = 0
        for j, n in enumerate(prefix):
            ks, vs = (side(state["prefix_table"][j], n, head, i) for i in (0, 1))
            for b in range(first[j], first[j + 1]):
                c, m = q_lens[b], mine[b]
                k, v = (torch.cat((p, side(state["table"][b], m, head, i))) for i, p in ((0, ks), (1, vs)))
                x = state["q"][begin:begin + c, head * share:(head + 1) * share].double().transpose(0, 1)
                logits = (x @ k.t()) * d ** -0.5
                if case["causal"]:
                    last = n + m - c + torch.arange(c, device=dev).view(-1, 1)
                    logits = logits.masked_fill((torch.arange(n + m, device=dev) >= n) & (torch.arange(n + m, device=dev) > last), -torch.inf)
                if n + m:
                    p = torch.softmax(logits, -1).nan_to_num(0.0)
                    out[begin:begin + c, head * share:(head + 1) * share] = (p @ v).transpose(0, 1)
                begin += c
    return out
