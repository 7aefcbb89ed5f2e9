"""What is measured of the serving operators beside the quantized linear layer.

Three operators of one decoder layer in serving, around its INT4 projections:

  append     the rotation of queries and keys by position, the round-to-nearest
             INT4 quantization of keys and values (one FP32 scale per token,
             head and group of up to 128 channels) and their store into a paged
             cache; then the read-back of the same tokens from the cache, which
             gives the stored values in the model's type
  attention  softmax(q k^T) v over that cache, from one query token a request to
             whole prompts, with shared key heads, ragged lengths, causal masks
             and windows
  lora       low-rank adapters of many requests beside a shared projection:
             y + scale * (x A^T) B^T, each row with its own adapter or none

run() computes them in their plain form with elementary torch operations, or,
where `own` is true, with the framework's kernels.

The cache.  One uint8 tensor [pages, kv heads, region]; a region holds one
page (P tokens, a multiple of 16) of one head.  With D channels a head,
W = min(D, 128) and NB = D / W blocks:

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

Codes are offset-binary nibbles u = q + 8, q in [-7, 7] (the quantizer of the
weights: s = fl32(max / 7), q = round_half_even(fl32(x / s))).
"""
import math
import random

import torch

own = False

BF16, F16 = "bf16", "f16"


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one token of one stream: the qkv projection of 2560 outputs, one key head of 256 channels
        dict(name="append 1 token", op="append", dtype=BF16, tokens=1, heads=8, kv_heads=1, dim=256, page=16, rot=256,
             interleaved=False, length=4096, padding=0),
        # a batch of decoding and short prompt tokens with padding rows, part of each head rotated, interleaved pairs
        dict(name="append 777 mixed", op="append", dtype=F16, tokens=777, heads=16, kv_heads=16, dim=64, page=32, rot=32,
             interleaved=True, length=32768, padding=9),
        # a long prompt
        dict(name="append 8192 prompt", op="append", dtype=BF16, tokens=8192, heads=32, kv_heads=8, dim=128, page=64,
             rot=128, interleaved=False, length=131072, padding=0),
        # one stream decoding on a short prefix
        dict(name="decode 1 x 1000", op="attention", dtype=BF16, batch=1, heads=8, kv_heads=1, dim=256, page=16,
             q_min=1, q_max=1, kv_min=1000, kv_max=1000, causal=True, window=0, lens=0),
        # a serving batch: ragged lengths, one of them empty
        dict(name="decode 64 ragged", op="attention", dtype=BF16, batch=64, heads=32, kv_heads=8, dim=128, page=64,
             q_min=1, q_max=1, kv_min=0, kv_max=8192, causal=True, window=0, lens=1),
        # a few requests with very long contexts
        dict(name="decode 4 x 131072", op="attention", dtype=BF16, batch=4, heads=32, kv_heads=8, dim=128, page=128,
             q_min=1, q_max=1, kv_min=131072, kv_max=131072, causal=True, window=0, lens=2),
        # one action chunk over its image and text prefix, every token seeing every other
        dict(name="action chunk 50", op="attention", dtype=BF16, batch=1, heads=8, kv_heads=1, dim=256, page=16,
             q_min=50, q_max=50, kv_min=1074, kv_max=1074, causal=False, window=0, lens=3),
        # prompts in pieces beside decoding requests, sliding window, no shared heads
        dict(name="mixed 12 windowed", op="attention", dtype=F16, batch=12, heads=16, kv_heads=16, dim=64, page=32,
             q_min=1, q_max=300, kv_min=300, kv_max=3000, causal=True, window=1024, lens=4),
        # a whole prompt
        dict(name="prompt 4096", op="attention", dtype=BF16, batch=1, heads=32, kv_heads=8, dim=128, page=64,
             q_min=4096, q_max=4096, kv_min=4096, kv_max=4096, causal=True, window=0, lens=5),
        # one token on the qkv projection
        dict(name="lora 1 row", op="lora", dtype=BF16, rows=1, n=2560, k=2048, adapters=4, rank=16, run=1, none=0.0),
        # a decoding batch, each row its own adapter, some without
        dict(name="lora 64 rows", op="lora", dtype=BF16, rows=64, n=4096, k=4096, adapters=48, rank=16, run=1, none=0.1),
        # prompts of several requests in one batch, on the gate and up projection
        dict(name="lora 4099 rows", op="lora", dtype=F16, rows=4099, n=32768, k=2048, adapters=6, rank=64, run=700, none=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice([BF16, F16])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16])
    page = rng.choice([16, 32, 48, 64, 128])
    op = rng.choice(["append", "attention", "attention", "lora"])
    if op == "append":
        tokens = _log(rng, 1, 8192)
        heads, kv_heads = min(heads, 32), kv_heads if heads <= 32 else 2
        return dict(op=op, dtype=dtype, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=min(dim, 128) if tokens > 4000 else dim,
                    page=page, rot=16 * rng.randint(0, min(dim, 128) // 16), interleaved=rng.random() < 0.5,
                    length=_log(rng, 2048, 131072), padding=rng.choice([0, 0, 5]))
    if op == "lora":
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, 4099), n=_log(rng, 100, 16384), k=128 * _log(rng, 4, 64),
                    adapters=rng.randint(1, 48), rank=8 * _log(rng, 1, 16), run=_log(rng, 1, 700), none=rng.choice([0.0, 0.1, 0.5]))
    if rng.random() < 0.6:  # one query token a request
        batch = _log(rng, 1, 64)
        most = _log(rng, 1, min(131072, 524288 // batch // max(1, kv_heads // 8) // (dim // 64)))
        q_min = q_max = 1
    else:
        batch = _log(rng, 1, 12)
        q_max = _log(rng, 2, max(2, 2048 // batch))
        q_min = rng.choice([1, q_max])
        most = q_max + _log(rng, 1, 2048)
    return dict(op=op, dtype=dtype, batch=batch, heads=min(heads, 4 * kv_heads) if q_max > 64 else heads, kv_heads=kv_heads, dim=dim,
                page=page, q_min=q_min, q_max=q_max, kv_min=rng.choice([0, most // 2, most]), kv_max=most,
                causal=rng.random() < 0.75, window=rng.choice([0, 0, 0, max(1, most // 3)]), lens=rng.randint(0, 1 << 30))


def _lengths(case):
    """Query and cache lengths of each request, the same for every seed."""
    r = random.Random(case["lens"])
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["batch"])]
    kv = [r.randint(case["kv_min"], case["kv_max"]) for _ in range(case["batch"])]
    if case["q_max"] > 1:  # prompt tokens are in the cache themselves
        kv = [max(a, b) for a, b in zip(q, kv)]
    if case["batch"] > 8:  # the longest and the shortest are there
        kv[0], kv[1] = max(kv[0], case["kv_max"]), max(case["kv_min"], q[1] if case["q_max"] > 1 else 0)
    return q, kv


# ---------------------------------------------------------------------------
# the cache's layout, all bytes of whole pages at a time
# ---------------------------------------------------------------------------


def _geometry(dim):
    w = min(dim, 128)
    return w, dim // w


def _region(page, dim):
    return page * dim + 8 * page * (dim // min(dim, 128))


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
    """Keys and values [pages, heads, page, dim] in 32 bits, and their scales as stored, of whole pages."""
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


def _offsets(tokens, page, dim, device):
    """Byte offsets inside a region of a token's key words [T, NB, 4, W/8], value half-words [T, NB, 16, W/64, 2] and
    scales [T, 2, NB, 4]."""
    w, nb = _geometry(dim)
    r = lambda n: torch.arange(n, device=device)  # noqa: E731
    c, t = (tokens // 16).view(-1, 1, 1, 1), (tokens % 16).view(-1, 1, 1, 1)
    k = (c * nb + r(nb).view(1, -1, 1, 1)) * 8 * w + (16 * r(4).view(1, 1, -1, 1) + t) * (w // 8) + r(w // 8)
    c, t = c.unsqueeze(-1), t.unsqueeze(-1)
    v = (page * dim // 2 + (c * nb + r(nb).view(1, -1, 1, 1, 1)) * 8 * w + (16 * (t // 4) + r(16).view(1, 1, -1, 1, 1)) * (w // 8)
         + 8 * r(w // 64).view(1, 1, 1, -1, 1) + 4 * (t % 4 // 2) + 2 * (t % 2) + r(2))
    s = page * dim + 4 * (page * r(2 * nb).view(1, 2, nb, 1) + tokens.view(-1, 1, 1, 1)) + r(4)
    return k, v, s


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 17)
    dt = _dtype(case)
    randn = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    if case["op"] == "append":
        t, d, page = case["tokens"], case["dim"], case["page"]
        pages = -(-t // page) + 2
        heads = case["heads"] + 2 * case["kv_heads"]
        qkv = (randn(t, heads, d) * torch.exp(0.5 * randn(1, heads, d))).view(t, heads * d).to(dt)
        order = torch.randperm(pages, generator=g, device=dev)
        at = torch.arange(t, device=dev) + min(3, page - 1)
        slots = order[at // page] * page + at % page
        if case["padding"]:
            slots[case["padding"] // 2::case["padding"]] = -1
        rope = None
        if case["rot"]:
            inv = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
            angle = torch.arange(case["length"], device=dev, dtype=torch.float64)[:, None] * inv
            rope = torch.cat((angle.cos(), angle.sin()), 1).float()
        first = int(torch.randint(0, max(1, case["length"] - t), (1,), generator=g, device=dev))
        positions = ((first + torch.arange(t, device=dev)) % case["length"]).to(torch.int32)
        pool = torch.zeros(pages, case["kv_heads"], _region(page, d), dtype=torch.uint8, device=dev)
        return dict(case=case, qkv=qkv, pool=pool, slots=slots, positions=positions, rope=rope)
    if case["op"] == "lora":
        m, n, k, l, r = (case[x] for x in ("rows", "n", "k", "adapters", "rank"))
        x, y = randn(m, k).to(dt), randn(m, n).to(dt)
        a, b = (randn(l, r, k) / math.sqrt(k)).to(dt), (randn(l, n, r) / math.sqrt(r)).to(dt)
        runs = -(-m // case["run"])
        index = torch.randint(0, l, (runs,), generator=g, device=dev, dtype=torch.int32)
        index[torch.rand(runs, generator=g, device=dev) < case["none"]] = -1
        index = index.repeat_interleave(case["run"])[:m].contiguous()
        scales = 0.5 + torch.rand(l, generator=g, device=dev)
        return dict(case=case, x=x, y=y, a=a, b=b, index=index, scales=scales)
    q_lens, kv_lens = _lengths(case)
    d, page, hk = case["dim"], case["page"], case["kv_heads"]
    used = [-(-n // page) for n in kv_lens]
    pages = sum(used) + 1
    pool = torch.empty(pages, hk, _region(page, d), dtype=torch.uint8, device=dev)
    # keys with channels of unlike size, as keys have
    spread = (torch.exp(0.5 * randn(hk, d)), torch.exp(0.2 * randn(hk, d)))
    _fill(pool, page, d, g, spread)
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(used), max(max(used), 1) + 1), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    # what lies behind a request's last token was never written
    scales = pool[:, :, page * d:].view(torch.float32).view(pages, hk, -1, page)
    for i, n in enumerate(kv_lens):
        if n % page:
            scales[int(table[i, n // page]), :, :, n % page:] = float("nan")
    q = (1.5 * randn(sum(q_lens), case["heads"], d)).to(dt)
    cu = torch.tensor([sum(q_lens[:i]) for i in range(len(q_lens) + 1)], dtype=torch.int32, device=dev)
    return dict(case=case, q=q, pool=pool, table=table, kv_lens=torch.tensor(kv_lens, dtype=torch.int32, device=dev),
                cu_q=cu if case["q_max"] > 1 else None, q_most=max(q_lens))


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------


def run(state):
    case = state["case"]
    if own:
        import weight_only_int4_rtn_amd as w4
        if case["op"] == "append":
            q = w4.kv4_append(state["qkv"], state["pool"], state["slots"], case["dim"], positions=state["positions"],
                              rope=state["rope"], interleaved=case["interleaved"])
            k, v = w4.kv4_read(state["pool"], state["slots"], case["dim"], dtype=state["qkv"].dtype)
            return {"q": q, "k": k, "v": v}
        if case["op"] == "attention":
            return w4.kv4_attention(state["q"], state["pool"], state["table"], state["kv_lens"], cu_q=state["cu_q"],
                                    causal=case["causal"], window=case["window"])
        return w4.lora_add(state["y"], state["x"], state["a"], state["b"], state["index"], scales=state["scales"])
    return {"append": _plain_append, "attention": _plain_attention, "lora": _plain_lora}[case["op"]](state)


def _rotate(x, rope, positions, interleaved):
    if rope is None:
        return x
    rot = rope.shape[1]
    half = rot // 2
    row = rope[positions.long()].unsqueeze(1)
    cos, sin = row[..., :half], row[..., half:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_append(state):
    case, qkv, pool, slots = state["case"], state["qkv"], state["pool"], state["slots"]
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    w, nb = _geometry(d)
    x = qkv.float().view(-1, hq + 2 * hk, d)
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    q, k = (_rotate(z, state["rope"], state["positions"], case["interleaved"]) for z in (q, k))
    kv = torch.stack((k, v), 1).view(-1, 2, hk, nb, w)
    # quotients in 64 bits, then rounded: the definition's correctly rounded 32-bit divisions, whose ties decide codes
    s = (kv.abs().amax(-1).double() / 7.0).float()
    z = (kv.double() / s.double().unsqueeze(-1)).float()
    u = torch.where((s == 0).unsqueeze(-1), 8.0, torch.round(z).clamp(-8, 7) + 8.0).to(torch.uint8)
    there = slots >= 0
    u, s, to = u[there], s[there], slots[there]
    rows = to // page
    at_k, at_v, at_s = _offsets(to % page, page, d, pool.device)
    n = to.shape[0]
    # words of keys (quarter, word, byte), half-words of values (lane, group, byte)
    uk = u[:, 0].view(n, hk, nb, w // 32, 4, 2, 2, 2).permute(0, 1, 2, 4, 3, 7, 5, 6)
    uv = u[:, 1].view(n, hk, nb, 16, w // 64, 2, 2)
    head = torch.arange(hk, device=pool.device)
    put = lambda at, b: pool.index_put_((rows.view([-1] + [1] * at.dim()), head.view([1, -1] + [1] * (at.dim() - 1)), at.unsqueeze(1)), b)  # noqa: E731
    put(at_k, (uk[..., 0] | (uk[..., 1] << 4)).reshape(n, hk, nb, 4, w // 8))
    put(at_v, uv[..., 0] | (uv[..., 1] << 4))
    put(at_s, s.permute(0, 2, 1, 3).contiguous().view(torch.uint8).view(n, hk, 2, nb, 4))
    # the same tokens read back
    get = lambda at: pool[rows.view([-1] + [1] * at.dim()), head.view([1, -1] + [1] * (at.dim() - 1)), at.unsqueeze(1)]  # noqa: E731
    bk, bv, bs = get(at_k), get(at_v), get(at_s)
    bk = torch.stack((bk & 15, bk >> 4), -1).view(n, hk, nb, 4, w // 32, 2, 2, 2).permute(0, 1, 2, 4, 3, 6, 7, 5).reshape(n, hk, nb, w)
    bv = torch.stack((bv & 15, bv >> 4), -1).view(n, hk, nb, w)
    bs = bs.contiguous().view(torch.float32).view(n, hk, 2, nb, 1)
    out = [torch.zeros(qkv.shape[0], hk, d, dtype=qkv.dtype, device=qkv.device) for _ in range(2)]
    for o, b, i in zip(out, (bk, bv), (0, 1)):
        o[there] = ((b.float() - 8.0) * bs[:, :, i]).view(n, hk, d).to(qkv.dtype)
    return {"q": q.to(qkv.dtype), "k": out[0], "v": out[1]}


def _plain_attention(state):
    case, q, pool, table, kv_lens, cu = (state[x] for x in ("case", "q", "pool", "table", "kv_lens", "cu_q"))
    hk, d, page, batch = case["kv_heads"], case["dim"], case["page"], case["batch"]
    share = case["heads"] // hk
    most = state["q_most"]
    table = table[:, :max(1, -(-case["kv_max"] // page), -(-most // page) if cu is not None else 1)]
    k, v = _values(pool[table.clamp(min=0).long().flatten()], page, d)
    k, v = (x.view(batch, -1, hk, page, d).transpose(1, 2).reshape(batch, hk, -1, d) for x in (k, v))
    tokens = torch.arange(k.shape[2], device=q.device)
    inside = tokens < kv_lens.view(-1, 1)
    v = torch.where(inside.view(batch, 1, -1, 1), v, 0.0)
    cu = torch.arange(batch + 1, device=q.device) if cu is None else cu.long()
    counts = cu[1:] - cu[:-1]
    rows = torch.arange(most, device=q.device)
    real = rows < counts.view(-1, 1)
    qs = q.float()[(cu[:-1].view(-1, 1) + rows).clamp(max=q.shape[0] - 1)]
    qs = qs.view(batch, most, hk, share, d).permute(0, 2, 3, 1, 4).reshape(batch, hk, share * most, d)
    seen = inside.view(batch, 1, -1).expand(batch, most, -1)
    position = (kv_lens.view(-1, 1) - counts.view(-1, 1) + rows).unsqueeze(-1)
    if case["causal"]:
        seen = seen & (tokens <= position)
    if case["window"]:
        seen = seen & (tokens > position - case["window"])
        if not case["causal"]:
            seen = seen & (tokens < position + case["window"])
    seen = seen.view(batch, 1, 1, most, -1)
    scores = ((qs / math.sqrt(d)) @ k.transpose(2, 3)).view(batch, hk, share, most, -1)
    scores = torch.where(seen, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(top), 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p.view(batch, hk, share * most, -1) @ v).view(batch, hk, share, most, d)
    out = torch.where(total > 0, out / total, 0.0)
    return out.permute(0, 3, 1, 2, 4).reshape(batch, most, hk * share, d)[real].to(q.dtype)


def _plain_lora(state):
    x, y, a, b, index, scales = (state[n] for n in ("x", "y", "a", "b", "index", "scales"))
    l, r, k = a.shape
    mine = index.view(-1, 1) == torch.arange(l, device=x.device)
    t = (x.float() @ a.float().view(l * r, k).t()).view(-1, l, r)
    t = t * (mine * scales).unsqueeze(-1)
    return (y.float() + t.view(-1, l * r) @ b.float().transpose(1, 2).reshape(l * r, -1)).to(y.dtype)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    if case["op"] == "append":
        t, hq, hk, d = (case[x] for x in ("tokens", "heads", "kv_heads", "dim"))
        stored = t * hk * (d + 8 * (d // min(d, 128)))
        return {"bytes": 2 * t * (hq + 2 * hk) * d + 2 * t * hq * d + 2 * stored + 4 * t * hk * d + 4 * t * case["rot"] + 20 * t,
                "flops": 3 * t * (hq + hk) * case["rot"] + 10 * t * hk * d}
    if case["op"] == "lora":
        m, n, k, l, r = (case[x] for x in ("rows", "n", "k", "adapters", "rank"))
        live = min(l, -(-m // case["run"]))
        some = m * (1 - case["none"])
        return {"bytes": 2 * live * r * (n + k) + 2 * m * k + 4 * m * n + 4 * m, "flops": 2 * some * r * (n + k)}
    q_lens, kv_lens = _lengths(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    flops = bytes_ = 0
    for n, m in zip(q_lens, kv_lens):
        first, pairs = m, 0
        for i in range(n):
            p = m - n + i
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            hi = min(m, p + 1) if case["causal"] else min(m, p + case["window"]) if case["window"] else m
            pairs += max(0, hi - lo)
            first = min(first, lo) if hi > lo else first
        flops += 4 * pairs * hq * d
        bytes_ += (m - first) * hk * (d + 8 * (d // min(d, 128))) + 4 * n * hq * d
    return {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    state = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "lora": _exact_lora}[case["op"]](state)


def _exact_append(state):
    case = state["case"]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    x = state["qkv"].double().view(-1, hq + 2 * hk, d)
    rot = case["rot"]
    if rot:
        turn = state["rope"].double()[state["positions"].long()]
        z = torch.complex(turn[:, :rot // 2], turn[:, rot // 2:]).unsqueeze(1)
        part = x[:, :hq + hk, :rot]
        pairs = part.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else part.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
        x[:, :hq + hk, :rot] = (turned if case["interleaved"] else turned.transpose(-1, -2)).flatten(-2)
    there = (state["slots"] >= 0).view(-1, 1, 1)
    got = {"q": x[:, :hq].clone()}
    for name, part in (("k", x[:, hq:hq + hk]), ("v", x[:, hq + hk:])):
        groups = part.unflatten(-1, (-1, min(d, 128)))
        # the definition's two roundings to 32 bits: the scale and the quotient, whose ties the code follows
        s = (groups.abs().amax(-1, keepdim=True) / 7.0).float().double()
        codes = torch.where(s > 0, torch.round((groups / s).float().double()), 0.0)
        got[name] = torch.where(there, (codes * s).flatten(-2), 0.0)
    return got


def _exact_attention(state):
    case = state["case"]
    q_lens, kv_lens = _lengths(case)
    hq, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    if sum(4 * n * m * hq * d for n, m in zip(q_lens, kv_lens)) > 4e12 or sum(kv_lens) * hk * d > 3e9:
        return None
    share, w = hq // hk, min(d, 128)
    nb = d // w
    dev = state["q"].device
    flat = state["pool"].view(state["pool"].shape[0], hk, -1)
    ch = torch.arange(d, device=dev)
    b, e = ch // w, ch % w
    # where channel `e` of block `b` lies: bytes and bits that do not depend on the token
    k_at, k_nib = b * 8 * w + (e % 32 // 8) * 2 * w + 4 * (e // 32), (e % 8 // 2) + 4 * (e % 2)
    per = w // 16
    v_at, v_nib = b * 8 * w + (e // per) * (w // 8) + 8 * (e % per // 4), e % 4
    out = torch.zeros_like(state["q"], dtype=torch.float64)
    row = 0
    for i, (n, m) in enumerate(zip(q_lens, kv_lens)):
        q = state["q"][row:row + n].double()
        token = torch.arange(m, device=dev)
        pages, t = state["table"][i].long()[token // page], token % page
        base = (t // 16 * nb * 8 * w).view(-1, 1)
        byte_k = base + (t % 16 * (w // 8)).view(-1, 1) + k_at + k_nib // 2
        byte_v = page * d // 2 + base + (2 * w * (t % 16 // 4) + 4 * (t % 4 // 2) + 2 * (t % 2)).view(-1, 1) + v_at + v_nib // 2
        position = m - n + torch.arange(n, device=dev).view(-1, 1)
        seen = torch.ones(n, m, dtype=torch.bool, device=dev)
        if case["causal"]:
            seen &= token <= position
        if case["window"]:
            seen &= (position - token).abs() < case["window"] if not case["causal"] else position - token < case["window"]
        for h in range(hk):
            if m == 0:
                continue
            region = flat[:, h]
            scale = region[:, page * d:].contiguous().view(torch.float32).view(-1, 2, nb, page)[pages, :, :, t].double()
            k, v = (((region[pages.view(-1, 1), at] >> (4 * (nib % 2)).to(torch.uint8)) & 15).double() - 8.0
                    for at, nib in ((byte_k, k_nib), (byte_v, v_nib)))
            k = k * scale[:, 0].repeat_interleave(w, 1)
            v = v * scale[:, 1].repeat_interleave(w, 1)
            for j in range(share):
                z = (q[:, h * share + j] @ k.t()) * d ** -0.5
                z = z.masked_fill(~seen, -math.inf)
                p = torch.softmax(z, 1).nan_to_num(0.0)
                out[row:row + n, h * share + j] = p @ v
        row += n
    return out


def _exact_lora(state):
    x, y, a, b, index, scales = (state[n] for n in ("x", "y", "a", "b", "index", "scales"))
    out = y.double()
    for l in range(a.shape[0]):
        rows = (index == l).nonzero().flatten()
        if rows.numel():
            low = x[rows].double() @ a[l].double().t()
            out[rows] += float(scales[l]) * (low @ b[l].double().t())
    return out
