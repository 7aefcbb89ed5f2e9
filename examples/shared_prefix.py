"""One decoder layer for many requests that begin with the same text, on 8-bit
float weights and a 4-bit cache:

    qkv = x Wqkv^T                       (8-bit floats)
    q, cache <- rotate by position, quantize keys and values, store
    o = attention over the shared prefix, met once for all requests, and each request's own tokens
    h = x + o Wo^T
    y = h + (up * silu(gate)) Wdown^T,   [up | gate] = h Wup_gate^T

The prefix runs once as a request of its own; then the requests' prompts as one
ragged batch; then one token a request and step from a captured graph, in which
only the contents of the slot, position and length buffers change.  (Norms are
left out: they are the caller's.)

    python examples/shared_prefix.py [--requests 64] [--prefix 4096] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import weight_only_int4_rtn_amd as w4  # noqa: E402


class Layer:
    """Weights and cache of one layer: `heads` query heads share `kv_heads` key heads of head_dim channels."""

    def __init__(self, hidden=2048, inner=16384, heads=8, kv_heads=1, head_dim=256, pages=1024, page_size=16, context=8192,
                 device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        weight = lambda n, k: w4.quantize_fp8_weight(torch.randn(n, k, generator=g, device=device) * k ** -0.5)  # noqa: E731
        self.hidden, self.heads, self.kv_heads, self.head_dim, self.page_size = hidden, heads, kv_heads, head_dim, page_size
        self.sizes = {"qkv": ((heads + 2 * kv_heads) * head_dim, hidden), "o": (hidden, heads * head_dim),
                      "up_gate": (2 * inner, hidden), "down": (hidden, inner)}
        self.weights = {name: weight(*size) for name, size in self.sizes.items()}
        self.pool = w4.kv4_pool(pages, page_size, kv_heads, head_dim, device=device)
        self.rope = w4.rope_table(context, head_dim, device=device)

    def linear(self, name, x, act=w4.Act.NONE, workspace=None):
        return w4.linear_fp8(x, *self.weights[name], act=act, workspace=workspace)

    def forward(self, x, slots, positions, attend, workspace=None):
        """x [tokens, hidden] -> every stage's output; attend(q) is the attention of the rotated queries."""
        qkv = self.linear("qkv", x, workspace=workspace)
        q = w4.kv4_append(qkv, self.pool, slots, self.head_dim, positions=positions, rope=self.rope)
        o = attend(q)
        h = x + self.linear("o", o.flatten(1), workspace=workspace)
        up_gate = self.linear("up_gate", h, workspace=workspace)
        y = h + self.linear("down", up_gate, act=w4.Act.SWIGLU, workspace=workspace)
        return dict(x=x, qkv=qkv, q=q, o=o, h=h, up_gate=up_gate, y=y)

    def workspace_bytes(self, tokens, batch, prefix_width, table_width, ragged=False):
        """A workspace that serves every call of forward() for these sizes, attention on one shared prefix among them."""
        return max([w4.linear_fp8_workspace_bytes(tokens, *size) for size in self.sizes.values()]
                   + [w4.kv4_prefix_attention_workspace_bytes(tokens, batch, 1, self.heads, self.kv_heads, self.head_dim, prefix_width,
                                                              table_width, self.page_size, ragged=ragged), 16])


class Batch:
    """A prefix and requests behind it on pages of a layer's cache."""

    def __init__(self, prefix, prompts, room, page_size, device="cuda"):
        first, width = -(-prefix // page_size), -(-room // page_size)
        self.prefix, self.page_size, self.device, self.lens = prefix, page_size, device, [0] * len(prompts)
        self.prefix_table = torch.arange(first, dtype=torch.int32).view(1, first)
        self.table = first + torch.arange(len(prompts) * width, dtype=torch.int32).view(len(prompts), width)
        self.pages = first + len(prompts) * width
        self.on_device = tuple(t.to(device) for t in (self.prefix_table, torch.tensor([prefix], dtype=torch.int32), self.table))

    def slots_of(self, row, at):
        return row.long()[at // self.page_size] * self.page_size + at % self.page_size

    def take(self, counts):
        """The next counts[i] tokens of each request: (slots, positions) per token, own lengths, cu_q."""
        slots, positions = [], []
        for i, n in enumerate(counts):
            at = torch.arange(self.lens[i], self.lens[i] + n)
            slots.append(self.slots_of(self.table[i], at))
            positions.append((self.prefix + at).to(torch.int32))
            self.lens[i] += n
        cu = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32)
        return tuple(t.to(self.device) for t in (torch.cat(slots), torch.cat(positions), torch.tensor(self.lens, dtype=torch.int32), cu))


def run(layer: Layer, prefix, prompts, steps, seed=1):
    """The prefix, the prompts, then `steps` tokens of each request; every stage's outputs of each of them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda n: torch.randn(n, layer.hidden, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    batch = Batch(prefix, prompts, max(prompts) + steps, layer.page_size)
    assert batch.pages <= layer.pool.shape[0]
    shared, lens, table = batch.on_device
    at = torch.arange(prefix)
    cu = torch.tensor([0, prefix], dtype=torch.int32, device="cuda")
    out = [layer.forward(new(prefix), batch.slots_of(batch.prefix_table[0], at).cuda(), at.to(torch.int32).cuda(),
                         lambda q: w4.kv4_attention(q, layer.pool, shared, lens, cu_q=cu))]
    slots, positions, own, cu_q = batch.take(prompts)
    out.append(layer.forward(new(sum(prompts)), slots, positions,
                             lambda q: w4.kv4_prefix_attention(q, layer.pool, shared, lens, table, own, cu_q=cu_q)))
    if steps == 0:
        return batch, out

    # one decoding step, captured: its buffers are rewritten between replays
    n = len(prompts)
    hold = [new(n), *batch.take([1] * n)[:3]]
    ws = torch.zeros(layer.workspace_bytes(n, n, shared.shape[1], table.shape[1]), dtype=torch.uint8, device="cuda")
    attend = lambda q: w4.kv4_prefix_attention(q, layer.pool, shared, lens, table, hold[3], workspace=ws)  # noqa: E731
    step = lambda: layer.forward(hold[0], hold[1], hold[2], attend, workspace=ws)  # noqa: E731
    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        stages = step()
    for i in range(steps):
        if i:
            for buffer, value in zip(hold, (new(n), *batch.take([1] * n)[:3])):
                buffer.copy_(value)
        graph.replay()
        out.append({name: t.clone() for name, t in stages.items()})
    return batch, out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--prefix", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    prompts = [20 + 31 * i % 200 for i in range(a.requests)]
    room = max(prompts) + a.steps
    layer = Layer(pages=-(-a.prefix // 16) + a.requests * -(-room // 16))
    run(layer, a.prefix, prompts, a.steps)  # warm up
    torch.cuda.synchronize()
    t = time.perf_counter()
    batch, out = run(layer, a.prefix, prompts, a.steps)
    torch.cuda.synchronize()
    seen = sum(batch.lens) + a.requests * a.prefix
    print(f"{a.requests} requests on a prefix of {a.prefix} tokens, {sum(prompts)} prompt tokens, {a.steps} steps: "
          f"{(time.perf_counter() - t) * 1e3:.1f} ms, cache {layer.pool.numel() / 1e6:.1f} MB for {seen} tokens that the requests see, "
          f"last output {float(out[-1]['y'].float().abs().mean()):.4f} mean size")


if __name__ == "__main__":
    main()
