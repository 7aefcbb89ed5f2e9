"""The attention half of one decoder layer in serving, on INT4 weights and a
4-bit cache:

    qkv = x Wqkv^T (INT4) + the request's adapter
    q, cache <- rotate by position, quantize keys and values, store
    o = attention over the cache
    y = o Wo^T (INT4) + the request's adapter

Prompts of several requests run as one ragged batch, then one token a request
and step from a captured graph, in which only the contents of the slot, position
and length buffers change.

    python examples/decoder_layer.py [--requests 8] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import weight_only_int4_rtn_amd as w4  # noqa: E402


class AttentionLayer:
    """Weights, adapters and cache of one layer: `heads` query heads share
    `kv_heads` key heads of head_dim channels; adapters of one rank."""

    def __init__(self, hidden=2048, heads=8, kv_heads=1, head_dim=256, adapters=4, rank=16, pages=256, page_size=16,
                 context=4096, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.heads, self.kv_heads, self.head_dim, self.hidden = heads, kv_heads, head_dim, hidden
        self.n_qkv = (heads + 2 * kv_heads) * head_dim
        self.qkv = w4.pack(*w4.quantize(randn(self.n_qkv, hidden) * hidden ** -0.5))
        self.o = w4.pack(*w4.quantize(randn(hidden, heads * head_dim) * (heads * head_dim) ** -0.5))
        low = lambda n, k: ((randn(adapters, rank, k) * k ** -0.5).to(dtype), (randn(adapters, n, rank) * 0.1).to(dtype))  # noqa: E731
        self.qkv_low, self.o_low = low(self.n_qkv, hidden), low(hidden, heads * head_dim)
        self.low_scales = torch.full((adapters,), 0.5, device=device)
        self.page_size = page_size
        self.pool = w4.kv4_pool(pages, page_size, kv_heads, head_dim, device=device)
        self.rope = w4.rope_table(context, head_dim, device=device)

    def forward(self, x, adapter, slots, positions, block_table, kv_lens, cu_q=None, workspace=None):
        """x [tokens, hidden] -> [tokens, hidden]; adapter, slots, positions per token, the rest per request."""
        ws = dict(workspace=workspace)
        qkv = w4.linear(x, self.qkv, self.n_qkv, **ws)
        w4.lora_add(qkv, x, *self.qkv_low, adapter, scales=self.low_scales, out=qkv, **ws)
        q = w4.kv4_append(qkv, self.pool, slots, self.head_dim, positions=positions, rope=self.rope)
        o = w4.kv4_attention(q, self.pool, block_table, kv_lens, cu_q=cu_q, **ws).flatten(1)
        y = w4.linear(o, self.o, self.hidden, **ws)
        return w4.lora_add(y, o, *self.o_low, adapter, scales=self.low_scales, out=y, **ws)

    def workspace_bytes(self, tokens, batch, table_width, ragged=False):
        """A workspace that serves every call of forward() for these sizes."""
        wide, adapters, rank = self.heads * self.head_dim, self.low_scales.numel(), self.qkv_low[0].shape[1]
        return max(w4.workspace_bytes(tokens, self.n_qkv, self.hidden), w4.workspace_bytes(tokens, self.hidden, wide),
                   w4.lora_add_workspace_bytes(tokens, self.n_qkv, self.hidden, adapters, rank),
                   w4.lora_add_workspace_bytes(tokens, self.hidden, wide, adapters, rank),
                   w4.kv4_attention_workspace_bytes(tokens, batch, self.heads, self.kv_heads, self.head_dim, table_width,
                                                    self.page_size, ragged=ragged), 16)


class Batch:
    """Requests on pages of a layer's cache: block table, lengths, and the slots of their next tokens."""

    def __init__(self, prompts, room, page_size, adapters, device="cuda"):
        width = -(-room // page_size)
        self.page_size, self.lens = page_size, [0] * len(prompts)
        self.table = torch.arange(len(prompts) * width, dtype=torch.int32).view(len(prompts), width)
        self.device_table = self.table.to(device)
        self.adapter = torch.tensor([adapters[i % len(adapters)] for i in range(len(prompts))], dtype=torch.int32)
        self.device = device

    def take(self, counts):
        """The next counts[i] tokens of each request: (adapter, slots, positions) per token, kv_lens, cu_q."""
        slots, positions, adapter = [], [], []
        for i, n in enumerate(counts):
            at = torch.arange(self.lens[i], self.lens[i] + n)
            slots.append(self.table[i].long()[at // self.page_size] * self.page_size + at % self.page_size)
            positions.append(at.to(torch.int32))
            adapter.append(self.adapter[i].repeat(n))
            self.lens[i] += n
        cu = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32)
        lens = torch.tensor(self.lens, dtype=torch.int32)
        return tuple(t.to(self.device) for t in (torch.cat(adapter), torch.cat(slots), torch.cat(positions), lens, cu))


def run(layer: AttentionLayer, prompts, steps: int, seed=1):
    """Prompts, then `steps` tokens of each request; returns the outputs of the prompts and of every step."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda n: torch.randn(n, layer.hidden, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    batch = Batch(prompts, max(prompts) + steps, layer.page_size, [0, 1, -1, 2])
    x = new(sum(prompts))
    adapter, slots, positions, lens, cu = batch.take(prompts)
    inputs, outputs = [x], [layer.forward(x, adapter, slots, positions, batch.device_table, lens, cu_q=cu)]
    if steps == 0:
        return batch, inputs, outputs

    # one decoding step, captured: its buffers are rewritten between replays
    n = len(prompts)
    hold = [new(n), *batch.take([1] * n)[:4]]
    ws = torch.zeros(layer.workspace_bytes(n, n, batch.device_table.shape[1]), dtype=torch.uint8, device="cuda")
    step = lambda: layer.forward(hold[0], hold[1], hold[2], hold[3], batch.device_table, hold[4], workspace=ws)  # noqa: E731
    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = step()
    for i in range(steps):
        if i:
            for buffer, value in zip(hold, (new(n), *batch.take([1] * n)[:4])):
                buffer.copy_(value)
        graph.replay()
        inputs.append(hold[0].clone())
        outputs.append(y.clone())
    return batch, inputs, outputs


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    prompts = [40 + 97 * i % 600 for i in range(a.requests)]
    room = max(prompts) + a.steps
    layer = AttentionLayer(pages=a.requests * -(-room // 16))
    run(layer, prompts, a.steps)  # warm up
    torch.cuda.synchronize()
    t = time.perf_counter()
    batch, _, outputs = run(layer, prompts, a.steps)
    torch.cuda.synchronize()
    print(f"{a.requests} requests, prompts of {prompts}, {a.steps} steps: {(time.perf_counter() - t) * 1e3:.1f} ms, "
          f"cache {layer.pool.numel() / 1e6:.1f} MB for {sum(batch.lens)} tokens "
          f"({2 * 2 * layer.kv_heads * layer.head_dim * sum(batch.lens) / 1e6:.1f} MB in 16 bits), "
          f"last output {float(outputs[-1].float().abs().mean()):.4f} mean size")


if __name__ == "__main__":
    main()
