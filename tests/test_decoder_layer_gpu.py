"""The example's layer, prompts and then captured decoding steps, against a
plain implementation of the same layer in 64 bits on the host: the linears from
their dequantized weights, the cache from the quantizer's FP32 steps.

The host follows the device's own 16-bit intermediate values (the projections'
outputs and the rotated queries are rounded to bf16 between the operators), so
every operator is held to its own error and none to the one before it."""
import os
import sys

import numpy as np
import pytest
import torch

from tests import kv4_ref as ref
from tests.gpu_util import require_gpu, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_example_layer_prompts_and_captured_steps():
    require_gpu()
    import decoder_layer as ex
    import weight_only_int4_rtn_amd as w4
    prompts, steps = [37, 5, 120], 4
    layer = ex.AttentionLayer(hidden=512, heads=8, kv_heads=2, head_dim=64, adapters=3, rank=8, pages=3 * 8, page_size=16,
                              context=256)
    say("decoder layer: prompts", prompts, "steps", steps)
    batch, inputs, outputs = ex.run(layer, prompts, steps)
    torch.cuda.synchronize()
    assert batch.lens == [p + steps for p in prompts]

    # the cache holds, for every token in order, what the example's projections and the plain quantizer give
    d, hk, h = layer.head_dim, layer.kv_heads, layer.heads
    table = layer.rope.cpu().numpy()
    keys, values = [[] for _ in prompts], [[] for _ in prompts]
    lens = [0] * len(prompts)
    for x, y, counts in zip(inputs, outputs, [prompts] + [[1] * len(prompts)] * steps):
        owner = [i for i, n in enumerate(counts) for _ in range(n)]
        adapter = batch.adapter[owner].cuda()
        qkv = w4.linear(x, layer.qkv, layer.n_qkv)
        w4.lora_add(qkv, x, *layer.qkv_low, adapter, scales=layer.low_scales, out=qkv)
        position = np.concatenate([np.arange(lens[i], lens[i] + n) for i, n in enumerate(counts)])
        z = qkv.cpu().float().numpy().reshape(-1, h + 2 * hk, d)
        z[:, :h + hk] = ref.rotated(z[:, :h + hk], table, position, False)
        q = torch.from_numpy(z[:, :h].copy()).to(torch.bfloat16)
        stored = ref.quantized(z[:, h:], d)
        row, attended = 0, []
        for i, n in enumerate(counts):
            keys[i].append(stored[row:row + n, :hk])
            values[i].append(stored[row:row + n, hk:])
            lens[i] += n
            k, v = np.concatenate(keys[i]), np.concatenate(values[i])
            attended.append(ref.attention(q[row:row + n], k, v, lens[i], n, True, 0, d ** -0.5))
            row += n
        o, tol = (torch.cat([a[j] for a in attended]).flatten(1) for j in (0, 1))
        # the output projection and adapters of the 64-bit attention: its error and a bf16 rounding pass through
        codes, scales = w4.unpack(layer.o, layer.hidden, h * d)
        c = codes.cpu().to(torch.int16)
        c = torch.stack((c & 15, c >> 4), -1).flatten(1)
        wo = ((c ^ 8) - 8).double().view(layer.hidden, -1, 128) * scales.cpu().double().unsqueeze(-1)
        wo = wo.view(layer.hidden, -1)
        a, b = (t.cpu().double() for t in layer.o_low)
        eff = [wo + (0.5 * b[l] @ a[l] if l >= 0 else 0) for l in batch.adapter.tolist()]
        for t in range(len(owner)):
            w = eff[owner[t]]
            want = w @ o[t]
            off = tol[t] + 2.0 ** -8 * o[t].abs()  # bf16 attention output
            # the linear's stated tolerance (1e-2 |x| max|W row|), its own and the sum's bf16 roundings, the adapter's FP32
            limit = w.abs() @ off + 1e-2 * o[t].norm() * wo.abs().amax(1) + 2.0 ** -8 * ((wo @ o[t]).abs() + want.abs()) + 1e-5
            worst = float(((y[t].cpu().double() - want).abs() / limit).max())
            assert worst <= 1, (counts, t, worst)
