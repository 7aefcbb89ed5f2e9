"""The example's layer on a shared prefix (prefix, prompts, captured decoding
steps), every stage against plain implementations in 64 bits on the host.

The host follows the device's own 16-bit values between the stages, so every
operator is held to its own error and none to the one before it."""
import os
import sys

import numpy as np
import pytest
import torch

from tests import fp8_ref as R
from tests import kv4_prefix_ref as pref
from tests import kv4_ref as ref
from tests.gpu_util import require_gpu, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix,prompts,apart", [(100, [7, 40, 1], False), (2500, [9, 1, 30, 16] * 12, True)], ids=["together", "apart"])
def test_example_layer_on_a_shared_prefix(prefix, prompts, apart):
    require_gpu()
    import shared_prefix as ex
    import weight_only_int4_rtn_amd as w4
    steps, hk, d = 3, 2, 64
    layer = ex.Layer(hidden=256, inner=384, heads=4, kv_heads=hk, head_dim=d, pages=600, page_size=16, context=4096)
    say("shared prefix", prefix, prompts)
    batch, out = ex.run(layer, prefix, prompts, steps)
    torch.cuda.synchronize()
    assert batch.lens == [p + steps for p in prompts] and len(out) == 2 + steps
    n = len(prompts)
    assert (w4.kv4_prefix_attention_tile_rows(n, n, 1, 4, hk, d, batch.prefix_table.shape[1], batch.table.shape[1], 16) > 0) == apart

    weights = {name: (c.cpu().view(torch.uint8).numpy(), s.cpu().numpy()) for name, (c, s) in layer.weights.items()}

    def linear(name, x, got, act="none", residual=None):
        """A product of the device's input; with a residual, the sum's bf16 rounding on top of the product's."""
        codes, scales = w4.quantize_fp8(x, act=w4.Act.SWIGLU) if act == "swiglu" else (None, None)
        cx, sx = R.quantize_rows(x.float().cpu().numpy()) if codes is None else (codes.cpu().view(torch.uint8).numpy(), scales.cpu().numpy())
        want, tol = R.linear(cx, sx, *weights[name])
        if residual is not None:
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
            want = want + residual.cpu().double()
        R.within(got, want, tol, name)

    table = layer.rope.cpu().numpy()
    keys, values = [[] for _ in range(n)], [[] for _ in range(n)]
    shared = None
    for t, st in enumerate(out):
        counts = [prefix] if t == 0 else prompts if t == 1 else [1] * n
        linear("qkv", st["x"], st["qkv"])
        begin = [0] if t == 0 else [prefix + sum(len(k) for k in keys[i]) for i in range(n)]
        position = np.concatenate([np.arange(b, b + c) for b, c in zip(begin, counts)])
        z = st["qkv"].cpu().float().numpy().reshape(-1, 4 + 2 * hk, d)
        z[:, :4 + hk] = ref.rotated(z[:, :4 + hk], table, position, False)
        assert torch.equal(st["q"].cpu(), torch.from_numpy(z[:, :4].copy()).to(torch.bfloat16))
        stored = ref.quantized(z[:, 4:], d)
        q, o, row = st["q"].cpu(), st["o"], 0
        if t == 0:
            shared = stored[:, :hk], stored[:, hk:]
            some = np.r_[0:5, prefix - 5:prefix]  # rows of the prefix's own attention, an existing operator
            for i in some:
                want, tol = ref.attention(q[i:i + 1], shared[0][:i + 1], shared[1][:i + 1], i + 1, 1, True, 0, d ** -0.5)
                ref.within(o[i:i + 1], want, tol, f"prefix row {i}")
        else:
            for i, c in enumerate(counts):
                keys[i].append(stored[row:row + c, :hk])
                values[i].append(stored[row:row + c, hk:])
                own = sum(len(k) for k in keys[i])
                k, v = np.concatenate([shared[0], *keys[i]]), np.concatenate([shared[1], *values[i]])
                want, tol = pref.attention(q[row:row + c], k, v, pref.seen_tokens(prefix, own, c, True), d ** -0.5)
                ref.within(o[row:row + c], want, tol, f"step {t} request {i}")
                row += c
        linear("o", st["o"].flatten(1), st["h"], residual=st["x"])
        linear("up_gate", st["h"], st["up_gate"])
        linear("down", st["up_gate"], st["y"], act="swiglu", residual=st["h"])
