"""Autograd inputs of the serving operators: refused where a graph would be recorded, accepted under no_grad (CPU
tensors: a call that passes the check goes on to the one for the device)."""
import pytest
import torch

import weight_only_int4_rtn_amd as w4


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def leaf(*shape, dtype=torch.bfloat16):
    return torch.nn.Parameter(t(*shape, dtype=dtype))


def lora(**kw):
    good = dict(y=t(5, 40), x=t(5, 64), a=t(2, 8, 64), b=t(2, 40, 8), index=t(5, dtype=torch.int32))
    return w4.lora_add(**{**good, **kw})


def attention(**kw):
    pool = w4.kv4_pool(2, 16, 2, 64, device="cpu")
    good = dict(q=t(3, 4, 64), pool=pool, block_table=t(3, 2, dtype=torch.int32), kv_lens=t(3, dtype=torch.int32))
    return w4.kv4_attention(**{**good, **kw})


def append(**kw):
    good = dict(qkv=t(4, 4 * 64), pool=w4.kv4_pool(2, 16, 1, 64, device="cpu"), slots=t(4, dtype=torch.int64), head_dim=64)
    return w4.kv4_append(**{**good, **kw})


CALLS = [
    (lora, dict(x=leaf(5, 64))), (lora, dict(y=leaf(5, 40))), (lora, dict(a=leaf(2, 8, 64), b=leaf(2, 40, 8))),
    (lora, dict(scales=leaf(2, dtype=torch.float32))), (lora, dict(out=leaf(5, 40))),
    (attention, dict(q=leaf(3, 4, 64))), (attention, dict(out=leaf(3, 4, 64))),
    (append, dict(qkv=leaf(4, 256))), (append, dict(q_out=leaf(4, 2, 64))),
    (append, dict(positions=t(4, dtype=torch.int32), rope=leaf(10, 64, dtype=torch.float32))),
]


@pytest.mark.parametrize("call,kw", CALLS, ids=[f"{f.__name__}-{'-'.join(k)}" for f, k in CALLS])
def test_refused_where_a_graph_is_recorded(call, kw):
    with pytest.raises(ValueError, match="inference only"):
        call(**kw)


@pytest.mark.parametrize("call,kw", CALLS, ids=[f"{f.__name__}-{'-'.join(k)}" for f, k in CALLS])
@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_parameters_are_taken_without_one(mode, call, kw):
    with mode(), pytest.raises(ValueError, match="GPU"):
        call(**kw)
    with pytest.raises(ValueError, match="inference only"):  # the mode is not remembered
        call(**kw)
