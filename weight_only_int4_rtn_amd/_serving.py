"""Serving operators around the layer's projections: keys and values in a
paged 4-bit cache, attention over it, and low-rank adapters beside a shared
projection (the kv4_* and lora_add entry points of include/w4a16.h).

Argument marshalling and checks from metadata only, as in ``_binding``."""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._binding import _act_tag, _check, _w_tag, _workspaces, lib, workspace_for

_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        L = lib()
        i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        L.kv4_pool_bytes.argtypes = [i64] * 4
        L.kv4_pool_bytes.restype = sz
        L.kv4_append.argtypes = [vp, i32, i64, i64, i64, i64, i64, vp, i64, i64, i32, vp, vp, vp, i64, i64, vp, vp]
        L.kv4_append.restype = i32
        L.kv4_read.argtypes = [vp, i64, i64, i64, i64, vp, i64, i32, vp, vp, vp]
        L.kv4_read.restype = i32
        L.kv4_attention_workspace_bytes.argtypes = [i64] * 7 + [i32, i32, i64]
        L.kv4_attention_workspace_bytes.restype = sz
        L.kv4_attention_tile_rows.argtypes = [i64] * 7 + [i32, i32, i64]
        L.kv4_attention_tile_rows.restype = i32
        L.kv4_attention.argtypes = [vp, i32, i64, i64, i64, i64, i64, vp, i64, i64, vp, i64, i64, vp, vp, i64, i32, i64,
                                    ctypes.c_float, vp, i64, vp, sz, vp]
        L.kv4_attention.restype = i32
        L.lora_add_workspace_bytes.argtypes = [i64] * 5
        L.lora_add_workspace_bytes.restype = sz
        L.lora_add.argtypes = [vp, i32, i64, i64, i64, vp, vp, i64, i64, i64, vp, vp, vp, i64, vp, i64, vp, sz, vp]
        L.lora_add.restype = i32
        _loaded = L
    return _loaded


# One decoding step makes each of these calls once a layer, so their cost on the
# host counts (7 to 10 us of Python a call when every check ran every time).  What
# a call derives from its tensors' shapes, strides and dtypes, the checks of
# those among it, is a function of that metadata alone and is remembered by it
# (the _..._plan functions; a refusal is not remembered).  The current stream's
# handle is taken directly: a Stream object costs 2 us.
_raw_stream = torch._C._cuda_getCurrentRawStream
_remember = functools.lru_cache(maxsize=4096)


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype)


def _dense(shape, stride) -> bool:
    """Whether a tensor of this shape and these strides is contiguous."""
    want = 1
    for n, st in zip(reversed(shape), reversed(stride)):
        if n > 1 and st != want:
            return 0 in shape
        want *= n
    return True


def _vector(meta, dtype, n, what):
    shape, stride, have = meta
    if have != dtype or len(shape) != 1 or shape[0] != n:
        raise ValueError(f"{what} must be a [{n}] tensor of {dtype}, got {tuple(shape)} of {have}")
    if n > 1 and stride[0] != 1:
        raise ValueError(f"{what} must be contiguous")


def _workspace(workspace, need: int, device: int, stream: int):
    """(pointer, bytes) of the caller's workspace, or of this stream's."""
    if workspace is None:
        if need == 0:
            return None, 0
        if torch.cuda.is_current_stream_capturing():
            raise ValueError(f"this call needs a {need}-byte workspace: under graph capture pass a "
                             "zero-filled workspace= allocated before the capture")
        workspace = _workspaces.get((device, stream))
        if workspace is None or workspace.numel() < need:
            workspace = workspace_for(torch.device("cuda", device), stream, need)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _device_index(first, *others) -> int:
    """The GPU that all of the tensors (or None) are on."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be on a GPU device")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors must be on one device, got {first.device} and {t.device}")
    return index


def _no_grad(*ts):
    """Refuses inputs and outputs of a graph that autograd would record; parameters are taken under no_grad."""
    for t in ts:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise ValueError("inference only: autograd inputs are not supported (call it under torch.no_grad())")


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------


def _region(page_size: int, head_dim: int) -> int:
    return page_size * head_dim + 8 * page_size * (head_dim // min(head_dim, 128))


def kv4_pool(pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda") -> torch.Tensor:
    """A 4-bit cache of ``pages`` pages of ``page_size`` tokens: uint8
    [pages, kv_heads, bytes of a page of one head].  page_size is a multiple
    of 16 (at most 4096); head_dim is 64, 128 or 256."""
    if _lib().kv4_pool_bytes(pages, page_size, kv_heads, head_dim) == 0:
        raise ValueError(f"no such cache: pages={pages}, page_size={page_size} (a multiple of 16, at most 4096), "
                         f"kv_heads={kv_heads}, head_dim={head_dim} (64, 128 or 256)")
    return torch.zeros(pages, kv_heads, _region(page_size, head_dim), dtype=torch.uint8, device=device)


@_remember
def _page_size(shape, stride, dtype, head_dim: int) -> int:
    if head_dim not in (64, 128, 256):
        raise ValueError(f"head_dim is 64, 128 or 256, got {head_dim}: no heads of so many channels")
    if dtype != torch.uint8 or len(shape) != 3 or not _dense(shape, stride):
        raise ValueError("pool must be a contiguous uint8 [pages, kv_heads, region] tensor (kv4_pool)")
    page, rest = divmod(shape[2], head_dim + 8 * (head_dim // min(head_dim, 128)))
    if rest or page % 16 or not 16 <= page <= 4096 or shape[0] < 1 or shape[1] < 1:
        raise ValueError(f"pool of shape {tuple(shape)} does not hold pages of heads of {head_dim} channels")
    return page


def kv4_page_size(pool: torch.Tensor, head_dim: int) -> int:
    """Tokens of a page of ``pool`` (from kv4_pool) with heads of head_dim channels."""
    return _page_size(pool.shape, pool.stride(), pool.dtype, head_dim)


def rope_table(length: int, rot_dim: int, base: float = 10000.0, factor: float = 1.0, original_length: int | None = None,
               low_turns: float = 1.0, high_turns: float = 32.0, magnitude: float = 1.0, device="cuda") -> torch.Tensor:
    """Rotation table of kv4_append: FP32 [length, rot_dim], row p the cosines
    then the sines of p * base^(-2i / rot_dim), i < rot_dim / 2, computed in 64
    bits (FP32 angles lose far positions).

    For contexts longer than a model was trained on, ``factor`` > 1 stretches
    the angles: all of them by 1 / factor, or, with ``original_length`` given,
    by wavelength: those that turn more than ``high_turns`` times over the
    original length stay, those that turn less than ``low_turns`` are divided
    by factor, with a linear ramp between.  ``magnitude`` multiplies the table
    (a correction of the logits' temperature)."""
    if length < 1 or rot_dim < 16 or rot_dim % 16:
        raise ValueError(f"a table of at least one position and a multiple of 16 channels, got {length} x {rot_dim}")
    if base <= 0 or factor < 1 or (original_length is not None and not 0 < low_turns < high_turns):
        raise ValueError("base > 0, factor >= 1 and 0 < low_turns < high_turns are needed")
    freq = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    if original_length is None:
        freq = freq / factor
    else:
        turns = original_length * freq / (2 * math.pi)
        keep = ((turns - low_turns) / (high_turns - low_turns)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / factor)
    angle = torch.arange(length, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), 1).mul_(magnitude).float()


@_remember
def _append_plan(qkv, pool, slots, head_dim, rope, positions, q_out):
    page = _page_size(*pool, head_dim)
    shape, stride, dtype = qkv
    tag = _act_tag(dtype)
    pages, kv_heads = pool[0][0], pool[0][1]
    if len(shape) != 2 or stride[1] != 1 or (shape[0] > 1 and stride[0] % 8):
        raise ValueError("qkv must be 2-D with contiguous rows and a row stride that is a multiple of 8")
    tokens, width = shape
    heads = width // head_dim - 2 * kv_heads
    if width % head_dim or heads < 0:
        raise ValueError(f"qkv rows of {width} do not hold 2 x {kv_heads} key and value heads of {head_dim}")
    _vector(slots, torch.int64, tokens, "slots")
    rope_len = rot = 0
    if rope is not None:
        if positions is None:
            raise ValueError("a rotation needs positions")
        if rope[2] != torch.float32 or len(rope[0]) != 2 or not _dense(*rope[:2]):
            raise ValueError("rope must be a contiguous float32 [positions, rot_dim] table (rope_table)")
        rope_len, rot = rope[0]
        if rot % 16 or not 16 <= rot <= head_dim or rope_len < 1:
            raise ValueError(f"rope has {rope_len} x {rot}: rot_dim is a multiple of 16, at most head_dim")
        _vector(positions, torch.int32, tokens, "positions")
    if q_out is not None and (q_out[0] != (tokens, heads, head_dim) or q_out[2] != dtype or not _dense(*q_out[:2])):
        raise ValueError("q_out must be a contiguous [tokens, heads, head_dim] tensor of qkv's dtype")
    return tag, tokens, stride[0] if tokens > 1 else -(-width // 8) * 8, heads, kv_heads, rope_len, rot, pages, page


def kv4_append(qkv: torch.Tensor, pool: torch.Tensor, slots: torch.Tensor, head_dim: int,
               positions: torch.Tensor | None = None, rope: torch.Tensor | None = None, interleaved: bool = False,
               q_out: torch.Tensor | None = None) -> torch.Tensor:
    """Stores keys and values of ``qkv`` [tokens, (heads + 2 kv_heads) head_dim]
    (bf16/f16, a fused projection's output) in ``pool`` at ``slots`` [tokens]
    int64 (page * page_size + token; outside the pool, -1 say: not stored),
    rotated by ``rope`` (rope_table) at ``positions`` [tokens] int32 and
    quantized to 4 bits; returns the rotated queries [tokens, heads, head_dim].
    Without ``rope`` nothing is rotated and positions are not read.  A group
    of channels with a NaN or an infinity reads back as NaN.
    See kv4_append in include/w4a16.h."""
    plan = _append_plan(_meta(qkv), _meta(pool), _meta(slots), head_dim, _meta(rope),
                        None if rope is None else _meta(positions), _meta(q_out))
    tag, tokens, ld, heads, kv_heads, rope_len, rot, pages, page = plan
    _no_grad(qkv, rope, q_out)
    index = _device_index(qkv, pool, slots, positions if rope is not None else None, rope, q_out)
    if q_out is None:
        q_out = qkv.new_empty((tokens, heads, head_dim))
    table = at = None
    if rope is not None:
        table, at = rope.data_ptr(), positions.data_ptr()
    st = _lib().kv4_append(qkv.data_ptr(), tag, tokens, ld, heads, kv_heads, head_dim, table, rope_len, rot,
                           1 if interleaved else 0, at, slots.data_ptr(), pool.data_ptr(), pages, page, q_out.data_ptr(),
                           _raw_stream(index))
    if st:
        _check(st, "kv4_append")
    return q_out


@_remember
def _read_plan(pool, slots, head_dim, dtype):
    page = _page_size(*pool, head_dim)
    tag = _w_tag(dtype)
    if len(slots[0]) != 1:
        raise ValueError("slots must be a 1-D int64 tensor")
    _vector(slots, torch.int64, slots[0][0], "slots")
    return tag, slots[0][0], pool[0][0], pool[0][1], page


def kv4_read(pool: torch.Tensor, slots: torch.Tensor, head_dim: int, dtype: torch.dtype = torch.bfloat16):
    """The values stored at ``slots`` [tokens] int64: (k, v), each
    [tokens, kv_heads, head_dim] of ``dtype`` (float32, bfloat16 or float16);
    zeros where a slot is outside the pool."""
    tag, tokens, pages, kv_heads, page = _read_plan(_meta(pool), _meta(slots), head_dim, dtype)
    index = _device_index(pool, slots)
    k = pool.new_empty((tokens, kv_heads, head_dim), dtype=dtype)
    v = torch.empty_like(k)
    st = _lib().kv4_read(pool.data_ptr(), pages, page, kv_heads, head_dim, slots.data_ptr(), tokens, tag, k.data_ptr(),
                         v.data_ptr(), _raw_stream(index))
    if st:
        _check(st, "kv4_read")
    return k, v


def _window(window) -> int:
    """A window that the C ABI's int64 holds: longer ones hide nothing either."""
    if not isinstance(window, int) or window < 0:
        raise ValueError("window is 0 (none) or a positive number of tokens")
    return min(window, (1 << 63) - 1)


@_remember
def _attention_need(*sizes) -> int:
    return int(_lib().kv4_attention_workspace_bytes(*sizes))


@_remember
def _lora_need(*sizes) -> int:
    return int(_lib().lora_add_workspace_bytes(*sizes))


def kv4_attention_workspace_bytes(tokens: int, batch: int, heads: int, kv_heads: int, head_dim: int, table_width: int,
                                  page_size: int, ragged: bool = False, causal: bool = True, window: int = 0) -> int:
    """Workspace kv4_attention needs for these sizes (``ragged``: cu_q is given)."""
    return _attention_need(tokens, batch, heads, kv_heads, head_dim, table_width, page_size, int(bool(ragged)),
                           int(bool(causal)), _window(window))


def kv4_attention_tile_rows(tokens: int, batch: int, heads: int, kv_heads: int, head_dim: int, table_width: int, page_size: int,
                            ragged: bool = False, causal: bool = True, window: int = 0) -> int:
    """Rows of a workgroup's tile in kv4_attention for these sizes: 16 or 64, each a kernel of its own (0: invalid sizes)."""
    return _lib().kv4_attention_tile_rows(tokens, batch, heads, kv_heads, head_dim, table_width, page_size, int(bool(ragged)),
                                          int(bool(causal)), _window(window))


@_remember
def _attention_plan(q, pool, table, kv_lens, cu_q, out, causal, window):
    shape, stride, dtype = q
    if len(shape) != 3 or stride[2] != 1 or (shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError("q must be [tokens, heads, head_dim] with contiguous tokens")
    tokens, heads, dim = shape
    page = _page_size(*pool, dim)
    tag = _act_tag(dtype)
    pages, kv_heads = pool[0][0], pool[0][1]
    if heads < 1 or heads % kv_heads:
        raise ValueError(f"{heads} query heads do not share {kv_heads} key heads evenly")
    if table[2] != torch.int32 or len(table[0]) != 2 or table[0][1] < 1 or table[1][1] != 1:
        raise ValueError("block_table must be an int32 [batch, width] tensor with contiguous rows")
    batch, width = table[0]
    _vector(kv_lens, torch.int32, batch, "kv_lens")
    if cu_q is not None:
        _vector(cu_q, torch.int32, batch + 1, "cu_q")
    elif tokens != batch:
        raise ValueError(f"{tokens} query tokens for {batch} requests: pass cu_q")
    if tokens and not batch:
        raise ValueError("query tokens without a request")
    window = _window(window)
    if out is not None and (out[0] != shape or out[2] != dtype or not _dense(*out[:2])):
        raise ValueError("out must be a contiguous tensor of q's shape and dtype")
    need = _attention_need(tokens, batch, heads, kv_heads, dim, width, page, 0 if cu_q is None else 1, causal, window)
    return (tag, tokens, stride[0] if tokens > 1 else heads * dim, heads, kv_heads, dim, pages, page, width,
            table[1][0] if batch > 1 else width, batch, window, need)


def kv4_attention(q: torch.Tensor, pool: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor,
                  cu_q: torch.Tensor | None = None, causal: bool = True, window: int = 0, scale: float | None = None,
                  out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """softmax(scale q k^T) v over the 4-bit cache: q [tokens, heads, head_dim]
    (bf16/f16) -> [tokens, heads, head_dim].  ``block_table`` [batch, width]
    int32 holds each request's pages, ``kv_lens`` [batch] int32 its tokens in
    the cache, the query tokens among them; ``cu_q`` [batch + 1] int32 where
    each request's query tokens begin (None: one each).  ``scale`` defaults to
    head_dim ** -0.5.  See kv4_attention in include/w4a16.h."""
    causal = 1 if causal else 0
    plan = _attention_plan(_meta(q), _meta(pool), _meta(block_table), _meta(kv_lens), _meta(cu_q), _meta(out), causal, window)
    tag, tokens, ldq, heads, kv_heads, dim, pages, page, width, ldt, batch, window, need = plan
    _no_grad(q, out)
    index = _device_index(q, pool, block_table, kv_lens, cu_q, out, workspace)
    if out is None:
        out = q.new_empty((tokens, heads, dim))
    stream = _raw_stream(index)
    ws, ws_bytes = _workspace(workspace, need, index, stream)
    st = _lib().kv4_attention(q.data_ptr(), tag, tokens, ldq, heads, kv_heads, dim, pool.data_ptr(), pages, page,
                              block_table.data_ptr(), width, ldt, kv_lens.data_ptr(), None if cu_q is None else cu_q.data_ptr(),
                              batch, causal, window, dim ** -0.5 if scale is None else scale, out.data_ptr(), heads * dim, ws,
                              ws_bytes, stream)
    if st:
        _check(st, "kv4_attention")
    return out


# ---------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------


def lora_add_workspace_bytes(m: int, n: int, k: int, adapters: int, rank: int) -> int:
    """Workspace lora_add needs for these sizes."""
    return _lora_need(m, n, k, adapters, rank)


@_remember
def _lora_plan(x, y, a, b, index, scales, out, in_place):
    """None where x or y are not 2-D with rows the kernel can walk."""
    tag = _act_tag(x[2])
    if len(a[0]) != 3 or len(b[0]) != 3 or not _dense(*a[:2]) or not _dense(*b[:2]):
        raise ValueError("a [adapters, rank, k] and b [adapters, n, rank] must be contiguous 3-D tensors")
    adapters, rank, k = a[0]
    n = b[0][1]
    if b[0] != (adapters, n, rank) or adapters < 1:
        raise ValueError(f"a {tuple(a[0])} and b {tuple(b[0])} are not [adapters, rank, k] and [adapters, n, rank]")
    if rank % 8 or not 8 <= rank <= 128:
        raise ValueError(f"rank is a multiple of 8, at most 128, got {rank}: pad the adapters with zeros")
    if not x[2] == y[2] == a[2] == b[2]:
        raise ValueError(f"x, y, a and b must have one dtype, got {x[2]}, {y[2]}, {a[2]}, {b[2]}")
    if k < 8 or k % 8 or x[0][-1:] != (k,) or y[0][-1:] != (n,) or x[0][:-1] != y[0][:-1]:
        raise ValueError(f"x [..., {k}] (a multiple of 8) and y [..., {n}] are needed, got {tuple(x[0])}, {tuple(y[0])}")
    m = math.prod(x[0][:-1])
    if n > 1 and y[1][-1] != 1 or (len(y[0]) != 2 and not _dense(*y[:2]) and in_place):
        raise ValueError("y must have contiguous rows (and be contiguous to be added to in place, unless 2-D)")
    _vector(index, torch.int32, m, "index")
    if scales is not None:
        _vector(scales, torch.float32, adapters, "scales")
    if out is not None and not in_place and (out[0] != y[0] or out[2] != y[2] or not _dense(*out[:2])):
        raise ValueError("out must be y, or a contiguous tensor of y's shape and dtype")
    if len(x[0]) != 2 or x[1][1] != 1 or (m > 1 and x[1][0] % 8):
        return None
    ldy = y[1][0] if m > 1 else n
    need = _lora_need(m, n, k, adapters, rank) if m and n else 0
    return tag, m, k, x[1][0] if m > 1 else k, adapters, rank, n, ldy, ldy if in_place else n, need


def lora_add(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, index: torch.Tensor,
             scales: torch.Tensor | None = None, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y + scales[l] (x A_l^T) B_l^T with l = index[row]: low-rank adapters of
    many requests beside a shared projection's output y [..., n] of x [..., k]
    (bf16/f16).  ``a`` [adapters, rank, k] and ``b`` [adapters, n, rank], rank a
    multiple of 8 up to 128; ``index`` [rows] int32, -1 (or any other number
    that is no adapter) for none; ``scales`` [adapters] float32, default 1.
    ``out=y`` adds in place."""
    plan = _lora_plan(_meta(x), _meta(y), _meta(a), _meta(b), _meta(index), _meta(scales), _meta(out), out is y)
    if plan is None:
        # rows the kernel cannot walk in place: 2-D copies or views of them
        k, n, m = a.shape[-1], b.shape[1], index.shape[0]
        x = x.reshape(m, k)
        if x.stride(1) != 1 or (x.shape[0] > 1 and x.stride(0) % 8):
            x = x.contiguous()
        y2 = y.reshape(m, n)
        out2 = y2 if out is y else None if out is None else out.view(m, n)
        got = lora_add(y2, x, a, b, index, scales=scales, out=out2, workspace=workspace)
        return out if out is not None else got.view(y.shape)
    tag, m, k, ldx, adapters, rank, n, ldy, ldo, need = plan
    _no_grad(x, y, a, b, scales, out)
    device = _device_index(x, y, a, b, index, scales, out, workspace)
    if out is None:
        out = y.new_empty((m, n))
    if m == 0 or n == 0:
        return out
    stream = _raw_stream(device)
    ws, ws_bytes = _workspace(workspace, need, device, stream)
    st = _lib().lora_add(x.data_ptr(), tag, m, k, ldx, a.data_ptr(), b.data_ptr(), adapters, rank, n, index.data_ptr(),
                         None if scales is None else scales.data_ptr(), y.data_ptr(), ldy, out.data_ptr(), ldo, ws, ws_bytes,
                         stream)
    if st:
        _check(st, "lora_add")
    return out
