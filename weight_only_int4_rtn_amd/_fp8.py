"""The linear layer on 8-bit floats (e4m3) with one FP32 scale per 128 x 128
weights and per row and 128 columns of the input (the *_fp8_* entry points of
include/w4a16.h).

Argument marshalling and checks from metadata only, as in ``_binding``."""
from __future__ import annotations

import ctypes
import math

import torch

from ._binding import BF16, GROUP, Act, _act_tag, _check, _w_tag, lib
from ._serving import _dense, _device_index, _meta, _no_grad, _launch, _raw_stream, _remember, _workspace

E4M3 = 3  # W4A16_E4M3 of include/w4a16.h
CODES = torch.float8_e4m3fn
_MAX_K = 1 << 22
_MAX_STEP = {1: _MAX_K, 2: 1 << 24, 4: 1 << 24}  # elements between rows that a kernel takes, by their size

_loaded = None


def _lib():
    global _loaded
    if _loaded is None:
        L = lib()
        i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
        L.quantize_fp8_rows.argtypes = [vp, i32, i32, i64, i64, i64, vp, vp, vp]
        L.quantize_fp8_rows.restype = i32
        L.quantize_fp8_blocks.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp]
        L.quantize_fp8_blocks.restype = i32
        L.fp8_linear_workspace_bytes.argtypes = [i32, i64, i64, i64]
        L.fp8_linear_workspace_bytes.restype = sz
        L.fp8_linear_tile.argtypes = [i64, i64, i64, ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.fp8_linear_tile.restype = i32
        L.fp8_linear.argtypes = [vp, i32, vp, i32, i64, i64, i64, vp, vp, i64, vp, vp, i32, i64, vp, sz, vp]
        L.fp8_linear.restype = i32
        _loaded = L
    return _loaded


def _rows(shape, stride, elem: int):
    """(rows, elements between them) of a tensor [..., width] that a kernel can walk, or None: contiguous rows at even
    distances that are multiples of 16 bytes, none too long."""
    m = math.prod(shape[:-1])
    if shape[-1] > 1 and stride[-1] != 1:
        return None
    if m <= 1:
        return m, -(-shape[-1] * elem // 16) * 16 // elem
    step, want = None, None
    for n, st in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if step is None:
            step = want = st
        if st != want:
            return None
        want *= n
    return (m, step) if shape[-1] <= step <= _MAX_STEP[elem] and step * elem % 16 == 0 else None


def _width(width: int, act: Act) -> int:
    """k of rows of ``width`` values."""
    if act == Act.SWIGLU and width % 2:
        raise ValueError("SwiGLU input rows hold [up | gate]: an even number of columns")
    k = width // 2 if act == Act.SWIGLU else width
    if k % GROUP or not GROUP <= k <= _MAX_K:
        raise ValueError(f"k is a multiple of {GROUP}, at most 2^22, got {k}")
    return k


@_remember
def _quantize_plan(x, act):
    shape, stride, dtype = x
    tag, act = _act_tag(dtype), Act(act)
    if len(shape) < 1:
        raise ValueError("x must have at least one dimension")
    k = _width(shape[-1], act)
    rows = _rows(shape, stride, 2)
    return tag, int(act), k, rows, (*shape[:-1], k), (*shape[:-1], k // GROUP)


def quantize_fp8(x: torch.Tensor, act: Act = Act.NONE) -> tuple[torch.Tensor, torch.Tensor]:
    """Rows of x [..., k] (bf16/f16, k a multiple of 128) in 8-bit floats:
    (codes [..., k] float8_e4m3fn, scales [..., k / 128] float32), one scale
    max|x| / 448 per row and 128 columns.  ``act``: activation applied first, as
    in ``linear`` (SwiGLU rows hold [up | gate], 2k values).  A group with a NaN
    or an infinity becomes NaN.  See quantize_fp8_rows in include/w4a16.h."""
    tag, act, k, rows, shape, groups = _quantize_plan(_meta(x), act)
    _no_grad(x)
    index = _device_index(x)
    if rows is None or x.data_ptr() % 16:
        x = x.clone(memory_format=torch.contiguous_format)
        rows = math.prod(shape[:-1]), x.shape[-1]
    codes, scales = x.new_empty(shape, dtype=CODES), x.new_empty(groups, dtype=torch.float32)
    st = _launch(index, _lib().quantize_fp8_rows, x.data_ptr(), tag, act, rows[0], k, rows[1], codes.data_ptr(), scales.data_ptr(),
                 _raw_stream(index))
    if st:
        _check(st, "quantize_fp8")
    return codes, scales


def quantize_fp8_weight(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Weights w [n, k] (float32, bf16 or f16, k a multiple of 128) in 8-bit floats
    for ``linear_fp8``: (codes [n, k] float8_e4m3fn, scales [ceil(n / 128), k / 128]
    float32), one scale max|w| / 448 per block of 128 x 128."""
    if w.dim() != 2:
        raise ValueError(f"w must be [n, k], got {tuple(w.shape)}")
    tag = _w_tag(w.dtype)
    n, k = w.shape[0], _width(w.shape[1], Act.NONE)
    _no_grad(w)
    index = _device_index(w)
    rows = _rows(w.shape, w.stride(), w.element_size())
    if rows is None or w.data_ptr() % 16:
        w, rows = w.clone(memory_format=torch.contiguous_format), (n, k)
    codes, scales = w.new_empty((n, k), dtype=CODES), w.new_empty((-(-n // GROUP), k // GROUP), dtype=torch.float32)
    st = _launch(index, _lib().quantize_fp8_blocks, w.data_ptr(), tag, n, k, rows[1], codes.data_ptr(), scales.data_ptr(), _raw_stream(index))
    if st:
        _check(st, "quantize_fp8_weight")
    return codes, scales


def linear_fp8_workspace_bytes(m: int, n: int, k: int, codes: bool = False) -> int:
    """Workspace linear_fp8 needs for these sizes (``codes``: x is quantized already)."""
    return int(_lib().fp8_linear_workspace_bytes(E4M3 if codes else BF16, m, n, k))


def linear_fp8_tile(m: int, n: int, k: int) -> tuple[int, int, int]:
    """Rows and columns of a workgroup's tile in linear_fp8 for these sizes, each pair a kernel of its own (16 x 16: the one for
    few rows), and the parts that k is cut into ((0, 0, 0): invalid or empty sizes)."""
    columns, splits = ctypes.c_int(), ctypes.c_int()
    rows = _lib().fp8_linear_tile(m, n, k, ctypes.byref(columns), ctypes.byref(splits))
    return rows, columns.value, splits.value


@_remember
def _linear_plan(x, codes, scales, bias, x_scales, out_dtype, act):
    shape, stride, dtype = x
    act = Act(act)
    is_codes = dtype == CODES
    if is_codes and act != Act.NONE:
        raise ValueError("x of codes takes no activation")
    if is_codes != (x_scales is not None):
        raise ValueError("x_scales go with x of float8_e4m3fn codes (quantize_fp8)")
    tag = E4M3 if is_codes else _act_tag(dtype)
    out_dtype = out_dtype or (torch.bfloat16 if is_codes else dtype)
    out_tag = _act_tag(out_dtype)
    if not is_codes and out_dtype != dtype:
        raise ValueError(f"the output has x's dtype {dtype}, not {out_dtype}")
    if len(shape) < 1:
        raise ValueError("x must have at least one dimension")
    k = _width(shape[-1], act)
    m = math.prod(shape[:-1])
    if codes[2] != CODES or len(codes[0]) != 2 or codes[0][1] != k or not _dense(*codes[:2]):
        raise ValueError(f"codes must be a contiguous float8_e4m3fn [n, {k}] tensor (quantize_fp8_weight), got {tuple(codes[0])} of {codes[2]}")
    n = codes[0][0]
    if scales[2] != torch.float32 or scales[0] != (-(-n // GROUP), k // GROUP) or not _dense(*scales[:2]):
        raise ValueError(f"scales must be a contiguous float32 [{-(-n // GROUP)}, {k // GROUP}] tensor, got {tuple(scales[0])} of {scales[2]}")
    if bias is not None and (bias[2] != out_dtype or bias[0] != (n,) or (n > 1 and bias[1][0] != 1)):
        raise ValueError(f"bias must be a contiguous [{n}] tensor of {out_dtype}")
    if is_codes and (x_scales[2] != torch.float32 or x_scales[0] != (*shape[:-1], k // GROUP) or not _dense(*x_scales[:2])):
        raise ValueError(f"x_scales must be a contiguous float32 {(*shape[:-1], k // GROUP)} tensor")
    rows = _rows(shape, stride, 1 if is_codes else 2)
    need = int(_lib().fp8_linear_workspace_bytes(tag, m, n, k))
    return tag, out_tag, int(act), out_dtype, m, n, k, rows, (*shape[:-1], n), need


def linear_fp8(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, bias: torch.Tensor | None = None, act: Act = Act.NONE,
               x_scales: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y = act(x) W^T + bias on 8-bit floats: x [..., k] (bf16/f16; quantized in the
    call as by ``quantize_fp8``) -> y [..., n] of x's dtype, W = ``codes`` [n, k]
    float8_e4m3fn times ``scales`` [ceil(n / 128), k / 128] (``quantize_fp8_weight``,
    or a checkpoint's).  With ``act=Act.SWIGLU`` the rows of x are [up | gate], 2k
    values.  x of float8_e4m3fn codes comes with ``x_scales`` [..., k / 128]; y is
    then of ``out_dtype`` (default bfloat16).  See fp8_linear in include/w4a16.h."""
    tag, out_tag, act, out_dtype, m, n, k, rows, shape, need = _linear_plan(_meta(x), _meta(codes), _meta(scales), _meta(bias),
                                                                            _meta(x_scales), out_dtype, act)
    _no_grad(x, codes, scales, bias, x_scales)
    index = _device_index(x, codes, scales, bias, x_scales, workspace)
    if rows is None or x.data_ptr() % 16:
        x = x.clone(memory_format=torch.contiguous_format)
        rows = m, x.shape[-1]
    y = x.new_empty(shape, dtype=out_dtype)
    if m == 0 or n == 0:
        return y
    if codes.data_ptr() % 16:
        raise ValueError("codes must be 16-byte aligned")
    stream = _raw_stream(index)
    ws, ws_bytes = _workspace(workspace, need, index, stream)
    st = _launch(index, _lib().fp8_linear, x.data_ptr(), tag, None if x_scales is None else x_scales.data_ptr(), act, m, k, rows[1],
                 codes.data_ptr(), scales.data_ptr(), n, None if bias is None else bias.data_ptr(), y.data_ptr(), out_tag, n, ws, ws_bytes,
                 stream)
    if st:
        _check(st, "linear_fp8")
    return y
