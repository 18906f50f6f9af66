"""The 8-bit and the ragged matrix products of include/nvfp4_moe_products.h on torch
tensors: argument marshalling only, like the layer's own binding.

Rows are sorted by group: rows ``offsets[e] .. offsets[e+1]-1`` belong to group (expert)
``e``; ``offsets`` is an int32 CUDA tensor of ``groups + 1`` entries that is never read
back, or None for one group of all rows. Matrices are ``[groups][n][k]`` (``[n][k]`` for
one group), as the layer's own expert planes are. Rows are contiguous and start every
whole number of 16 bytes; outputs that these functions allocate do too, so they can be
the next product's input.

Every call enqueues on `stream` (default: torch's current stream on the tensors' device),
never synchronises, and raises NVFP4MoEError for what the library refuses. Given another
stream than the current one, keep the inputs alive until it is done with them; outputs
are allocated on it.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import OK, NVFP4MoEError, lib

TYPE_BF16, TYPE_F16, TYPE_F32, TYPE_INT8 = 0, 1, 2, 3
INT8_MAX_K = 131071
MAX_GROUPS = 1024
_TYPES = {torch.bfloat16: TYPE_BF16, torch.float16: TYPE_F16, torch.float32: TYPE_F32, torch.int8: TYPE_INT8}


class QuantizeIO(C.Structure):
    _fields_ = [("rows", C.c_int32), ("cols", C.c_int32), ("in_type", C.c_int), ("swiglu", C.c_int32),
                ("in_", C.c_void_p), ("in_stride", C.c_int64), ("q", C.c_void_p), ("q_stride", C.c_int64),
                ("scale", C.c_void_p)]


class GemmIO(C.Structure):
    _fields_ = [("groups", C.c_int32), ("rows", C.c_int32), ("n", C.c_int32), ("k", C.c_int32),
                ("type", C.c_int), ("out_type", C.c_int), ("accumulate", C.c_int32), ("offsets", C.c_void_p),
                ("x", C.c_void_p), ("x_stride", C.c_int64), ("x_scale", C.c_void_p), ("dy", C.c_void_p),
                ("dy_stride", C.c_int64), ("w", C.c_void_p), ("w_stride", C.c_int64), ("w_scale", C.c_void_p),
                ("out", C.c_void_p), ("out_stride", C.c_int64)]


def nvfp4_moe_quantize_int8(io: QuantizeIO, stream: int) -> int:
    return lib().nvfp4_moe_quantize_int8(C.byref(io), C.c_void_p(stream))


def nvfp4_moe_grouped_gemm(io: GemmIO, stream: int) -> int:
    return lib().nvfp4_moe_grouped_gemm(C.byref(io), C.c_void_p(stream))


def nvfp4_moe_grouped_gemm_dx(io: GemmIO, stream: int) -> int:
    return lib().nvfp4_moe_grouped_gemm_dx(C.byref(io), C.c_void_p(stream))


def nvfp4_moe_grouped_gemm_dw(io: GemmIO, stream: int) -> int:
    return lib().nvfp4_moe_grouped_gemm_dw(C.byref(io), C.c_void_p(stream))


def nvfp4_moe_products_status(stream: int) -> int:
    return lib().nvfp4_moe_products_status(C.c_void_p(stream))


# ---------------------------------------------------------------- torch glue

def products_status(stream=None) -> int:
    """Synchronises and returns the first device-side error of the products on the current
    device since the last read (0 if none), clearing it."""
    return nvfp4_moe_products_status((stream if stream is not None else torch.cuda.current_stream()).cuda_stream)


# These run before every launch, so what a good call needs is kept short: messages are put
# together only where a check fails.

_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream   # torch.cuda.current_stream().cuda_stream, without its object
_UNIT = {torch.bfloat16: 8, torch.float16: 8, torch.float32: 4, torch.int8: 16}   # values in 16 bytes


def _device_of(t, what: str) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{what}: expected CUDA tensors")
    return index


def _vector(t, n: int, dtype, name: str, index: int) -> int:
    """The address of n contiguous values."""
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name}: expected {n} contiguous {dtype} values on cuda:{index}")
    return t.data_ptr()


def _row_stride(t, rows: int, cols: int, name: str, index: int) -> int:
    """The row stride of [rows][cols] with contiguous rows."""
    if t.dim() != 2 or t.get_device() != index:
        raise ValueError(f"{name}: expected a matrix on cuda:{index}")
    ld, step = t.stride()
    if step != 1 and cols != 1:
        raise ValueError(f"{name}: expected contiguous rows")
    return ld if rows > 1 else _pad(cols, t.dtype)   # one row: no stride to take


def _matrix_stride(t, groups: int, n: int, k: int, name: str, index: int) -> int:
    """The row stride of [groups][n][k] or [n][k] whose matrices follow one another."""
    if t.get_device() != index:
        raise ValueError(f"{name}: expected a tensor on cuda:{index}")
    stride = t.stride()
    if stride[-1] != 1 and k != 1:
        raise ValueError(f"{name}: expected contiguous rows")
    if n > 1:
        ld = stride[-2]
    else:
        ld = stride[0] if groups > 1 else _pad(k, t.dtype)
    if groups > 1 and stride[0] != n * ld:
        raise ValueError(f"{name}: matrices have to follow one another, n rows apart")
    return ld


def _pad(cols: int, dtype) -> int:
    unit = _UNIT[dtype]
    return -(-cols // unit) * unit


def _new(shape, dtype, index: int, stream):
    """An empty tensor whose rows start every whole number of 16 bytes, allocated on `stream`."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _new(shape, dtype, index, None)
    cols = shape[-1]
    ld = _pad(cols, dtype)
    t = torch.empty((*shape[:-1], ld), dtype=dtype, device=index)
    return t if ld == cols else t[..., :cols]


def _enqueue(fn, io, index: int, stream, what: str) -> None:
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        rc = fn(C.byref(io), s)
    else:
        with torch.cuda.device(index):
            rc = fn(C.byref(io), s)
    if rc != OK:
        raise NVFP4MoEError(rc, what)


def quantize_int8(x, *, swiglu: bool = False, q=None, scale=None, stream=None):
    """Rows to int8 with an FP32 scale each: scale = max|v| / 127, q = v / scale to the
    nearest whole number (ties to even). x: [rows][cols] bf16, f16 or f32; with `swiglu`
    [rows][2*cols] holding gate | up, and v = SiLU(gate) * up.
    Returns (q int8 [rows][cols], scale f32 [rows])."""
    t = _TYPES.get(x.dtype, TYPE_INT8)
    if x.dim() != 2 or t == TYPE_INT8:
        raise ValueError("x: expected [rows][cols] bf16, f16 or f32")
    rows, width = x.shape
    if width == 0 or (swiglu and width % 2):
        raise ValueError("x: expected at least one value a row (gate | up: an even number)")
    cols = width // 2 if swiglu else width
    index = _device_of(x, "quantize_int8")
    x_ld = _row_stride(x, rows, width, "x", index)
    if q is None:
        q = _new((rows, cols), torch.int8, index, stream)
    elif q.dtype != torch.int8 or tuple(q.shape) != (rows, cols):
        raise ValueError(f"q: expected int8 [{rows}][{cols}]")
    q_ld = _row_stride(q, rows, cols, "q", index)
    if scale is None:
        if stream is None:
            scale = torch.empty(rows, dtype=torch.float32, device=index)
        else:
            with torch.cuda.stream(stream):
                scale = torch.empty(rows, dtype=torch.float32, device=index)
        s_ptr = scale.data_ptr()
    else:
        s_ptr = _vector(scale, rows, torch.float32, "scale", index)
    io = QuantizeIO(rows, cols, t, 1 if swiglu else 0, x.data_ptr(), x_ld, q.data_ptr(), q_ld, s_ptr)
    _enqueue(lib().nvfp4_moe_quantize_int8, io, index, stream, "nvfp4_moe_quantize_int8")
    return q, scale


def _out_type(out, shape, out_dtype) -> int:
    """The output's type, checked against what the caller asked for."""
    t = _TYPES.get(out_dtype if out is None else out.dtype, TYPE_INT8)
    if t == TYPE_INT8:
        raise ValueError("out, out_dtype: expected bf16, f16 or f32")
    if out is not None and (tuple(out.shape) != shape or (out_dtype is not None and out.dtype != out_dtype)):
        raise ValueError(f"out: expected {list(shape)}" + (f" of {out_dtype}" if out_dtype is not None else ""))
    return t


def _offsets(offsets, groups: int, index: int):
    if offsets is None:
        if groups != 1:
            raise ValueError("offsets: needed for more than one group")
        return None
    return _vector(offsets, groups + 1, torch.int32, "offsets", index)


def _operands(x, w, names: str):
    """(groups, rows, n, k) of rows x and matrices w."""
    if x.dim() != 2 or w.dim() not in (2, 3) or x.dtype != w.dtype:
        raise ValueError(f"{names}: expected a matrix of rows, [groups][n][k] or [n][k], and one type")
    n, k = w.shape[-2:]
    return (w.shape[0] if w.dim() == 3 else 1), x.shape[0], n, k


def grouped_gemm(x, w, offsets=None, *, x_scale=None, w_scale=None, out=None, out_dtype=None,
                 accumulate: bool = False, stream=None):
    """out[p] = x[p] W_e^T for the rows p of every group e. x: [rows][k], w: [groups][n][k]
    (or [n][k]), both bf16, f16, or int8 with x_scale [rows] and w_scale [groups][n] f32.
    out: [rows][n], by default of x's type (f32 for int8); rows of no group are not written.
    accumulate: out += (f32)."""
    groups, rows, n, k = _operands(x, w, "x, w")
    t = _TYPES.get(x.dtype, TYPE_F32)
    if t == TYPE_F32 or x.shape[1] != k:
        raise ValueError("x, w: expected [rows][k] and [groups][n][k], bf16, f16 or int8")
    index = _device_of(x, "grouped_gemm")
    off = _offsets(offsets, groups, index)
    x_ld = _row_stride(x, rows, k, "x", index)
    w_ld = _matrix_stride(w, groups, n, k, "w", index)
    xs = ws = None
    if t == TYPE_INT8:
        if x_scale is None or w_scale is None:
            raise ValueError("int8: needs x_scale and w_scale")
        xs = _vector(x_scale, rows, torch.float32, "x_scale", index)
        ws = _vector(w_scale, groups * n, torch.float32, "w_scale", index)
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale, w_scale: for int8 only")
    if out is None:
        if accumulate:
            raise ValueError("accumulate: needs out")
        if out_dtype is None:
            out_dtype = torch.float32 if t == TYPE_INT8 else x.dtype
        o = _out_type(None, None, out_dtype)
        out = _new((rows, n), out_dtype, index, stream)
    else:
        o = _out_type(out, (rows, n), out_dtype)
    io = GemmIO(groups, rows, n, k, t, o, 1 if accumulate else 0, off, x.data_ptr(), x_ld, xs, None, 0, w.data_ptr(), w_ld,
                ws, out.data_ptr(), _row_stride(out, rows, n, "out", index))
    _enqueue(lib().nvfp4_moe_grouped_gemm, io, index, stream, "nvfp4_moe_grouped_gemm")
    return out


def gemm_int8(x, w, x_scale, w_scale, *, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """out[t][j] = x_scale[t] * w_scale[j] * sum_k x[t][k] w[j][k], the sum exact. x: [rows][k]
    int8, w: [n][k] int8, scales f32. out: [rows][n], f32 by default. accumulate: out += (f32)."""
    if x.dtype != torch.int8 or w.dim() != 2:
        raise ValueError("x, w: expected int8 [rows][k] and [n][k]")
    return grouped_gemm(x, w, None, x_scale=x_scale, w_scale=w_scale, out=out, out_dtype=out_dtype,
                        accumulate=accumulate, stream=stream)


def grouped_gemm_dx(dy, w, offsets=None, *, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """The gradient of grouped_gemm for x: dx[p] = dy[p] W_e. dy: [rows][n], w: [groups][n][k],
    both bf16 or f16. out: [rows][k], by default of dy's type; rows of no group are not written."""
    groups, rows, n, k = _operands(dy, w, "dy, w")
    t = _TYPES.get(dy.dtype, TYPE_F32)
    if t not in (TYPE_BF16, TYPE_F16) or dy.shape[1] != n:
        raise ValueError("dy, w: expected [rows][n] and [groups][n][k], bf16 or f16")
    index = _device_of(dy, "grouped_gemm_dx")
    off = _offsets(offsets, groups, index)
    dy_ld = _row_stride(dy, rows, n, "dy", index)
    w_ld = _matrix_stride(w, groups, n, k, "w", index)
    if out is None:
        if accumulate:
            raise ValueError("accumulate: needs out")
        out_dtype = dy.dtype if out_dtype is None else out_dtype
        o = _out_type(None, None, out_dtype)
        out = _new((rows, k), out_dtype, index, stream)
    else:
        o = _out_type(out, (rows, k), out_dtype)
    io = GemmIO(groups, rows, n, k, t, o, 1 if accumulate else 0, off, None, 0, None, dy.data_ptr(), dy_ld, w.data_ptr(), w_ld,
                None, out.data_ptr(), _row_stride(out, rows, k, "out", index))
    _enqueue(lib().nvfp4_moe_grouped_gemm_dx, io, index, stream, "nvfp4_moe_grouped_gemm_dx")
    return out


def grouped_gemm_dw(dy, x, offsets=None, *, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """The gradient of grouped_gemm for w: dW_e = sum over the rows p of e of dy[p]^T x[p].
    dy: [rows][n], x: [rows][k], both bf16 or f16. out: [groups][n][k] ([n][k] without
    offsets), f32 by default; zeros for a group without rows. accumulate: out += (f32)."""
    t = _TYPES.get(dy.dtype, TYPE_F32)
    if dy.dim() != 2 or x.dim() != 2 or dy.shape[0] != x.shape[0] or dy.dtype != x.dtype or t not in (TYPE_BF16, TYPE_F16):
        raise ValueError("dy, x: expected [rows][n] and [rows][k], both bf16 or f16")
    index = _device_of(x, "grouped_gemm_dw")
    (rows, k), n = x.shape, dy.shape[1]
    groups = 1 if offsets is None else offsets.numel() - 1
    off = _offsets(offsets, groups, index)
    dy_ld = _row_stride(dy, rows, n, "dy", index)
    x_ld = _row_stride(x, rows, k, "x", index)
    shape = (n, k) if offsets is None else (groups, n, k)
    if out is None:
        if accumulate:
            raise ValueError("accumulate: needs out")
        out_dtype = torch.float32 if out_dtype is None else out_dtype
        o = _out_type(None, None, out_dtype)
        out = _new(shape, out_dtype, index, stream)
    else:
        o = _out_type(out, shape, out_dtype)
    io = GemmIO(groups, rows, n, k, t, o, 1 if accumulate else 0, off, x.data_ptr(), x_ld, None, dy.data_ptr(), dy_ld, None, 0,
                None, out.data_ptr(), _matrix_stride(out, groups, n, k, "out", index))
    _enqueue(lib().nvfp4_moe_grouped_gemm_dw, io, index, stream, "nvfp4_moe_grouped_gemm_dw")
    return out
