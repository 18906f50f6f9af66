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


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _vector(t, n: int, dtype, name: str, device):
    """The address of a contiguous vector (or matrix) of n values."""
    _need(t.dtype == dtype and t.numel() == n and t.is_contiguous() and t.device == device,
          f"{name}: expected {n} contiguous {dtype} values on {device}")
    return t.data_ptr()


def _rows(t, cols: int, name: str, device):
    """(address, row stride) of [rows][cols] with contiguous rows."""
    _need(t.dim() == 2 and t.shape[1] == cols and t.device == device and (cols == 1 or t.stride(1) == 1),
          f"{name}: expected rows of {cols} contiguous values on {device}")
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else max(t.stride(0), _pad(cols, t.dtype)))


def _matrices(t, name: str, device):
    """(address, row stride) of [groups][n][k] or [n][k] whose matrices follow one another."""
    _need(t.dim() in (2, 3) and t.device == device and (t.shape[-1] == 1 or t.stride(-1) == 1),
          f"{name}: expected [groups][n][k] or [n][k] with contiguous rows on {device}")
    n, k = t.shape[-2:]
    if t.dim() == 3 and t.shape[0] > 1 and n == 1:
        ld = t.stride(0)
    else:
        ld = t.stride(-2) if n > 1 else max(t.stride(-2), _pad(k, t.dtype))
        _need(t.dim() == 2 or t.shape[0] <= 1 or t.stride(0) == n * ld,
              f"{name}: matrices have to follow one another, n rows apart")
    return t.data_ptr(), ld


def _pad(cols: int, dtype) -> int:
    unit = 16 // dtype.itemsize
    return -(-cols // unit) * unit


def _new(shape, dtype, device):
    """An empty tensor whose rows start every whole number of 16 bytes."""
    cols = shape[-1]
    ld = _pad(cols, dtype)
    t = torch.empty(*shape[:-1], ld, dtype=dtype, device=device)
    return t if ld == cols else t[..., :cols]


def _enqueue(what: str, fill, out, shape, dtype, device, stream):
    """Allocates `out` unless given, and makes the call on the right device and stream.
    fill(out) -> (function, io)."""
    if device.type != "cuda":
        raise ValueError(f"{what}: expected CUDA tensors")
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            return _enqueue(what, fill, out, shape, dtype, device, stream)
    if out is None:
        if stream is None:
            out = _new(shape, dtype, device)
        else:
            with torch.cuda.stream(stream):
                out = _new(shape, dtype, device)
    fn, io = fill(out)
    rc = fn(io, torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream)
    if rc != OK:
        raise NVFP4MoEError(rc, what)
    return out


def quantize_int8(x, *, swiglu: bool = False, q=None, scale=None, stream=None):
    """Rows to int8 with an FP32 scale each: scale = max|v| / 127, q = v / scale to the
    nearest whole number (ties to even). x: [rows][cols] bf16, f16 or f32; with `swiglu`
    [rows][2*cols] holding gate | up, and v = SiLU(gate) * up.
    Returns (q int8 [rows][cols], scale f32 [rows])."""
    _need(x.dim() == 2 and x.dtype in _TYPES and x.dtype != torch.int8, "x: expected [rows][cols] bf16, f16 or f32")
    rows, width = x.shape
    _need(width > 0 and not (swiglu and width % 2), "x: expected at least one value a row (gate | up: an even number)")
    cols = width // 2 if swiglu else width
    device = x.device
    x_ptr, x_ld = _rows(x, width, "x", device)
    if q is not None:
        _need(q.dtype == torch.int8 and q.dim() == 2 and q.shape[0] == rows, f"q: expected int8 [{rows}][{cols}]")
        _rows(q, cols, "q", device)
    if scale is not None:
        _vector(scale, rows, torch.float32, "scale", device)

    def fill(q):
        nonlocal scale
        if scale is None:
            if stream is None:
                scale = torch.empty(rows, dtype=torch.float32, device=device)
            else:
                with torch.cuda.stream(stream):
                    scale = torch.empty(rows, dtype=torch.float32, device=device)
        return nvfp4_moe_quantize_int8, QuantizeIO(rows, cols, _TYPES[x.dtype], int(swiglu), x_ptr, x_ld, q.data_ptr(),
                                                   q.stride(0) if rows > 1 else max(q.stride(0), cols), scale.data_ptr())

    q = _enqueue("nvfp4_moe_quantize_int8", fill, q, (rows, cols), torch.int8, device, stream)
    return q, scale


def _check_out(out, shape, out_dtype, device):
    if out is None:
        _need(out_dtype in _TYPES and out_dtype != torch.int8, "out_dtype: expected bf16, f16 or f32")
        return out_dtype
    _need(tuple(out.shape) == tuple(shape) and out.dtype in _TYPES and out.dtype != torch.int8
          and (out_dtype is None or out.dtype == out_dtype), f"out: expected {list(shape)}, bf16, f16 or f32")
    _need(out.device == device, f"out: expected a tensor on {device}")
    return out.dtype


def _groups(offsets, w_shape, device):
    groups = w_shape[0] if len(w_shape) == 3 else 1
    if offsets is None:
        _need(groups == 1, "offsets: needed for more than one group")
        return groups, None
    return groups, _vector(offsets, groups + 1, torch.int32, "offsets", device)


def grouped_gemm(x, w, offsets=None, *, x_scale=None, w_scale=None, out=None, out_dtype=None,
                 accumulate: bool = False, stream=None):
    """out[p] = x[p] W_e^T for the rows p of every group e. x: [rows][k], w: [groups][n][k]
    (or [n][k]), both bf16, f16, or int8 with x_scale [rows] and w_scale [groups][n] f32.
    out: [rows][n], by default of x's type (f32 for int8); rows of no group are not written.
    accumulate: out += (f32)."""
    _need(w.dim() in (2, 3) and x.dim() == 2, "expected x [rows][k] and w [groups][n][k] or [n][k]")
    _need(x.dtype == w.dtype and x.dtype in _TYPES and x.dtype != torch.float32,
          "x and w: expected the same type, bf16, f16 or int8")
    _need(not accumulate or out is not None, "accumulate: needs out")
    device, rows, (n, k) = x.device, x.shape[0], w.shape[-2:]
    groups, off = _groups(offsets, w.shape, device)
    x_ptr, x_ld = _rows(x, k, "x", device)
    w_ptr, w_ld = _matrices(w, "w", device)
    xs = ws = None
    if x.dtype == torch.int8:
        _need(x_scale is not None and w_scale is not None, "int8: needs x_scale and w_scale")
        xs = _vector(x_scale, rows, torch.float32, "x_scale", device)
        ws = _vector(w_scale, groups * n, torch.float32, "w_scale", device)
    else:
        _need(x_scale is None and w_scale is None, "x_scale, w_scale: for int8 only")
    if out is None and out_dtype is None:
        out_dtype = torch.float32 if x.dtype == torch.int8 else x.dtype
    dtype = _check_out(out, (rows, n), out_dtype, device)

    def fill(out):
        o_ptr, o_ld = _rows(out, n, "out", device)
        return nvfp4_moe_grouped_gemm, GemmIO(groups, rows, n, k, _TYPES[x.dtype], _TYPES[dtype], int(accumulate), off,
                                              x_ptr, x_ld, xs, None, 0, w_ptr, w_ld, ws, o_ptr, o_ld)

    return _enqueue("nvfp4_moe_grouped_gemm", fill, out, (rows, n), dtype, device, stream)


def gemm_int8(x, w, x_scale, w_scale, *, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """out[t][j] = x_scale[t] * w_scale[j] * sum_k x[t][k] w[j][k], the sum exact. x: [rows][k]
    int8, w: [n][k] int8, scales f32. out: [rows][n], f32 by default. accumulate: out += (f32)."""
    _need(x.dtype == torch.int8 and w.dtype == torch.int8 and w.dim() == 2, "expected int8 x [rows][k] and w [n][k]")
    return grouped_gemm(x, w, None, x_scale=x_scale, w_scale=w_scale, out=out, out_dtype=out_dtype,
                        accumulate=accumulate, stream=stream)


def grouped_gemm_dx(dy, w, offsets=None, *, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """The gradient of grouped_gemm for x: dx[p] = dy[p] W_e. dy: [rows][n], w: [groups][n][k],
    both bf16 or f16. out: [rows][k], by default of dy's type; rows of no group are not written."""
    _need(w.dim() in (2, 3) and dy.dim() == 2, "expected dy [rows][n] and w [groups][n][k] or [n][k]")
    _need(dy.dtype == w.dtype and dy.dtype in (torch.bfloat16, torch.float16), "dy and w: expected the same type, bf16 or f16")
    _need(not accumulate or out is not None, "accumulate: needs out")
    device, rows, (n, k) = dy.device, dy.shape[0], w.shape[-2:]
    groups, off = _groups(offsets, w.shape, device)
    dy_ptr, dy_ld = _rows(dy, n, "dy", device)
    w_ptr, w_ld = _matrices(w, "w", device)
    dtype = _check_out(out, (rows, k), out_dtype or (None if out is not None else dy.dtype), device)

    def fill(out):
        o_ptr, o_ld = _rows(out, k, "out", device)
        return nvfp4_moe_grouped_gemm_dx, GemmIO(groups, rows, n, k, _TYPES[dy.dtype], _TYPES[dtype], int(accumulate), off,
                                                 None, 0, None, dy_ptr, dy_ld, w_ptr, w_ld, None, o_ptr, o_ld)

    return _enqueue("nvfp4_moe_grouped_gemm_dx", fill, out, (rows, k), dtype, device, stream)


def grouped_gemm_dw(dy, x, offsets=None, *, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """The gradient of grouped_gemm for w: dW_e = sum over the rows p of e of dy[p]^T x[p].
    dy: [rows][n], x: [rows][k], both bf16 or f16. out: [groups][n][k] ([n][k] without
    offsets), f32 by default; zeros for a group without rows. accumulate: out += (f32)."""
    _need(dy.dim() == 2 and x.dim() == 2 and dy.shape[0] == x.shape[0], "expected dy [rows][n] and x [rows][k]")
    _need(dy.dtype == x.dtype and dy.dtype in (torch.bfloat16, torch.float16), "dy and x: expected the same type, bf16 or f16")
    _need(not accumulate or out is not None, "accumulate: needs out")
    _need(offsets is None or (offsets.dim() == 1 and offsets.numel() >= 2), "offsets: expected groups + 1 entries")
    device, rows, n, k = x.device, x.shape[0], dy.shape[1], x.shape[1]
    shape = (n, k) if offsets is None else (offsets.numel() - 1, n, k)
    groups, off = _groups(offsets, shape, device)
    dy_ptr, dy_ld = _rows(dy, n, "dy", device)
    x_ptr, x_ld = _rows(x, k, "x", device)
    dtype = _check_out(out, shape, out_dtype or (None if out is not None else torch.float32), device)

    def fill(out):
        o_ptr, o_ld = _matrices(out, "out", device)
        return nvfp4_moe_grouped_gemm_dw, GemmIO(groups, rows, n, k, _TYPES[x.dtype], _TYPES[dtype], int(accumulate), off,
                                                 x_ptr, x_ld, None, dy_ptr, dy_ld, None, 0, None, o_ptr, o_ld)

    return _enqueue("nvfp4_moe_grouped_gemm_dw", fill, out, shape, dtype, device, stream)
