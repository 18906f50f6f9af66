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
are allocated on it. What goes wrong on the device, a product's bounded wait that gave up,
is told by `products_status()`.

Nothing is recorded for autograd: outputs are detached, whatever the inputs require. The
gradients are calls of their own, for a torch.autograd.Function or a training step that is
written out.
"""
from __future__ import annotations

import ctypes as C
import importlib.util
import os
import struct

import torch

from . import ERR, OK, NVFP4MoEError, build, lib

TYPE_BF16, TYPE_F16, TYPE_F32, TYPE_INT8 = 0, 1, 2, 3
INT8_MAX_K = 131071
MAX_GROUPS = 1024
MAX_EXTENT = 1 << 30
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


def nvfp4_moe_test_products_stall(n: int) -> None:
    """Test hook (include/nvfp4_moe_test.h): waits of the next n tile launches run out."""
    lib().nvfp4_moe_test_products_stall(C.c_int32(n))


def products_status(stream=None) -> int:
    """Synchronises and returns the first device-side error of the products on the current
    device since the last read (0 if none), clearing it."""
    return nvfp4_moe_products_status((stream if stream is not None else torch.cuda.current_stream()).cuda_stream)


# ---------------------------------------------------------------- torch glue
#
# These run before every launch, and a decode product takes the GPU two or three
# microseconds: what a good call needs is written out and kept short, the structures are
# packed rather than built field by field, and messages are put together only where a check
# fails.

_current_device = torch._C._cuda_getDevice         # torch.cuda.current_device() (a CUDA tensor is at hand: no set-up to do)
_raw_stream = torch._C._cuda_getCurrentRawStream   # torch.cuda.current_stream().cuda_stream, without its object
_empty = torch.empty_strided   # half the time of torch.empty, and it pads rows without a view
_UNIT = {torch.bfloat16: 8, torch.float16: 8, torch.float32: 4, torch.int8: 16}   # values in 16 bytes
_pack_gemm = struct.Struct("@7iPPqPPqPqPPq").pack     # GemmIO
_pack_quantize = struct.Struct("@4iPqPqP").pack       # QuantizeIO


def _load_marshal():
    """csrc/marshal.cpp: the common calls, natively; without it they take the Python below."""
    path = build.marshal_path()
    if not os.path.exists(path):
        return None
    spec = importlib.util.spec_from_file_location(f"{__package__}._marshal", path)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError:
        return None
    return module


_marshal = _load_marshal()
_native = None   # _marshal, once the library is loaded


def _set_up():
    global _native
    if _marshal is not None:
        L = lib()
        _marshal.setup(*[C.cast(getattr(L, f), C.c_void_p).value
                         for f in ("nvfp4_moe_grouped_gemm", "nvfp4_moe_grouped_gemm_dx", "nvfp4_moe_grouped_gemm_dw",
                                   "nvfp4_moe_quantize_int8")])
        _native = _marshal


def _refuse(what: str):
    raise ValueError(what)


def _vector(t, n: int, dtype, name: str, index: int) -> int:
    """The address of n contiguous values."""
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != index:
        _refuse(f"{name}: expected {n} contiguous {dtype} values on cuda:{index}")
    return t.data_ptr()


def _rows(t, index: int, name: str):
    """(rows, cols, row stride) of a matrix with contiguous rows."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or t.get_device() != index or (stride[1] != 1 and shape[1] != 1):
        _refuse(f"{name}: expected a matrix with contiguous rows on cuda:{index}")
    rows, cols = shape
    if rows > 1:
        return rows, cols, stride[0]
    unit = _UNIT[t.dtype]
    return rows, cols, (cols + unit - 1) & -unit   # one row: no stride to take


def _matrices(t, index: int, name: str):
    """(groups, n, k, row stride) of [groups][n][k] or [n][k] whose matrices follow one another."""
    shape, stride = t.shape, t.stride()
    if t.get_device() != index:
        _refuse(f"{name}: expected a tensor on cuda:{index}")
    if len(shape) == 2:
        n, k = shape
        groups, ld = 1, stride[0]
    elif len(shape) == 3:
        groups, n, k = shape
        ld = stride[1]
        if groups > 1:
            if n == 1:
                ld = stride[0]
            elif stride[0] != n * ld:
                _refuse(f"{name}: matrices have to follow one another, n rows apart")
    else:
        _refuse(f"{name}: expected [groups][n][k] or [n][k]")
    if stride[-1] != 1 and k != 1:
        _refuse(f"{name}: expected contiguous rows")
    if n <= 1 and groups <= 1:
        unit = _UNIT[t.dtype]
        ld = (k + unit - 1) & -unit
    return groups, n, k, ld


def _offsets(offsets, groups: int, index: int) -> int:
    if offsets is None:
        if groups != 1:
            _refuse("offsets: needed for more than one group")
        return 0
    return _vector(offsets, groups + 1, torch.int32, "offsets", index)


def _output(out, shape, dtype, accumulate: bool, index: int, stream):
    """(output, its type, its row stride): `out` checked, or a new tensor whose rows start every
    whole number of 16 bytes, allocated on `stream`."""
    if out is None:
        if accumulate:
            _refuse("accumulate: needs out")
        t = _TYPES.get(dtype, TYPE_INT8)
        if t == TYPE_INT8:
            _refuse("out_dtype: expected bf16, f16 or f32")
        if stream is not None or len(shape) == 3:
            out, ld = _new(shape, dtype, index, stream)
        else:
            unit = _UNIT[dtype]
            ld = (shape[1] + unit - 1) & -unit
            out = _empty(shape, (ld, 1), dtype=dtype, device=index)
        return out, t, ld
    t = _TYPES.get(out.dtype, TYPE_INT8)
    if t == TYPE_INT8 or tuple(out.shape) != tuple(shape) or (dtype is not None and out.dtype != dtype):
        _refuse(f"out: expected {list(shape)} of {dtype or 'bf16, f16 or f32'}")
    return out, t, (_matrices if len(shape) == 3 else _rows)(out, index, "out")[-1]


def _new(shape, dtype, index: int, stream):
    """(empty tensor whose rows start every whole number of 16 bytes, row stride)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _new(shape, dtype, index, None)
    unit = _UNIT[dtype]
    ld = (shape[-1] + unit - 1) & -unit
    return _empty(shape, (ld, 1) if len(shape) == 2 else (shape[1] * ld, ld, 1), dtype=dtype, device=index), ld


def _failed(rc: int, what: str):
    if ERR.get(rc) == "MISALIGNED":
        what += " (operands of a product start every row on a multiple of 16 bytes: copy into a matrix with padded rows," \
                " torch.empty(rows, padded)[:, :cols]; outputs, scales and offsets on one of their type's size)"
    raise NVFP4MoEError(rc, what)


def _enqueue(fn, io: bytes, index: int, stream, what: str) -> None:
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        rc = fn(io, s)
    else:
        with torch.cuda.device(index):
            rc = fn(io, s)
    if rc != OK:
        _failed(rc, what)
    if _native is None:
        _set_up()


def quantize_int8(x, *, swiglu: bool = False, q=None, scale=None, stream=None):
    """Rows to int8 with an FP32 scale each: scale = max|v| / 127, q = v / scale to the
    nearest whole number (ties to even). x: [rows][cols] bf16, f16 or f32; with `swiglu`
    [rows][2*cols] holding gate | up, and v = SiLU(gate) * up.
    Returns (q int8 [rows][cols], scale f32 [rows])."""
    if _native is not None and q is None and scale is None and stream is None:
        r = _native.quantize(x, swiglu)
        if type(r) is tuple:
            return r
        if r is not None:
            _failed(r, "nvfp4_moe_quantize_int8")
    t, index = _TYPES.get(x.dtype, TYPE_INT8), x.get_device()
    if t == TYPE_INT8 or index < 0:
        _refuse("quantize_int8: expected a CUDA tensor [rows][cols], bf16, f16 or f32")
    rows, cols, x_ld = _rows(x, index, "x")
    if swiglu:
        if cols % 2:
            _refuse("x: gate | up are an even number of values")
        cols //= 2
    if cols == 0:
        _refuse("x: expected at least one value a row")
    if q is None:
        q, q_ld = _new((rows, cols), torch.int8, index, stream)
    else:
        if q.dtype is not torch.int8 or tuple(q.shape) != (rows, cols):
            _refuse(f"q: expected int8 [{rows}][{cols}]")
        q_ld = _rows(q, index, "q")[2]
    if scale is not None:
        s_ptr = _vector(scale, rows, torch.float32, "scale", index)
    else:
        if stream is None:
            scale = _empty((rows,), (1,), dtype=torch.float32, device=index)
        else:
            with torch.cuda.stream(stream):
                scale = _empty((rows,), (1,), dtype=torch.float32, device=index)
        s_ptr = scale.data_ptr()
    io = _pack_quantize(rows, cols, t, 1 if swiglu else 0, x.data_ptr(), x_ld, q.data_ptr(), q_ld, s_ptr)
    _enqueue(lib().nvfp4_moe_quantize_int8, io, index, stream, "nvfp4_moe_quantize_int8")
    return q, scale


def grouped_gemm(x, w, offsets=None, *, x_scale=None, w_scale=None, out=None, out_dtype=None,
                 accumulate: bool = False, stream=None):
    """out[p] = x[p] W_e^T for the rows p of every group e. x: [rows][k], w: [groups][n][k]
    (or [n][k]), both bf16, f16, or int8 with x_scale [rows] and w_scale [groups][n] f32.
    out: [rows][n], by default of x's type (f32 for int8); rows of no group are not written.
    accumulate: out += (f32)."""
    return _product(x, w, offsets, x_scale, w_scale, out, out_dtype, accumulate, stream)


def _product(x, w, offsets, x_scale, w_scale, out, out_dtype, accumulate, stream):
    if _native is not None and out is None and stream is None and not accumulate:
        r = _native.product(0, x, w, offsets, x_scale, w_scale, out_dtype)
        if r is not None:
            return r if type(r) is not int else _failed(r, "nvfp4_moe_grouped_gemm")
    dtype, index = x.dtype, x.get_device()
    t = _TYPES.get(dtype, TYPE_F32)
    if index < 0 or t == TYPE_F32 or w.dtype is not dtype:
        _refuse("grouped_gemm: expected CUDA tensors of one type, bf16, f16 or int8")
    rows, cols, x_ld = _rows(x, index, "x")
    groups, n, k, w_ld = _matrices(w, index, "w")
    if cols != k:
        _refuse(f"x, w: rows of {cols} and of {k} values")
    xs = ws = 0
    if t == TYPE_INT8:
        if x_scale is None or w_scale is None:
            _refuse("int8: needs x_scale and w_scale")
        xs = _vector(x_scale, rows, torch.float32, "x_scale", index)
        ws = _vector(w_scale, groups * n, torch.float32, "w_scale", index)
        dtype = torch.float32
    elif x_scale is not None or w_scale is not None:
        _refuse("x_scale, w_scale: for int8 only")
    off = _offsets(offsets, groups, index)
    if out is None and out_dtype is None:
        out_dtype = dtype
    out, o, o_ld = _output(out, (rows, n), out_dtype, accumulate, index, stream)
    io = _pack_gemm(groups, rows, n, k, t, o, 1 if accumulate else 0, off, x.data_ptr(), x_ld, xs, 0, 0, w.data_ptr(), w_ld, ws,
                    out.data_ptr(), o_ld)
    _enqueue(lib().nvfp4_moe_grouped_gemm, io, index, stream, "nvfp4_moe_grouped_gemm")
    return out


def gemm_int8(x, w, x_scale, w_scale, *, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """out[t][j] = x_scale[t] * w_scale[j] * sum_k x[t][k] w[j][k], the sum exact. x: [rows][k]
    int8, w: [n][k] int8, scales f32. out: [rows][n], f32 by default. accumulate: out += (f32)."""
    if x.dtype is not torch.int8 or w.dim() != 2:
        _refuse("x, w: expected int8 [rows][k] and [n][k]")
    return _product(x, w, None, x_scale, w_scale, out, out_dtype, accumulate, stream)


def grouped_gemm_dx(dy, w, offsets=None, *, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """The gradient of grouped_gemm for x: dx[p] = dy[p] W_e. dy: [rows][n], w: [groups][n][k],
    both bf16 or f16. out: [rows][k], by default of dy's type; rows of no group are not written."""
    if _native is not None and out is None and stream is None and not accumulate:
        r = _native.product(1, dy, w, offsets, None, None, out_dtype)
        if r is not None:
            return r if type(r) is not int else _failed(r, "nvfp4_moe_grouped_gemm_dx")
    dtype, index = dy.dtype, dy.get_device()
    t = _TYPES.get(dtype, TYPE_F32)
    if index < 0 or t > TYPE_F16 or w.dtype is not dtype:
        _refuse("grouped_gemm_dx: expected CUDA tensors of one type, bf16 or f16")
    rows, cols, dy_ld = _rows(dy, index, "dy")
    groups, n, k, w_ld = _matrices(w, index, "w")
    if cols != n:
        _refuse(f"dy, w: rows of {cols} values and matrices of {n} rows")
    off = _offsets(offsets, groups, index)
    if out is None and out_dtype is None:
        out_dtype = dtype
    out, o, o_ld = _output(out, (rows, k), out_dtype, accumulate, index, stream)
    io = _pack_gemm(groups, rows, n, k, t, o, 1 if accumulate else 0, off, 0, 0, 0, dy.data_ptr(), dy_ld, w.data_ptr(), w_ld, 0,
                    out.data_ptr(), o_ld)
    _enqueue(lib().nvfp4_moe_grouped_gemm_dx, io, index, stream, "nvfp4_moe_grouped_gemm_dx")
    return out


def grouped_gemm_dw(dy, x, offsets=None, *, out=None, out_dtype=None, accumulate: bool = False, stream=None):
    """The gradient of grouped_gemm for w: dW_e = sum over the rows p of e of dy[p]^T x[p].
    dy: [rows][n], x: [rows][k], both bf16 or f16. out: [groups][n][k] ([n][k] without
    offsets), f32 by default; zeros for a group without rows. accumulate: out += (f32)."""
    if _native is not None and out is None and stream is None and not accumulate:
        r = _native.product(2, dy, x, offsets, None, None, out_dtype)
        if r is not None:
            return r if type(r) is not int else _failed(r, "nvfp4_moe_grouped_gemm_dw")
    dtype, index = x.dtype, x.get_device()
    t = _TYPES.get(dtype, TYPE_F32)
    if index < 0 or t > TYPE_F16 or dy.dtype is not dtype:
        _refuse("grouped_gemm_dw: expected CUDA tensors of one type, bf16 or f16")
    rows, k, x_ld = _rows(x, index, "x")
    dy_rows, n, dy_ld = _rows(dy, index, "dy")
    if dy_rows != rows:
        _refuse(f"dy, x: {dy_rows} and {rows} rows")
    groups = 1 if offsets is None else offsets.numel() - 1
    if groups < 1:
        _refuse("offsets: expected one more than there are groups")
    off = _offsets(offsets, groups, index)
    if out is None and out_dtype is None:
        out_dtype = torch.float32
    out, o, o_ld = _output(out, (n, k) if offsets is None else (groups, n, k), out_dtype, accumulate, index, stream)
    io = _pack_gemm(groups, rows, n, k, t, o, 1 if accumulate else 0, off, x.data_ptr(), x_ld, 0, dy.data_ptr(), dy_ld, 0, 0, 0,
                    out.data_ptr(), o_ld)
    _enqueue(lib().nvfp4_moe_grouped_gemm_dw, io, index, stream, "nvfp4_moe_grouped_gemm_dw")
    return out
