// The common case of products.py's calls, marshalled natively: plain CUDA tensors on the
// current device and its current stream, a new output. A decode product takes the GPU two
// or three microseconds and its launch three; reading four tensors' attributes and packing
// the call in Python took another four.
//
// Whatever is not that case (another device or stream, a given output, a tensor subclass,
// an argument that is refused) is answered with None and taken by the Python code, which
// checks, explains and refuses; nothing is decided here alone. The library's functions come
// in as addresses, so this module needs torch and Python, the library neither.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "nvfp4_moe_products.h"

namespace {

typedef int (*GemmFn)(const nvfp4_moe_gemm_io *, void *);
typedef int (*QuantizeFn)(const nvfp4_moe_quantize_io *, void *);
GemmFn g_gemm[3];   // product, dx, dw
QuantizeFn g_quantize;

// The tensor behind a plain torch.Tensor or Parameter, else null.
const at::Tensor *plain(PyObject *o) {
    if (!THPVariable_CheckTypeExact(Py_TYPE(o))) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    return t.is_cuda() && t.layout() == at::kStrided ? &t : nullptr;
}

int type_of(at::ScalarType t) {
    return t == at::kBFloat16 ? NVFP4_MOE_TYPE_BF16
           : t == at::kHalf   ? NVFP4_MOE_TYPE_F16
           : t == at::kFloat  ? NVFP4_MOE_TYPE_F32
           : t == at::kChar   ? NVFP4_MOE_TYPE_INT8
                              : -1;
}

int64_t padded(int64_t cols, at::ScalarType t) {
    const int64_t unit = 16 / (int64_t)c10::elementSize(t);
    return (cols + unit - 1) / unit * unit;
}

// [rows][cols] with contiguous rows: their stride.
bool row_stride(const at::Tensor &t, int64_t *ld) {
    if (t.dim() != 2 || (t.stride(1) != 1 && t.size(1) != 1)) return false;
    *ld = t.size(0) > 1 ? t.stride(0) : padded(t.size(1), t.scalar_type());
    return true;
}

// `n` contiguous values of a type on device `index`.
bool vector(const at::Tensor *t, int64_t n, at::ScalarType type, int index) {
    return t && t->scalar_type() == type && t->numel() == n && t->is_contiguous() && t->get_device() == index;
}

at::Tensor rows_of(at::IntArrayRef sizes, at::ScalarType type, c10::Device device) {
    const int64_t ld = padded(sizes.back(), type);
    const at::TensorOptions options = at::TensorOptions().dtype(type).device(device);
    return sizes.size() == 2 ? at::empty_strided(sizes, {ld, 1}, options)
                             : at::empty_strided(sizes, {sizes[1] * ld, ld, 1}, options);
}

bool fits(int64_t v) { return v >= 0 && v <= NVFP4_MOE_MAX_EXTENT; }

// product(mode, a, b, offsets, x_scale, w_scale, out_dtype) -> output, a status, or None.
// a, b: x, w (0, the product), dy, w (1, dx), dy, x (2, dw).
PyObject *product(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    if (n_args != 7) Py_RETURN_NONE;
    const long mode = PyLong_AsLong(args[0]);
    const at::Tensor *a = plain(args[1]), *b = plain(args[2]);
    if (mode < 0 || mode > 2 || !a || !b) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
    const at::ScalarType type = a->scalar_type();
    const int t = type_of(type), index = (int)a->get_device();
    const bool i8 = t == NVFP4_MOE_TYPE_INT8;
    if (b->scalar_type() != type || b->get_device() != index || t < 0 || t == NVFP4_MOE_TYPE_F32 || (i8 && mode != 0) ||
        c10::cuda::current_device() != index)
        Py_RETURN_NONE;
    int64_t a_ld, b_ld, groups = 1, n, k;
    if (!row_stride(*a, &a_ld)) Py_RETURN_NONE;
    const at::Tensor *off = args[3] == Py_None ? nullptr : plain(args[3]);
    if (args[3] != Py_None && !off) Py_RETURN_NONE;
    if (mode == 2) {
        if (!row_stride(*b, &b_ld) || b->size(0) != a->size(0)) Py_RETURN_NONE;
        n = a->size(1);
        k = b->size(1);
        if (off) groups = off->numel() - 1;
    } else {
        const int64_t d = b->dim();
        if (d != 2 && d != 3) Py_RETURN_NONE;
        n = b->size(d - 2);
        k = b->size(d - 1);
        if (d == 3) groups = b->size(0);
        if ((b->stride(d - 1) != 1 && k != 1) || a->size(1) != (mode == 0 ? k : n)) Py_RETURN_NONE;
        b_ld = n > 1 ? b->stride(d - 2) : groups > 1 ? b->stride(0) : padded(k, type);
        if (groups > 1 && b->stride(0) != n * b_ld) Py_RETURN_NONE;
    }
    const int64_t rows = a->size(0);
    if (!fits(rows) || !fits(n) || !fits(k) || groups < 1 || groups > NVFP4_MOE_MAX_GROUPS) Py_RETURN_NONE;
    if (off ? !vector(off, groups + 1, at::kInt, index) : groups != 1) Py_RETURN_NONE;
    const at::Tensor *xs = nullptr, *ws = nullptr;
    if (i8) {
        xs = plain(args[4]);
        ws = plain(args[5]);
        if (!vector(xs, rows, at::kFloat, index) || !vector(ws, groups * n, at::kFloat, index)) Py_RETURN_NONE;
    } else if (args[4] != Py_None || args[5] != Py_None)
        Py_RETURN_NONE;
    at::ScalarType out_type = i8 || mode == 2 ? at::kFloat : type;
    if (args[6] != Py_None) {
        if (!THPDtype_Check(args[6])) Py_RETURN_NONE;
        out_type = reinterpret_cast<THPDtype *>(args[6])->scalar_type;
    }
    const int o = type_of(out_type);
    if (o < 0 || o == NVFP4_MOE_TYPE_INT8) Py_RETURN_NONE;
    at::Tensor out = mode == 2 && off ? rows_of({groups, n, k}, out_type, a->device())
                     : mode == 2      ? rows_of({n, k}, out_type, a->device())
                                      : rows_of({rows, mode == 0 ? n : k}, out_type, a->device());
    nvfp4_moe_gemm_io io{};
    io.groups = (int32_t)groups;
    io.rows = (int32_t)rows;
    io.n = (int32_t)n;
    io.k = (int32_t)k;
    io.type = (nvfp4_moe_type)t;
    io.out_type = (nvfp4_moe_type)o;
    io.offsets = off ? static_cast<const int32_t *>(off->const_data_ptr()) : nullptr;
    const at::Tensor *x = mode == 0 ? a : mode == 2 ? b : nullptr, *dy = mode == 0 ? nullptr : a, *w = mode == 2 ? nullptr : b;
    if (x) {
        io.x = x->const_data_ptr();
        io.x_stride = mode == 0 ? a_ld : b_ld;
    }
    if (dy) {
        io.dy = dy->const_data_ptr();
        io.dy_stride = a_ld;
    }
    if (w) {
        io.w = w->const_data_ptr();
        io.w_stride = b_ld;
    }
    if (i8) {
        io.x_scale = static_cast<const float *>(xs->const_data_ptr());
        io.w_scale = static_cast<const float *>(ws->const_data_ptr());
    }
    io.out = out.mutable_data_ptr();
    io.out_stride = padded(out.size(-1), out_type);
    void *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = g_gemm[mode](&io, stream);
    Py_END_ALLOW_THREADS;
    return rc == NVFP4_MOE_OK ? THPVariable_Wrap(std::move(out)) : PyLong_FromLong(rc);
    END_HANDLE_TH_ERRORS
}

// quantize(x, swiglu) -> (q, scale), a status, or None.
PyObject *quantize(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    HANDLE_TH_ERRORS
    const at::Tensor *x = n_args == 2 ? plain(args[0]) : nullptr;
    if (!x) Py_RETURN_NONE;
    const bool swiglu = args[1] == Py_True;
    const int t = type_of(x->scalar_type()), index = (int)x->get_device();
    int64_t x_ld;
    if (t < 0 || t == NVFP4_MOE_TYPE_INT8 || (!swiglu && args[1] != Py_False) || !row_stride(*x, &x_ld) ||
        c10::cuda::current_device() != index)
        Py_RETURN_NONE;
    const int64_t rows = x->size(0), width = x->size(1), cols = swiglu ? width / 2 : width;
    if (!fits(rows) || !fits(cols) || cols == 0 || (swiglu && width % 2)) Py_RETURN_NONE;
    at::Tensor q = rows_of({rows, cols}, at::kChar, x->device());
    at::Tensor scale = at::empty_strided({rows}, {1}, at::TensorOptions().dtype(at::kFloat).device(x->device()));
    nvfp4_moe_quantize_io io{};
    io.rows = (int32_t)rows;
    io.cols = (int32_t)cols;
    io.in_type = (nvfp4_moe_type)t;
    io.swiglu = swiglu;
    io.in = x->const_data_ptr();
    io.in_stride = x_ld;
    io.q = static_cast<int8_t *>(q.mutable_data_ptr());
    io.q_stride = padded(cols, at::kChar);
    io.scale = static_cast<float *>(scale.mutable_data_ptr());
    void *stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index).stream();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = g_quantize(&io, stream);
    Py_END_ALLOW_THREADS;
    if (rc != NVFP4_MOE_OK) return PyLong_FromLong(rc);
    PyObject *pq = THPVariable_Wrap(std::move(q)), *ps = pq ? THPVariable_Wrap(std::move(scale)) : nullptr;
    PyObject *both = ps ? PyTuple_Pack(2, pq, ps) : nullptr;
    Py_XDECREF(pq);
    Py_XDECREF(ps);
    return both;
    END_HANDLE_TH_ERRORS
}

// setup(grouped_gemm, grouped_gemm_dx, grouped_gemm_dw, quantize_int8): their addresses.
PyObject *setup(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
    void *p[4];
    if (n_args != 4) {
        PyErr_SetString(PyExc_TypeError, "setup: four addresses");
        return nullptr;
    }
    for (int i = 0; i < 4; i++) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    for (int i = 0; i < 3; i++) g_gemm[i] = reinterpret_cast<GemmFn>(p[i]);
    g_quantize = reinterpret_cast<QuantizeFn>(p[3]);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"product", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(product)), METH_FASTCALL, nullptr},
    {"quantize", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize)), METH_FASTCALL, nullptr},
    {"setup", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(setup)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
