// Host side of include/nvfp4_moe_products.h: argument checks (all of them before
// anything is enqueued) and dispatch to the kernels.
#include "products.cuh"

using namespace nvmoe;

namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool is16(nvfp4_moe_type t) { return t == NVFP4_MOE_TYPE_BF16 || t == NVFP4_MOE_TYPE_F16; }
inline bool floating(nvfp4_moe_type t) { return is16(t) || t == NVFP4_MOE_TYPE_F32; }
inline int size_of(nvfp4_moe_type t) { return t == NVFP4_MOE_TYPE_F32 ? 4 : t == NVFP4_MOE_TYPE_INT8 ? 1 : 2; }

int check_device() {
    int dev = 0, major = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess || major != 10)
        return NVFP4_MOE_ERR_NO_DEVICE;
    return NVFP4_MOE_OK;
}

// Tensor maps hold byte strides below 2^40.
constexpr int64_t kMaxStride = int64_t(1) << 40;

// One matrix operand: present, 16-byte rows, strides that a tensor map can hold.
int check_operand(const void *p, int64_t ld, int32_t cols, int es, int64_t matrix_rows) {
    if (!p || ld < cols) return NVFP4_MOE_ERR_INVALID_ARG;
    if (ld >= kMaxStride / es || (matrix_rows > 0 && ld * es >= kMaxStride / matrix_rows))
        return NVFP4_MOE_ERR_UNSUPPORTED_DIMS;
    if (!aligned(p, 16) || (ld * es) % 16) return NVFP4_MOE_ERR_MISALIGNED;
    return NVFP4_MOE_OK;
}

int product(int mode, const nvfp4_moe_gemm_io *io, void *stream) {
    if (!io) return NVFP4_MOE_ERR_INVALID_ARG;
    if (io->groups < 1 || io->rows < 0 || io->n < 1 || io->k < 1) return NVFP4_MOE_ERR_INVALID_ARG;
    // tensor-map coordinates are 32-bit, and a tile may start past the last row or column
    if (io->groups > NVFP4_MOE_MAX_GROUPS || io->rows > NVFP4_MOE_MAX_EXTENT || io->n > NVFP4_MOE_MAX_EXTENT ||
        io->k > NVFP4_MOE_MAX_EXTENT || (mode == kDw && (int64_t)io->groups * io->n > NVFP4_MOE_MAX_EXTENT))
        return NVFP4_MOE_ERR_UNSUPPORTED_DIMS;
    const bool i8 = io->type == NVFP4_MOE_TYPE_INT8;
    if (!(is16(io->type) || (i8 && mode == kFwd)) || !floating(io->out_type)) return NVFP4_MOE_ERR_INVALID_ARG;
    if (io->accumulate && io->out_type != NVFP4_MOE_TYPE_F32) return NVFP4_MOE_ERR_INVALID_ARG;
    if (i8 && io->k > NVFP4_MOE_INT8_MAX_K) return NVFP4_MOE_ERR_UNSUPPORTED_DIMS;
    if (!io->offsets && io->groups != 1) return NVFP4_MOE_ERR_INVALID_ARG;
    if (io->rows == 0 && mode != kDw) return NVFP4_MOE_OK;
    const int es = size_of(io->type);
    // With no rows dw reads neither operand.
    if (mode != kDx && io->rows > 0)
        if (const int rc = check_operand(io->x, io->x_stride, io->k, es, 0)) return rc;
    if (mode != kFwd && io->rows > 0)
        if (const int rc = check_operand(io->dy, io->dy_stride, io->n, es, 0)) return rc;
    if (mode != kDw)
        if (const int rc = check_operand(io->w, io->w_stride, io->k, es, io->n)) return rc;
    if (i8 && (!io->x_scale || !io->w_scale)) return NVFP4_MOE_ERR_INVALID_ARG;
    const int32_t out_cols = mode == kFwd ? io->n : io->k;
    if (!io->out || io->out_stride < out_cols) return NVFP4_MOE_ERR_INVALID_ARG;
    if ((mode != kDx && io->out == io->x) || (mode != kFwd && io->out == io->dy) || (mode != kDw && io->out == io->w))
        return NVFP4_MOE_ERR_INVALID_ARG;
    if (!aligned(io->out, size_of(io->out_type)) || !aligned(io->offsets, 4) ||
        (i8 && (!aligned(io->x_scale, 4) || !aligned(io->w_scale, 4))))
        return NVFP4_MOE_ERR_MISALIGNED;
    if (const int rc = check_device()) return rc;
    Product p{};
    p.groups = io->groups;
    p.rows = io->rows;
    p.n = io->n;
    p.k = io->k;
    p.out_add = io->accumulate != 0;
    p.offsets = io->offsets;
    p.x = io->x;
    p.dy = io->dy;
    p.w = io->w;
    p.x_ld = io->x_stride;
    p.dy_ld = io->dy_stride;
    p.w_ld = io->w_stride;
    p.out_ld = io->out_stride;
    p.x_scale = io->x_scale;
    p.w_scale = io->w_scale;
    p.out = io->out;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = product_streams(mode, p, es) ? launch_product_stream(p, io->type, io->out_type, s)
                                                   : launch_product_mma(mode, p, io->type, io->out_type, s);
    return e == cudaSuccess ? NVFP4_MOE_OK : NVFP4_MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

int nvfp4_moe_quantize_int8(const nvfp4_moe_quantize_io *io, void *stream) {
    if (!io || io->rows < 0 || io->cols < 1) return NVFP4_MOE_ERR_INVALID_ARG;
    if (!floating(io->in_type) || (io->swiglu != 0 && io->swiglu != 1)) return NVFP4_MOE_ERR_INVALID_ARG;
    if (io->cols > NVFP4_MOE_MAX_EXTENT) return NVFP4_MOE_ERR_UNSUPPORTED_DIMS;
    if (io->rows == 0) return NVFP4_MOE_OK;
    if (!io->in || !io->q || !io->scale) return NVFP4_MOE_ERR_INVALID_ARG;
    if (io->in_stride < (int64_t)io->cols * (1 + io->swiglu) || io->q_stride < io->cols)
        return NVFP4_MOE_ERR_INVALID_ARG;
    if (io->in == io->q) return NVFP4_MOE_ERR_INVALID_ARG;
    if (!aligned(io->in, size_of(io->in_type)) || !aligned(io->scale, 4)) return NVFP4_MOE_ERR_MISALIGNED;
    if (const int rc = check_device()) return rc;
    return launch_quantize(*io, static_cast<cudaStream_t>(stream)) == cudaSuccess ? NVFP4_MOE_OK
                                                                                  : NVFP4_MOE_ERR_CUDA;
}

int nvfp4_moe_grouped_gemm(const nvfp4_moe_gemm_io *io, void *stream) { return product(kFwd, io, stream); }
int nvfp4_moe_grouped_gemm_dx(const nvfp4_moe_gemm_io *io, void *stream) { return product(kDx, io, stream); }
int nvfp4_moe_grouped_gemm_dw(const nvfp4_moe_gemm_io *io, void *stream) { return product(kDw, io, stream); }

void nvfp4_moe_test_products_stall(int32_t n) { test_product_stall(n); }

int nvfp4_moe_products_status(void *stream) {
    if (const int rc = check_device()) return rc;
    return product_status(static_cast<cudaStream_t>(stream));
}

}  // extern "C"
