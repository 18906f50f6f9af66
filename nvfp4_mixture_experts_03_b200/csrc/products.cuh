// Launch parameters shared by the 8-bit and ragged products' host code and kernels.
#pragma once
#include "common.cuh"
#include "nvfp4_moe_products.h"

namespace nvmoe {

// What a product computes (out has contiguous columns):
//   kFwd  out[p][j] = sum_c x[p][c] w[e][j][c]      rows p of group e, columns j < n, c < k
//   kDx   out[p][j] = sum_c dy[p][c] w[e][c][j]     rows p of group e, columns j < k, c < n
//   kDw   out[e][i][j] = sum_p dy[p][i] x[p][j]     rows i < n, columns j < k, p of group e
enum ProductMode : int { kFwd = 0, kDx = 1, kDw = 2 };

struct Product {
    int32_t groups, rows, n, k;
    int32_t out_add;
    const int32_t *offsets;   // null: one group of all rows
    const void *x, *dy, *w;
    int64_t x_ld, dy_ld, w_ld, out_ld;   // row strides in elements
    const float *x_scale, *w_scale;
    void *out;
};

template <typename T>
__device__ inline float to_f32(T v);
template <>
__device__ inline float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ inline float to_f32(__half v) { return __half2float(v); }
template <>
__device__ inline float to_f32(float v) { return v; }
template <>
__device__ inline float to_f32(int8_t v) { return (float)v; }

template <typename T>
__device__ inline T from_f32(float v);
template <>
__device__ inline __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ inline __half from_f32(float v) { return __float2half_rn(v); }
template <>
__device__ inline float from_f32(float v) { return v; }

// An exact int8 sum times its two scales. Their own product may leave FP32's range where the
// result does not (1e-30 * 1e-10 is subnormal, 1e25 * 1e25 infinite, and 0 * inf NaN), so unless
// both are of usual size the smaller one goes first: |sum| is 0 or at least 1, so sum * smaller
// loses nothing to underflow that the scale had not lost, and overflows only where the result
// does. Scales of usual size keep the one multiplication less on the way from the sum.
__device__ inline bool usual_scale(float v) { return v == 0.0f || (fabsf(v) >= 0x1p-40f && fabsf(v) <= 0x1p40f); }
__device__ inline float scaled_usual(int32_t sum, float a, float b) { return (float)sum * (a * b); }
__device__ inline float scaled(int32_t sum, float a, float b) {
    if (usual_scale(a) && usual_scale(b)) return scaled_usual(sum, a, b);
    const bool first = fabsf(a) < fabsf(b);
    return (float)sum * (first ? a : b) * (first ? b : a);
}

// The products follow one another in short chains, and a small one's launch and start take
// as long as its work: each is a programmatic dependent of the kernel before it in the
// stream, lets its own dependents launch at once, and waits for that kernel, all of it,
// before it touches global memory. Every CTA has to wait, even one without work: the next
// kernel relies on this one's end for the ends of all before it.
__device__ inline void start_after_previous() {
    grid_dep_launch();
    grid_dep_wait();
}
inline void set_programmatic(cudaLaunchAttribute *attr) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
}

// A launch that reports its own error, and none that was pending before it.
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    set_programmatic(&attr);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

cudaError_t launch_quantize(const nvfp4_moe_quantize_io &io, cudaStream_t s);
cudaError_t launch_product_mma(int mode, const Product &p, nvfp4_moe_type type, nvfp4_moe_type out_type,
                               cudaStream_t s);
bool product_streams(int mode, const Product &p, int elem_bytes);   // few enough rows to be streamed
cudaError_t launch_product_stream(const Product &p, nvfp4_moe_type type, nvfp4_moe_type out_type, cudaStream_t s);
void test_product_stall(int n);       // test hook (nvfp4_moe_test.h)
int product_status(cudaStream_t s);   // the first wait that gave up on the current device, cleared

}  // namespace nvmoe
