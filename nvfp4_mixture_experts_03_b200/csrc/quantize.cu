// Rows to int8 codes and one FP32 scale per row, optionally of h = SiLU(gate) * up.
//
// scale = max|v| / 127 (FP32), q = the whole number nearest to the exact v / scale,
// ties to the even one. v * (1 / scale) in FP32 is within 2^-16 of that quotient
// (|quotient| <= 127 and two roundings of 2^-24 each), so rounding it is right unless
// it stands within that of a half; only then is the quotient's side of the half taken
// from the remainder v - q * scale, which one fused multiply-add gives exactly (it is a
// whole multiple of the smaller ulp and at most about scale / 2, so it fits 24 bits).
#include "products.cuh"

namespace nvmoe {
namespace {

constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: v + kMagic holds rint(v) in its low bits

// The code by the remainder: right for every finite v and scale > 0.
__device__ __noinline__ int exact_code(float v, float scale) {
    // Scales below 2^-100 and their values are brought up by 2^64, exactly: 1 / scale
    // would overflow.
    if (scale < 0x1p-100f) {
        v *= 0x1p64f;
        scale *= 0x1p64f;
    }
    const float t = fminf(fmaxf(v / scale, -128.0f), 128.0f);   // a subnormal scale may be far off max|v| / 127
    if (fabsf(t) >= 127.5f) return t > 0.0f ? 127 : -127;
    float q = rintf(t);
    const float d = fmaf(-q, scale, v), d2 = 2.0f * fabsf(d);
    if (d2 > scale || (d2 == scale && ((int)q & 1))) q += d > 0.0f ? 1.0f : -1.0f;
    return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

template <typename T, bool kSwiglu>
__global__ void __launch_bounds__(256) quantize_kernel(const nvfp4_moe_quantize_io io) {
    __shared__ uint32_t part[8];
    const T *in = static_cast<const T *>(io.in) + (size_t)blockIdx.x * io.in_stride;
    int8_t *q = io.q + (size_t)blockIdx.x * io.q_stride;
    auto value = [&](int c) {
        if (kSwiglu) return silu(to_f32(in[c])) * to_f32(in[io.cols + c]);
        return to_f32(in[c]);
    };
    uint32_t m = 0;
    for (int c = threadIdx.x; c < io.cols; c += 256) m = max(m, __float_as_uint(value(c)) & 0x7fffffffu);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int i = 0; i < 8; i++) m = max(m, part[i]);
    const bool bad = m >= 0x7f800000u;
    const float scale = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float(m) / 127.0f;
    if (threadIdx.x == 0) io.scale[blockIdx.x] = scale;
    for (int c = threadIdx.x; c < io.cols; c += 256)
        q[c] = scale > 0.0f ? (int8_t)exact_code(value(c), scale) : 0;
}

template <typename T>
void launch(const nvfp4_moe_quantize_io &io, cudaStream_t s) {
    if (io.swiglu)
        quantize_kernel<T, true><<<io.rows, 256, 0, s>>>(io);
    else
        quantize_kernel<T, false><<<io.rows, 256, 0, s>>>(io);
}

}  // namespace

cudaError_t launch_quantize(const nvfp4_moe_quantize_io &io, cudaStream_t s) {
    if (io.in_type == NVFP4_MOE_TYPE_BF16)
        launch<__nv_bfloat16>(io, s);
    else if (io.in_type == NVFP4_MOE_TYPE_F16)
        launch<__half>(io, s);
    else
        launch<float>(io, s);
    return cudaGetLastError();
}

}  // namespace nvmoe
