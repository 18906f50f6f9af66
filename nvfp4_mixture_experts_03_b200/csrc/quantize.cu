// Rows to int8 codes and one FP32 scale per row, optionally of h = SiLU(gate) * up.
//
// scale = max|v| / 127 (FP32), q = the whole number nearest to the exact v / scale,
// ties to the even one. v * (1 / scale) in FP32 is within 2^-16 of that quotient
// (|quotient| <= 127 and two roundings of 2^-24 each), so rounding it is right unless
// it stands within that of a half; only then is the quotient's side of the half taken
// from the remainder v - q * scale, which one fused multiply-add gives exactly (it is a
// whole multiple of the smaller ulp and at most about scale / 2, so it fits 24 bits).
//
// Bound by memory: every input value is read once and kept in registers, as FP32,
// between the maximum and the rounding; a code costs one multiply, one add that leaves
// the rounded number in the low bits, the distance to it, and its share of a byte
// permute. A warp takes a row where there are rows enough to fill the GPU and the row
// fits its registers, else the whole CTA does.
#include "products.cuh"

namespace nvmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunks = 8;              // chunks of 8 values that a thread keeps
constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: v + kMagic holds rint(v) in its low bits
constexpr float kNearHalf = 0.5f - 0x1p-15f;
constexpr float kTiny = 0x1p-100f;

// The code by the remainder: right for every finite v and scale > 0.
__device__ __noinline__ int exact_code(float v, float scale) {
    // Scales below 2^-100 and their values are brought up by 2^64, exactly: 1 / scale
    // would overflow.
    if (scale < kTiny) {
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

// Values c .. c+7 of a row as FP32 (zeros from cols on); kVec: p + c is 16-byte aligned.
template <typename T, bool kVec>
__device__ inline void load8(const T *p, int c, int cols, float (&v)[8]) {
    if (kVec && c + 8 <= cols) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = *reinterpret_cast<const float4 *>(p + c), b = *reinterpret_cast<const float4 *>(p + c + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            const uint4 a = *reinterpret_cast<const uint4 *>(p + c);
            const T *h = reinterpret_cast<const T *>(&a);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] = to_f32(h[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = c + j < cols ? to_f32(p[c + j]) : 0.0f;
    }
}

template <typename T, bool kSwiglu, bool kVec>
__device__ inline void value8(const T *in, int c, int cols, float (&v)[8]) {
    load8<T, kVec>(in, c, cols, v);
    if (kSwiglu) {
        float u[8];
        load8<T, kVec>(in + cols, c, cols, u);
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = silu(v[j]) * u[j];
    }
}

template <bool kVec>
__device__ inline void code8(const float (&v)[8], float scale, float inv, int8_t *q, int c, int cols) {
    uint32_t r[8];
    float far = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float t = v[j] * inv, m = t + kMagic;
        r[j] = __float_as_uint(m);
        far = fmaxf(far, fabsf(t - (m - kMagic)));
    }
    if (!(scale >= kTiny) || far > kNearHalf) {
#pragma unroll 1
        for (int j = 0; j < 8; j++) {
            float vj = v[0];
#pragma unroll
            for (int i = 1; i < 8; i++) vj = i == j ? v[i] : vj;
            const int code = scale > 0.0f ? exact_code(vj, scale) : 0;
#pragma unroll
            for (int i = 0; i < 8; i++) r[i] = i == j ? (uint32_t)code : r[i];
        }
    }
    if (kVec && c + 8 <= cols) {
        uint2 o;
        o.x = __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
        o.y = __byte_perm(__byte_perm(r[4], r[5], 0x0040), __byte_perm(r[6], r[7], 0x0040), 0x5410);
        *reinterpret_cast<uint2 *>(q + c) = o;
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (c + j < cols) q[c + j] = (int8_t)r[j];
    }
}

// kPer threads take a row (32 or kThreads). kKeep: its values stay in registers (cols
// <= kPer * 8 * kChunks), else they are read twice.
template <typename T, bool kSwiglu, bool kVec, int kPer, bool kKeep>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const nvfp4_moe_quantize_io io) {
    __shared__ uint32_t part[kThreads / 32];
    const int row = kPer == 32 ? blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (kPer == 32 && row >= io.rows) return;
    const int me = threadIdx.x & (kPer - 1);
    const int cols = io.cols;
    const T *in = static_cast<const T *>(io.in) + (size_t)row * io.in_stride;
    int8_t *q = io.q + (size_t)row * io.q_stride;

    float v[kKeep ? kChunks : 1][8];
    uint32_t m = 0;   // max |v| as bits: NaN and infinities order above every number
    if (kKeep) {
#pragma unroll
        for (int i = 0; i < kChunks; i++)
            if (8 * kPer * i < cols) value8<T, kSwiglu, kVec>(in, 8 * (kPer * i + me), cols, v[i]);
#pragma unroll
        for (int i = 0; i < kChunks; i++)
            if (8 * kPer * i < cols)
#pragma unroll
                for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(v[i][j]) & 0x7fffffffu);
    } else {
        for (int c = 8 * me; c < cols; c += 8 * kPer) {
            value8<T, kSwiglu, kVec>(in, c, cols, v[0]);
#pragma unroll
            for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(v[0][j]) & 0x7fffffffu);
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (kPer != 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 32; i++) m = max(m, part[i]);
    }
    const float scale = m >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(m) / 127.0f;
    const float inv = 1.0f / scale;
    if (me == 0) io.scale[row] = scale;
    if (kKeep) {
#pragma unroll
        for (int i = 0; i < kChunks; i++) {
            const int c = 8 * (kPer * i + me);
            if (c < cols) code8<kVec>(v[i], scale, inv, q, c, cols);
        }
    } else {
        for (int c = 8 * me; c < cols; c += 8 * kPer) {
            value8<T, kSwiglu, kVec>(in, c, cols, v[0]);
            code8<kVec>(v[0], scale, inv, q, c, cols);
        }
    }
}

template <typename T, bool kSwiglu, bool kVec>
void launch(const nvfp4_moe_quantize_io &io, cudaStream_t s) {
    // A warp a row from four rows per SM up; fewer rows are done sooner by whole CTAs.
    if (io.cols <= 32 * 8 * kChunks && io.rows >= 592)
        quantize_kernel<T, kSwiglu, kVec, 32, true><<<cdiv(io.rows, kThreads / 32), kThreads, 0, s>>>(io);
    else if (io.cols <= kThreads * 8 * kChunks)
        quantize_kernel<T, kSwiglu, kVec, kThreads, true><<<io.rows, kThreads, 0, s>>>(io);
    else
        quantize_kernel<T, kSwiglu, kVec, kThreads, false><<<io.rows, kThreads, 0, s>>>(io);
}

template <typename T>
void launch(const nvfp4_moe_quantize_io &io, cudaStream_t s) {
    auto al = [](const void *p, int a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
    const bool vec = al(io.in, 16) && (io.rows == 1 || io.in_stride * sizeof(T) % 16 == 0) && al(io.q, 8) &&
                     (io.rows == 1 || io.q_stride % 8 == 0) && (!io.swiglu || (size_t)io.cols * sizeof(T) % 16 == 0);
    if (io.swiglu)
        vec ? launch<T, true, true>(io, s) : launch<T, true, false>(io, s);
    else
        vec ? launch<T, false, true>(io, s) : launch<T, false, false>(io, s);
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
