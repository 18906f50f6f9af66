// Rows to int8 codes and one FP32 scale per row, optionally of h = SiLU(gate) * up.
//
// scale = max|v| / 127 (FP32), q = the whole number nearest to the exact v / scale, ties to
// the even one. q is rounded from v * (1 / scale), which may fall on the wrong side of a half;
// the remainder d = v - q * scale tells: one fused multiply-add gives it exactly (it is a
// whole multiple of the smaller ulp and at most about scale / 2, so it fits 24 bits), and q
// is right wherever 2 |d| < scale. Only else is it corrected. That is no rare case with
// 16-bit values: every v = max / 2 stands 63.5 steps of a rounded scale from zero.
//
// Bound by memory: every input is read once and waits in registers (16-bit values as they
// are, h as FP32) between the maximum and the rounding. A code takes one multiply-add that
// leaves the rounded number in the low bits of a float, one add that takes it out, one
// multiply-add for d, two codes to an instruction, and the maximum of |d| over eight. A warp
// takes a row where there are rows enough to fill the GPU, else a CTA does.
#include "products.cuh"

namespace nvmoe {
namespace {

constexpr int kThreads = 256;
constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: v + kMagic holds rint(v) in its low bits
constexpr float kTiny = 0x1p-100f;

// The code for any finite v and scale > 0, for scales below kTiny: both are brought up by
// 2^64, exactly (1 / scale would overflow).
__device__ __noinline__ int tiny_code(float v, float scale) {
    v *= 0x1p64f;
    scale *= 0x1p64f;
    const float t = fminf(fmaxf(v / scale, -128.0f), 128.0f);   // a subnormal scale may be far off max|v| / 127
    if (fabsf(t) >= 127.5f) return t > 0.0f ? 127 : -127;
    float q = rintf(t);
    const float d = fmaf(-q, scale, v), d2 = 2.0f * fabsf(d);
    if (d2 > scale || (d2 == scale && ((int)q & 1))) q += d > 0.0f ? 1.0f : -1.0f;
    return (int)fminf(fmaxf(q, -127.0f), 127.0f);
}

__device__ inline float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ inline float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n mov.b64 {%0, %1}, w;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// SiLU(g) * u = g / (1 + e^-g) * u, right to some ten units of 2^-24. e^x as 2^y with y = x log2(e)
// rounded, times e^(x - y ln 2), whose exponent is taken in two parts of ln 2 (Cody and Waite's
// reduction) and is so small that 1 + it will do: without it the rounding of y alone costs |x| units
// (the layer's silu() leaves it out: a row of strongly negative gates only was coded from values
// 2^-18 off; 8191 x 768 BF16 6.9 us with it, 7.2 with this one, 8.3 with expf). Past +-88 the sum is
// 1, or so large that its inverse is 0; g itself still carries NaN and infinities on.
__device__ inline float swiglu(float g, float u) {
    constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147182f, kLn2Rest = (float)(0.693147180559945309 - (double)kLn2);
    const float x = -fminf(fmaxf(g, -88.0f), 88.0f), y = x * kLog2e;
    float e, inv;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    e = fmaf(e, fmaf(-y, kLn2Rest, fmaf(-y, kLn2, x)), e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(1.0f + e));
    return g * inv * u;
}

// Eight values of a row as a thread keeps them: 16-bit ones as read, else FP32.
template <typename T, bool kSwiglu>
struct Chunk {
    static constexpr bool kRaw = sizeof(T) == 2 && !kSwiglu;
    uint32_t w[kRaw ? 4 : 8];
    __device__ float2 pair(int i) const {
        if constexpr (kRaw) {
            const T *h = reinterpret_cast<const T *>(&w[i]);
            return make_float2(to_f32(h[0]), to_f32(h[1]));
        } else
            return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
    // Its largest magnitude, joined to m, as bits: NaN and infinities order above every
    // number (of 16-bit values in both halves of m).
    __device__ uint32_t top(uint32_t m) const {
        if constexpr (kRaw) {
#pragma unroll
            for (int i = 0; i < 4; i++) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++) m = max(m, w[i] & 0x7fffffffu);
        }
        return m;
    }
    // The largest magnitude of a thread's chunks as the bits of an FP32 number.
    __device__ static uint32_t top_bits(uint32_t m) {
        if constexpr (kRaw) {
            m = max(m & 0xffffu, m >> 16);
            const uint16_t h = (uint16_t)m;
            return __float_as_uint(to_f32(*reinterpret_cast<const T *>(&h))) & 0x7fffffffu;
        } else
            return m;
    }
};

// Values c .. c+7 as words (zeros from cols on); kVec: p + c is 16-byte aligned.
template <typename T, bool kVec>
__device__ inline void load8(const T *p, int c, int cols, uint32_t (&w)[sizeof(T) * 2]) {
    if (kVec && c + 8 <= cols) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; i++) {
            const uint4 a = *(reinterpret_cast<const uint4 *>(p + c) + i);
            w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if constexpr (sizeof(T) == 4)
                w[j] = c + j < cols ? __float_as_uint(p[c + j]) : 0u;
            else {
                const uint32_t h = c + j < cols ? *reinterpret_cast<const uint16_t *>(p + c + j) : 0u;
                w[j >> 1] = j & 1 ? w[j >> 1] | h << 16 : h;
            }
        }
    }
}

// Loads a chunk; with 16-bit gate | up their eight words stand where form_chunk leaves h, so
// that all of a thread's loads are under way before the first of them is needed.
template <typename T, bool kSwiglu, bool kVec>
__device__ inline void load_chunk(Chunk<T, kSwiglu> &k, const T *in, int c, int cols) {
    if constexpr (!kSwiglu)
        load8<T, kVec>(in, c, cols, k.w);
    else if constexpr (sizeof(T) == 2) {
        uint32_t g[4], u[4];
        load8<T, kVec>(in, c, cols, g);
        load8<T, kVec>(in + cols, c, cols, u);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            k.w[i] = g[i];
            k.w[4 + i] = u[i];
        }
    } else {
        uint32_t g[8], u[8];
        load8<T, kVec>(in, c, cols, g);
        load8<T, kVec>(in + cols, c, cols, u);
#pragma unroll
        for (int i = 0; i < 8; i++) k.w[i] = __float_as_uint(swiglu(__uint_as_float(g[i]), __uint_as_float(u[i])));
    }
}
template <typename T, bool kSwiglu>
__device__ inline void form_chunk(Chunk<T, kSwiglu> &k) {
    if constexpr (kSwiglu && sizeof(T) == 2) {
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 8; i++) r[i] = k.w[i];
        const T *g = reinterpret_cast<const T *>(r), *u = reinterpret_cast<const T *>(r + 4);
#pragma unroll
        for (int i = 0; i < 8; i++) k.w[i] = __float_as_uint(swiglu(to_f32(g[i]), to_f32(u[i])));
    }
}

template <typename T, bool kSwiglu, bool kVec>
__device__ inline void code_chunk(const Chunk<T, kSwiglu> &k, float scale, float inv, int8_t *q, int c, int cols) {
    uint32_t r[8];
    if (scale >= kTiny) {
        float2 d[4];
        float far = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 v = k.pair(i), m = fma2(v, make_float2(inv, inv), make_float2(kMagic, kMagic));
            const float2 n = add2(make_float2(kMagic, kMagic), make_float2(-m.x, -m.y));   // -q
            d[i] = fma2(n, make_float2(scale, scale), v);
            r[2 * i] = __float_as_uint(m.x);
            r[2 * i + 1] = __float_as_uint(m.y);
            far = fmaxf(far, fmaxf(fabsf(d[i].x), fabsf(d[i].y)));
        }
        if (2.0f * far >= scale) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float e = j & 1 ? d[j >> 1].y : d[j >> 1].x, e2 = 2.0f * fabsf(e);
                if (e2 > scale || (e2 == scale && (r[j] & 1))) r[j] += e > 0.0f ? 1u : ~0u;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 v = k.pair(i);
            r[2 * i] = scale > 0.0f ? (uint32_t)tiny_code(v.x, scale) : 0u;       // a scale of 0 or NaN: codes 0
            r[2 * i + 1] = scale > 0.0f ? (uint32_t)tiny_code(v.y, scale) : 0u;
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

// kPer threads take a row (32 or kThreads). kKeep chunks of it stay in a thread's registers
// (cols <= kPer * 8 * kKeep); 0: the row is read twice.
template <typename T, bool kSwiglu, bool kVec, int kPer, int kKeep>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const nvfp4_moe_quantize_io io) {
    __shared__ uint32_t part[kThreads / 32];
    start_after_previous();
    const int row = kPer == 32 ? blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (kPer == 32 && row >= io.rows) return;
    const int me = threadIdx.x & (kPer - 1);
    const int cols = io.cols;
    const T *in = static_cast<const T *>(io.in) + (size_t)row * io.in_stride;
    int8_t *q = io.q + (size_t)row * io.q_stride;

    Chunk<T, kSwiglu> v[kKeep ? kKeep : 1];
    uint32_t m = 0;
    if (kKeep) {
#pragma unroll
        for (int i = 0; i < kKeep; i++)
            if (8 * (kPer * i + me) < cols) load_chunk<T, kSwiglu, kVec>(v[i], in, 8 * (kPer * i + me), cols);
#pragma unroll
        for (int i = 0; i < kKeep; i++)
            if (8 * (kPer * i + me) < cols) {
                form_chunk(v[i]);
                m = v[i].top(m);
            }
    } else {
        for (int c = 8 * me; c < cols; c += 8 * kPer) {
            load_chunk<T, kSwiglu, kVec>(v[0], in, c, cols);
            form_chunk(v[0]);
            m = v[0].top(m);
        }
    }
    m = __reduce_max_sync(0xffffffffu, Chunk<T, kSwiglu>::top_bits(m));
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
        for (int i = 0; i < kKeep; i++) {
            const int c = 8 * (kPer * i + me);
            if (c < cols) code_chunk<T, kSwiglu, kVec>(v[i], scale, inv, q, c, cols);
        }
    } else {
        for (int c = 8 * me; c < cols; c += 8 * kPer) {
            load_chunk<T, kSwiglu, kVec>(v[0], in, c, cols);
            form_chunk(v[0]);
            code_chunk<T, kSwiglu, kVec>(v[0], scale, inv, q, c, cols);
        }
    }
}

template <typename T, bool kSwiglu, bool kVec, int kPer, int kKeep>
cudaError_t launch_as(const nvfp4_moe_quantize_io &io, cudaStream_t s) {
    const int grid = kPer == 32 ? cdiv(io.rows, kThreads / 32) : io.rows;
    return launch_kernel(quantize_kernel<T, kSwiglu, kVec, kPer, kKeep>, dim3(grid), kThreads, s, io);
}

template <typename T, bool kSwiglu, bool kVec>
cudaError_t launch(const nvfp4_moe_quantize_io &io, cudaStream_t s) {
    // A warp a row where there are rows enough to fill the GPU that way, else a CTA (us, warps /
    // CTAs a row: 1000 x 768 BF16 2.3 / 2.2, 2048 x 768 2.6 / 3.3, 8192 x 768 6.3 / 10.5; 4096 x 2048
    // 8.7 / 8.4, 32768 x 2048 35 / 50, FP32 55 / 60). h of more than 1024 columns takes too many
    // registers of a warp (32768 x 2048 SwiGLU of BF16 125 / 67, now 74).
    const int chunks = cdiv(io.cols, 8);
    if (chunks <= 32 && io.rows >= 8)
        return launch_as<T, kSwiglu, kVec, 32, 1>(io, s);
    else if (chunks <= 32 * 4 && io.rows >= 1536)
        return launch_as<T, kSwiglu, kVec, 32, 4>(io, s);
    else if (!kSwiglu && chunks <= 32 * 8 && io.rows >= 8192)
        return launch_as<T, false, kVec, 32, 8>(io, s);
    else if (chunks <= kThreads)
        return launch_as<T, kSwiglu, kVec, kThreads, 1>(io, s);
    else if (chunks <= kThreads * 4)
        return launch_as<T, kSwiglu, kVec, kThreads, 4>(io, s);
    else if (chunks <= kThreads * 8)
        return launch_as<T, kSwiglu, kVec, kThreads, 8>(io, s);
    else
        return launch_as<T, kSwiglu, kVec, kThreads, 0>(io, s);
}

template <typename T>
cudaError_t launch(const nvfp4_moe_quantize_io &io, cudaStream_t s) {
    auto al = [](const void *p, int a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
    const bool vec = al(io.in, 16) && (io.rows == 1 || io.in_stride * sizeof(T) % 16 == 0) && al(io.q, 8) &&
                     (io.rows == 1 || io.q_stride % 8 == 0) && (!io.swiglu || (size_t)io.cols * sizeof(T) % 16 == 0);
    if (io.swiglu) return vec ? launch<T, true, true>(io, s) : launch<T, true, false>(io, s);
    return vec ? launch<T, false, true>(io, s) : launch<T, false, false>(io, s);
}

}  // namespace

cudaError_t launch_quantize(const nvfp4_moe_quantize_io &io, cudaStream_t s) {
    return io.in_type == NVFP4_MOE_TYPE_BF16  ? launch<__nv_bfloat16>(io, s)
           : io.in_type == NVFP4_MOE_TYPE_F16 ? launch<__half>(io, s)
                                              : launch<float>(io, s);
}

}  // namespace nvmoe
