// Products of a few rows (single tokens being decoded): the matrices are streamed once
// through mma.sync, straight from global memory to registers.
//
// One CTA computes 16 output columns (16 rows of w[e]) for up to 8 * NT rows of one group,
// its eight warps splitting k. D = w (16 x K) x^T (K x 8): lane (g, q) of a warp loads 16
// consecutive bytes of matrix rows g and g + 8 and of x row g; a lane's four words are its
// operands of two MMAs. Which k a word stands for is the same on both sides, so the
// products are those of the plain order. The warps' sums are added in warp order: the same
// bits on every run.
//
// Bound by latency, then by memory: nothing is staged or laid out, no tensor map, no
// barrier but the one before the join. Many warps with a few loads each in flight do better
// than few with many (1 x 8192 x 8192 BF16: 19.7 us, 6.8 TB/s, with 2 pieces a lane and 4 CTAs an
// SM; 26.0 with 4 pieces and 3 CTAs), as long as the loop that needs no masks has none.
#include <algorithm>

#include "products.cuh"

namespace nvmoe {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kCols = 16;
constexpr int kDeep = 2;   // 16-byte pieces of each row that a lane has in flight

__device__ inline uint4 ld_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Keeps the first n bytes of 16 (what a row holds past its length may be NaN).
__device__ inline void keep(uint4 &v, int n) {
    v.x &= n >= 4 ? ~0u : (1u << (8 * max(n, 0))) - 1;
    v.y &= n >= 8 ? ~0u : (1u << (8 * max(n - 4, 0))) - 1;
    v.z &= n >= 12 ? ~0u : (1u << (8 * max(n - 8, 0))) - 1;
    v.w &= n >= 16 ? ~0u : (1u << (8 * max(n - 12, 0))) - 1;
}

__device__ inline void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                             __half) {
    mma_16816(d, a0, a1, a2, a3, b0, b1);
}
__device__ inline void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                             __nv_bfloat16) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ inline void mma16(int32_t (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                             int8_t) {
    asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename O>
__device__ inline void put(O *o, float v, bool add) {
    *o = from_f32<O>(add ? v + to_f32(*o) : v);
}

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : NT == 2 ? 3 : 2) product_stream_kernel(const __grid_constant__ Product p, const int out_type) {
    constexpr bool kI8 = std::is_same<T, int8_t>::value;
    using Acc = typename std::conditional<kI8, int32_t, float>::type;
    __shared__ Acc part[kWarps][8 * NT][kCols + 1];
    start_after_previous();
    const int col0 = blockIdx.x * kCols;
    // Rows row0 .. row0+nrow-1 of group e: with offsets, block y stands for row y and works
    // if that row opens a batch of 8 * NT rows of its group.
    int e = 0, row0 = blockIdx.y * 8 * NT, end = p.rows;
    if (p.offsets) {
        row0 = blockIdx.y;
        // The group is the one ahead of the first offset past row0: as many are not, if they are in
        // order (the count's upper half: how many are not in order).
        int found = 0;
        for (int i = threadIdx.x; i < p.groups; i += kThreads) {
            const int v = p.offsets[i];
            found += (v <= row0) + (v > p.offsets[i + 1] ? 1 << 16 : 0);
        }
        found = __reduce_add_sync(0xffffffffu, found);
        __shared__ int count[kWarps];
        if ((threadIdx.x & 31) == 0) count[threadIdx.x >> 5] = found;
        __syncthreads();
        found = 0;
#pragma unroll
        for (int w = 0; w < kWarps; w++) found += count[w];
        int lo = 0;
        if (found >> 16) {   // out of order: each clamped to no less than those before it
            found = 0;
            while (found < p.groups && p.offsets[found] <= row0) lo = max(lo, p.offsets[found++]);
        }
        if (found == 0) return;
        e = found - 1;
        lo = max(lo, p.offsets[e]);
        end = min(p.offsets[found], p.rows);
        if (row0 >= end) return;
        if ((row0 - lo) % (8 * NT)) return;
    }
    const int nrow = min(8 * NT, end - row0);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint32_t kb = (uint32_t)p.k * sizeof(T);   // bytes of a row
    const int64_t w_ld = p.w_ld * sizeof(T), x_ld = p.x_ld * sizeof(T);
    // 64 bytes of every row a piece, 64 * kDeep bytes a step; the warps take steps in turn.
    constexpr uint32_t kStepBytes = 64 * kDeep, kRound = kWarps * kStepBytes;
    const uint32_t first = warp * kStepBytes + 16 * q;
    // Rows past the matrix or the batch repeat its last one; their results are dropped.
    const char *w0 = static_cast<const char *>(p.w) + ((int64_t)e * p.n + min(col0 + g, p.n - 1)) * w_ld + first;
    const char *w1 = static_cast<const char *>(p.w) + ((int64_t)e * p.n + min(col0 + g + 8, p.n - 1)) * w_ld + first;
    const char *x[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) x[t] = static_cast<const char *>(p.x) + (int64_t)(row0 + min(8 * t + g, nrow - 1)) * x_ld + first;

    Acc acc[NT][4] = {};
    uint4 a0[kDeep], a1[kDeep], b[NT][kDeep];
    auto products = [&]() {
#pragma unroll
        for (int d = 0; d < kDeep; d++)
#pragma unroll
            for (int t = 0; t < NT; t++) {
                mma16(acc[t], a0[d].x, a1[d].x, a0[d].y, a1[d].y, b[t][d].x, b[t][d].y, T());
                mma16(acc[t], a0[d].z, a1[d].z, a0[d].w, a1[d].w, b[t][d].z, b[t][d].w, T());
            }
    };
    uint32_t k0 = warp * kStepBytes;
    for (; k0 + kStepBytes <= kb; k0 += kRound) {
#pragma unroll
        for (int d = 0; d < kDeep; d++) {
            a0[d] = ld_stream(w0 + 64 * d);
            a1[d] = ld_stream(w1 + 64 * d);
#pragma unroll
            for (int t = 0; t < NT; t++) b[t][d] = *reinterpret_cast<const uint4 *>(x[t] + 64 * d);
        }
        w0 += kRound;
        w1 += kRound;
#pragma unroll
        for (int t = 0; t < NT; t++) x[t] += kRound;
        products();
    }
    if (k0 < kb) {   // one warp's last step: zeros past the rows' ends
        const int left = (int)(kb - k0) - 16 * q;   // bytes from this lane's first
#pragma unroll
        for (int d = 0; d < kDeep; d++) {
            const int n = left - 64 * d;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            a0[d] = n > 0 ? ld_stream(w0 + 64 * d) : zero;
            a1[d] = n > 0 ? ld_stream(w1 + 64 * d) : zero;
#pragma unroll
            for (int t = 0; t < NT; t++) b[t][d] = n > 0 ? *reinterpret_cast<const uint4 *>(x[t] + 64 * d) : zero;
            if (n > 0 && n < 16) {
                keep(a0[d], n);
                keep(a1[d], n);
#pragma unroll
                for (int t = 0; t < NT; t++) keep(b[t][d], n);
            }
        }
        products();
    }
#pragma unroll
    for (int t = 0; t < NT; t++)
#pragma unroll
        for (int i = 0; i < 4; i++) part[warp][8 * t + 2 * q + (i & 1)][g + 8 * (i >> 1)] = acc[t][i];
    __syncthreads();
#pragma unroll
    for (int i = threadIdx.x; i < 8 * NT * kCols; i += kThreads) {
        const int c = i % kCols, r = i / kCols, col = col0 + c;
        if (r >= nrow || col >= p.n) continue;
        Acc sum = part[0][r][c];
#pragma unroll
        for (int w = 1; w < kWarps; w++) sum += part[w][r][c];
        float v;
        if constexpr (kI8)
            v = scaled(sum, p.x_scale[row0 + r], p.w_scale[(int64_t)e * p.n + col]);
        else
            v = sum;
        const int64_t at = (row0 + r) * p.out_ld + col;
        if (out_type == NVFP4_MOE_TYPE_F32)
            put(static_cast<float *>(p.out) + at, v, p.out_add);
        else if (out_type == NVFP4_MOE_TYPE_BF16)
            put(static_cast<__nv_bfloat16 *>(p.out) + at, v, false);
        else
            put(static_cast<__half *>(p.out) + at, v, false);
    }
}

template <typename T>
cudaError_t launch(const Product &p, nvfp4_moe_type out, cudaStream_t s) {
    // Batches of 8 rows where the rows are spread over groups (most have a row or two) or
    // are no more than that; a dense call's rows in one batch up to 32.
    const int nt = p.groups > 1 || p.rows <= 8 ? 1 : p.rows <= 16 ? 2 : 4;
    const dim3 grid(cdiv(p.n, kCols), p.offsets ? p.rows : cdiv(p.rows, 8 * nt));
    return launch_kernel(nt == 1   ? product_stream_kernel<T, 1>
                         : nt == 2 ? product_stream_kernel<T, 2>
                                   : product_stream_kernel<T, 4>,
                         grid, kThreads, s, p, (int)out);
}

}  // namespace

// Streaming reads a group's matrix again for every batch of its rows, and has a CTA for every
// 16 columns of each; the tensor-core tiles have some 6 us of start and end. Measured against
// them (us, streamed / tiles, BF16): dense 8 x 8192 x 8192 20 / 30, 32 x the same 35 / 31, 64 x 1536 x
// 2048 6.5 / 10.6, 64 x 2560 x 2560 10.7 / 12.0, 128 x 2048 x 768 7.4 / 7.5, 201 x the same 11.1 / 7.6, 32 x
// 8192 x 256 5.0 / 6.1, 64 x the same 8.4 / 6.1.
// By group a CTA stands for every row and 16 columns, so their number counts, the more the
// longer the offsets that each looks through; where a row is long, the tiles wait for the matrices
// too. Measured over 12 sizes of matrices in BF16 and int8, 2 to 512 groups, 1 to 192 rows (us,
// streamed / tiles; rows to the left of the bar are streamed): BF16 8 x 1536 x 2048 32: 12.1 / 12.7 | 48:
// 14.1 / 12.7; 512 x 2048 x 768 8: 7.0 / 7.1 | 16: 13.0 / 9.9; 512 x 1536 x 2048 24: 24.3 / 25.5 | 32:
// 29.8 / 34.0; 2 x 256 x 256 128: 4.2 / 4.7 | 192: 5.5 / 4.9; int8 64 x 1536 x 2048 24: 14.6 / 14.3 | 32:
// 17.2 / 15.9; 8 x 2048 x 768 16: 6.0 / 6.5 | 24: 7.2 / 6.9. On average over all of them the rule costs 0.8 %
// more than the better kernel, at worst 39 % (all rows in one of 512 groups); 3100 CTAs whatever
// the row and the groups cost 1.2 and 47 %.
bool product_streams(int mode, const Product &p, int elem_bytes) {
    if (mode != kFwd) return false;
    const int64_t blocks = cdiv(p.n, kCols);
    if (p.offsets) return p.rows * blocks <= (p.groups <= 128 ? 2200 : 1200) + std::min<int64_t>((int64_t)p.k * elem_bytes, 4096) / 3;
    if (p.rows <= 8) return true;
    const int64_t passes = cdiv(p.rows, 32);
    return passes * blocks <= 512 && passes * p.n * p.k * elem_bytes <= 30000000;
}

cudaError_t launch_product_stream(const Product &p, nvfp4_moe_type type, nvfp4_moe_type out, cudaStream_t s) {
    return type == NVFP4_MOE_TYPE_INT8   ? launch<int8_t>(p, out, s)
           : type == NVFP4_MOE_TYPE_BF16 ? launch<__nv_bfloat16>(p, out, s)
                                         : launch<__half>(p, out, s);
}

}  // namespace nvmoe
