// Products grouped by expert: 64 x 64 output tiles in shared memory, FP32 (or 32-bit
// integer) sums, one kernel for the product and both gradients.
#include "products.cuh"

namespace nvmoe {
namespace {

constexpr int kT = 64, kC = 16;

template <int MODE, typename T, typename O>
__global__ void __launch_bounds__(256) product_tiled_kernel(const Product p) {
    using Acc = typename std::conditional<std::is_same<T, int8_t>::value, int, float>::type;
    __shared__ Acc ls[kC][kT + 1], rs[kC][kT + 1];
    const int e = blockIdx.z;
    const int2 g = group_rows(p, e);
    const int row_lo = MODE == kDw ? 0 : g.x, row_hi = MODE == kDw ? p.n : g.y;
    const int cols = MODE == kFwd ? p.n : p.k;
    const int c_lo = MODE == kDw ? g.x : 0, c_hi = MODE == kDw ? g.y : MODE == kFwd ? p.k : p.n;
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    const T *w = static_cast<const T *>(p.w) + (size_t)e * p.n * p.w_ld;
    O *out = static_cast<O *>(p.out) + (MODE == kDw ? (size_t)e * p.n * p.out_ld : 0);
    const int col0 = blockIdx.x * kT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int row0 = row_lo + blockIdx.y * kT; row0 < row_hi; row0 += gridDim.y * kT) {
        Acc acc[4][4] = {};
        for (int c0 = c_lo; c0 < c_hi; c0 += kC) {
            for (int i = threadIdx.x; i < kT * kC; i += 256) {
                const int cc = MODE == kDw ? i / kT : i % kC, r = MODE == kDw ? i % kT : i / kC;
                const int c = c0 + cc, row = row0 + r;
                Acc v = 0;
                if (c < c_hi && row < row_hi)
                    v = (Acc)to_f32(MODE == kFwd  ? x[(size_t)row * p.x_ld + c]
                                    : MODE == kDx ? dy[(size_t)row * p.dy_ld + c]
                                                  : dy[(size_t)c * p.dy_ld + row]);
                ls[cc][r] = v;
                const int cc2 = MODE == kFwd ? i % kC : i / kT, r2 = MODE == kFwd ? i / kC : i % kT;
                const int c2 = c0 + cc2, col = col0 + r2;
                Acc u = 0;
                if (c2 < c_hi && col < cols)
                    u = (Acc)to_f32(MODE == kFwd  ? w[(size_t)col * p.w_ld + c2]
                                    : MODE == kDx ? w[(size_t)c2 * p.w_ld + col]
                                                  : x[(size_t)c2 * p.x_ld + col]);
                rs[cc2][r2] = u;
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < kC; c++)
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) acc[i][j] += ls[c][ty + 16 * i] * rs[c][tx + 16 * j];
            __syncthreads();
        }
        for (int i = 0; i < 4; i++)
            for (int j = 0; j < 4; j++) {
                const int row = row0 + ty + 16 * i, col = col0 + tx + 16 * j;
                if (row >= row_hi || col >= cols) continue;
                float v = (float)acc[i][j];
                if (std::is_same<T, int8_t>::value) v *= p.x_scale[row] * p.w_scale[(size_t)e * p.n + col];
                O *o = out + (size_t)row * p.out_ld + col;
                if (p.out_add) v += to_f32(*o);
                *o = from_f32<O>(v);
            }
    }
}

template <int MODE, typename T, typename O>
cudaError_t launch(const Product &p, cudaStream_t s) {
    const int rows = MODE == kDw ? p.n : p.rows, cols = MODE == kFwd ? p.n : p.k;
    dim3 grid(cdiv(cols, kT), min(cdiv(rows, kT), 64), p.groups);
    product_tiled_kernel<MODE, T, O><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}
template <int MODE, typename T>
cudaError_t by_out(const Product &p, nvfp4_moe_type out, cudaStream_t s) {
    return out == NVFP4_MOE_TYPE_F32    ? launch<MODE, T, float>(p, s)
           : out == NVFP4_MOE_TYPE_BF16 ? launch<MODE, T, __nv_bfloat16>(p, s)
                                        : launch<MODE, T, __half>(p, s);
}

}  // namespace

cudaError_t launch_product(int mode, const Product &p, nvfp4_moe_type type, nvfp4_moe_type out, cudaStream_t s) {
    if (type == NVFP4_MOE_TYPE_INT8) return by_out<kFwd, int8_t>(p, out, s);
    if (type == NVFP4_MOE_TYPE_BF16)
        return mode == kFwd  ? by_out<kFwd, __nv_bfloat16>(p, out, s)
               : mode == kDx ? by_out<kDx, __nv_bfloat16>(p, out, s)
                             : by_out<kDw, __nv_bfloat16>(p, out, s);
    return mode == kFwd  ? by_out<kFwd, __half>(p, out, s)
           : mode == kDx ? by_out<kDx, __half>(p, out, s)
                         : by_out<kDw, __half>(p, out, s);
}

}  // namespace nvmoe
