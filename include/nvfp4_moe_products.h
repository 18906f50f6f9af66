/*
 * nvfp4_moe_products.h -- the 8-bit and the ragged matrix products that stand
 * beside the routed NVFP4 layer of nvfp4_moe.h.
 *
 *   nvfp4_moe_quantize_int8     rows to int8 codes and one FP32 scale per row: the
 *                               activations that NVFP4_MOE_ACT_INT8 takes, and the
 *                               operands of the int8 product below; optionally of
 *                               h = SiLU(gate) * up, formed on the way
 *   nvfp4_moe_grouped_gemm      out[p] = x[p] W_e^T for the rows p of expert e:
 *                               experts (or a shared, dense expert: one group) whose
 *                               matrices are BF16, F16 or int8 instead of NVFP4
 *   nvfp4_moe_grouped_gemm_dx   dx[p] = dy[p] W_e          (gradient for the rows)
 *   nvfp4_moe_grouped_gemm_dw   dW_e = sum over p of e of dy[p]^T x[p]
 *                                                          (gradient for the matrices)
 *
 * Sources on the pages: the W4A8 path's 8-bit activations and the shared expert's
 * fused SwiGLU quantiser ("Strata NVFP4" README, "How it differs from upstream
 * Strata"); packs whose down projections are 8-bit (same README, the GPTQ section);
 * one launch for a whole expert group after one wait (same README, the prompt-reading
 * bullet). The pages write none of the formulas out; they are stated here.
 *
 * Rows are grouped as nvfp4_moe_forward's dbg_offsets gives them: rows
 * offsets[e] .. offsets[e+1]-1 belong to expert e. The offsets live on the device and
 * are never read back. They must not decrease and must stay within [0, rows]; each is
 * clamped into that range and to no less than those before it, so wrong ones give wrong
 * rows, but no access out of range.
 * Rows before offsets[0] and from offsets[groups] on belong to nobody: they are not
 * written (grouped_gemm, dx) and add nothing (dw), whatever they hold.
 *
 * Conventions are those of nvfp4_moe.h: DEVICE pointers owned by the caller, host
 * checks before anything is enqueued, no synchronisation, no allocation and no
 * workspace, work enqueued on `stream` of the current device (which must be an sm_100
 * device that can reach the pointers). Calls keep nothing from one to the next and may
 * run concurrently, on any streams and threads, as long as their outputs are disjoint;
 * all of them can be captured into graphs. Results do not depend on timing: the same
 * inputs give the same bits on every run. Every kernel is launched as a programmatic
 * dependent of the one before it in the stream and waits for all of it before it touches
 * memory; it lets a programmatic dependent that follows start at once, so such a kernel of
 * the caller's has to wait (griddepcontrol.wait) before it reads what these calls write.
 */
#ifndef NVFP4_MOE_PRODUCTS_H
#define NVFP4_MOE_PRODUCTS_H

#include "nvfp4_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NVFP4_MOE_TYPE_BF16 = 0,
    NVFP4_MOE_TYPE_F16 = 1,
    NVFP4_MOE_TYPE_F32 = 2,
    NVFP4_MOE_TYPE_INT8 = 3
} nvfp4_moe_type;

/* Largest k of an int8 product: (-128)^2 * k stays below 2^31, so that every sum of
 * products is exact in 32 bits. */
#define NVFP4_MOE_INT8_MAX_K 131071
/* Most groups of one product (experts of a layer), and the most rows, n, k or columns of
 * a call (dw: groups * n too). */
#define NVFP4_MOE_MAX_GROUPS 1024
#define NVFP4_MOE_MAX_EXTENT (1 << 30)

/* One quantiser call.
 *   rows, cols   rows >= 0 (0 is a no-op), cols >= 1 codes per row
 *   in_type      BF16, F16 or F32
 *   swiglu       0: the row's values are v = in[row][0..cols)
 *                1: in rows hold gate | up, 2*cols values; v = SiLU(gate) * up in FP32,
 *                to 2^-20 of the value for gates from -87 on (below, SiLU is under
 *                2^-119 and is taken for 0)
 *   in_stride    elements from one row to the next, >= the row's values
 *   q, q_stride  [rows][cols] int8, q_stride >= cols; bytes past cols are not written;
 *                q must not overlap in
 *   scale        [rows] f32
 * scale = max|v| / 127 rounded to FP32; q = the whole number nearest to the exact
 * quotient v / scale (ties to the even one), clamped to +-127. A row whose scale is 0
 * has codes 0. A row that holds a NaN or an infinity (or whose SiLU(gate) * up leaves
 * FP32's range) has scale NaN and codes 0, so that what is computed from it is NaN.
 * Pointers need their type's own alignment only; 16-byte aligned rows are faster. */
typedef struct {
    int32_t rows;
    int32_t cols;
    nvfp4_moe_type in_type;
    int32_t swiglu;
    const void *in;
    int64_t in_stride;
    int8_t *q;
    int64_t q_stride;
    float *scale;
} nvfp4_moe_quantize_io;

NVFP4_MOE_API int nvfp4_moe_quantize_int8(const nvfp4_moe_quantize_io *io, void *stream);

/* One product call; which fields a call reads:
 *                        grouped_gemm      grouped_gemm_dx    grouped_gemm_dw
 *   x  [rows][k]         read              -                  read
 *   dy [rows][n]         -                 read               read
 *   w  [groups][n][k]    read              read               -
 *   out                  [rows][n]         [rows][k]          [groups][n][k]
 * Row strides are in elements and at least the row's length; matrix e of w (and of
 * dw's out) starts n * stride elements after matrix e-1.
 *   groups       1..NVFP4_MOE_MAX_GROUPS
 *   rows         >= 0; with 0 rows grouped_gemm and dx are no-ops and dw writes zeros
 *   n, k         >= 1, any
 *   offsets      [groups+1] i32 on the device, or NULL with groups == 1 (all rows)
 *   type         of x, dy and w: BF16, F16, or (grouped_gemm only) INT8
 *   x_scale      INT8: [rows] f32;  w_scale  INT8: [groups][n] f32; else not read.
 *                out[p][j] = x_scale[p] * w_scale[e][j] * sum_k x[p][k] w[e][j][k],
 *                the sum exact in 32-bit integers; the scales may be of any size (no
 *                product of theirs leaves FP32's range unless the result does)
 *   out_type     BF16, F16 or F32; 16-bit sums are FP32, rounded once to out_type
 *   accumulate   nonzero: out += result, F32 outputs only
 * x, dy and w must be 16-byte aligned and their row strides a multiple of 16 bytes;
 * out needs its type's own alignment only (16-byte aligned rows are faster) and must not
 * overlap what the call reads. What a row holds between its length and its stride is
 * neither used nor written. dw writes zeros (or adds nothing) for an expert without rows. */
typedef struct {
    int32_t groups;
    int32_t rows;
    int32_t n;
    int32_t k;
    nvfp4_moe_type type;
    nvfp4_moe_type out_type;
    int32_t accumulate;
    const int32_t *offsets;
    const void *x;
    int64_t x_stride;
    const float *x_scale;
    const void *dy;
    int64_t dy_stride;
    const void *w;
    int64_t w_stride;
    const float *w_scale;
    void *out;
    int64_t out_stride;
} nvfp4_moe_gemm_io;

NVFP4_MOE_API int nvfp4_moe_grouped_gemm(const nvfp4_moe_gemm_io *io, void *stream);
NVFP4_MOE_API int nvfp4_moe_grouped_gemm_dx(const nvfp4_moe_gemm_io *io, void *stream);
NVFP4_MOE_API int nvfp4_moe_grouped_gemm_dw(const nvfp4_moe_gemm_io *io, void *stream);

/* Synchronises `stream` and returns the first device-side error that a call of this
 * header latched on the current device since the last such read (0 if none), clearing
 * it. The only one there is: NVFP4_MOE_ERR_TIMEOUT, a bounded wait of a product that gave
 * up, whose output is then not complete. (The products need no handle, so the word
 * belongs to the device; the layer's own status is nvfp4_moe_get_status.) */
NVFP4_MOE_API int nvfp4_moe_products_status(void *stream);

#ifdef __cplusplus
}
#endif
#endif /* NVFP4_MOE_PRODUCTS_H */
