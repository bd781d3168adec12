/*
 * misgemm -- the 8-bit linear layer on AMD Instinct MI355X (gfx950), C ABI.
 *
 * Products of matrices in 8-bit floating point with a scale for each block of
 * 128, and the operators that make and use their operands: quantisation both
 * ways round, and the root-mean-square norm with the residual's addition,
 * forward (with an output in 8 bits) and backward.
 *
 * The conventions are those of misgemm.h: device pointers owned by the
 * caller, row-major matrices with a leading dimension in elements, work
 * enqueued on `stream` without synchronising, arguments checked in parameter
 * order before any HIP call, thread-safe entry points. Outputs must not
 * overlap inputs, except where an entry point says so. Any pointer alignment
 * that the element type itself allows works, and any leading dimension;
 * 16-byte aligned pointers with rows a multiple of 16 bytes apart are read
 * and written fastest.
 */
#ifndef MISGEMM_FP8_H
#define MISGEMM_FP8_H

#include "misgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. E4M3 has 4 exponent and 3 fraction bits, no infinity and a
 * largest value of 448; E5M2 has 5 and 2, infinities and a largest finite
 * value of 57344 (the OCP 8-bit formats). */
#define MI_F32   0
#define MI_BF16  1
#define MI_F16   2
#define MI_E4M3  3
#define MI_E5M2  4

/* Scale tables of an 8-bit matrix X of R rows and C columns, whose values
 * stand for X(i,j) * scale:
 *   MI_BLOCK_ROW   one scale for each row and 128 columns:
 *                  scale[(j/128)*lds + i], ceil(C/128) rows of length R, lds >= R.
 *   MI_BLOCK_TILE  one scale for each 128 x 128 block:
 *                  scale[(i/128)*lds + j/128], ceil(R/128) rows of length ceil(C/128). */
#define MI_BLOCK_ROW   0
#define MI_BLOCK_TILE  1

/* Status codes beside those of misgemm.h. */
#define MISGEMM_BAD_TYPE      (-30)   /* an element type that the argument does not take */
#define MISGEMM_BAD_BLOCK     (-31)   /* neither MI_BLOCK_ROW nor MI_BLOCK_TILE */
#define MISGEMM_BAD_ROWS      (-32)   /* rows < 0 */
#define MISGEMM_BAD_COLS      (-33)   /* cols < 0 */
#define MISGEMM_NULL_INPUT    (-34)   /* an input that would be read is null */
#define MISGEMM_NULL_OUTPUT   (-35)   /* an output that must be given is null */
#define MISGEMM_NULL_SCALE    (-36)   /* a scale table is null */
#define MISGEMM_BAD_LD        (-37)   /* a leading dimension smaller than its row */
#define MISGEMM_BAD_LDS       (-38)   /* a scale table's leading dimension smaller than its row */

/*
 * mi_fp8_quantize: x in 8 bits with scales, and/or x^T in 8 bits with its own.
 *
 * For each block b of `block`'s kind, with T the largest finite value of
 * `ftype` (MI_E4M3 or MI_E5M2):
 *   a     = max(max |x| over b, 2^-100)      (NaN left out of the maximum)
 *   scale = a / T
 *   q     = x * (T / a), rounded to nearest, ties to even
 * in FP32. A block of zeros has q = 0. NaN stays NaN at its place. A block
 * that holds an infinity has an infinite scale and q = NaN at the infinity.
 *
 *   xtype, x, ldx        rows x cols matrix of MI_F32, MI_BF16 or MI_F16.
 *   q, ldq, scale, lds   rows x cols and its table, or q NULL: not wanted.
 *   qt, ldqt, scale_t, lds_t   x^T, cols x rows, quantised as such: its row
 *                        blocks are 128 rows of x long. Or qt NULL.
 * One pass over x makes both. One of q and qt must be given
 * (MISGEMM_NULL_OUTPUT). rows == 0 or cols == 0: nothing is done. More than
 * 65,535 * 128 rows, or 2^31 - 128 columns: MISGEMM_TOO_LARGE.
 */
int mi_fp8_quantize(int xtype, int rows, int cols, const void *x, int ldx, int ftype, int block,
                    void *q, int ldq, float *scale, int lds,
                    void *qt, int ldqt, float *scale_t, int lds_t, hipStream_t stream);

/*
 * mi_fp8_gemm: C <- alpha * A * B^T + beta * C with 8-bit operands.
 *
 *   C(i,j) = alpha * sum_b sA(i,b) * sB(j,b) * (sum_{k in b} A(i,k)*B(j,k)) + beta * C(i,j)
 *
 * over blocks b of 128 values of k (the last one may be shorter).
 *   atype, A, lda, scaleA, ldsa   M x K in MI_E4M3 or MI_E5M2, table MI_BLOCK_ROW.
 *   btype, B, ldb, scaleB, ldsb   N x K likewise, table of kind `block`.
 *   ctype, C, ldc                 M x N in MI_F32, MI_BF16 or MI_F16.
 * Blocks are scaled and added in FP32, and the result is rounded to C's type
 * once. Within a block the matrix cores sum in FP32 where C is MI_F32. Where
 * C has 16 bits they take the 8-bit products as they are, at twice the rate,
 * and cut off what is below 2^-13 of the largest of each eight neighbouring
 * ones. On normal values that puts C off by 0.8e-5 to 1.4e-5 of its typical
 * size, and by up to 4e-5 where columns differ in size, far below its
 * rounding. It is not bounded by C's rounding: each eight products may lose
 * 7 * 2^-13 (8.5e-4) of the largest of them, which counts where small values
 * stand beside a few large ones or large products cancel. A caller that needs
 * such sums takes C in MI_F32, and rounds it.
 * sA(i,b) * sB(j,b) is formed first, in FP32, and so has to lie between 2^-126
 * and 2^128. Below that what a block adds loses bits (it is less than 2^-87
 * then, since a block's sum is less than 2^39), beyond it C is infinite or
 * NaN. Scales that mi_fp8_quantize makes have such products where the product
 * of the two blocks' maxima is above 2^-126 * T * T: 2.5e-33 for two E4M3
 * operands, 4e-29 for two in E5M2. Smaller operands are scaled up before they
 * are quantised.
 * The order of the sum is fixed by M, N, K, C's width, `block`, whether A and B
 * are 16-byte aligned with rows a multiple of 16 bytes apart, leading
 * dimensions from 2^24 on, and, where k is split, whether the stream has a
 * workspace: calls alike in these give identical bits.
 * beta == 0: C is not read. alpha == 0 or K == 0: A, B and their tables are
 * not read. M == 0 or N == 0: nothing is done. C must not overlap A or B.
 * From 2^23 blocks of 128 x 128 outputs on, and where M, N or K passes
 * 2^31 - 257: MISGEMM_TOO_LARGE.
 *
 * A call that splits k over workgroups uses the stream's workspace as
 * mi_sgemm does (see there for allocation, graph capture and release); where
 * there is none it runs unsplit.
 */
int mi_fp8_gemm(int atype, int btype, int block, int ctype, int M, int N, int K, float alpha,
                const void *A, int lda, const float *scaleA, int ldsa,
                const void *B, int ldb, const float *scaleB, int ldsb,
                float beta, void *C, int ldc, hipStream_t stream);

/*
 * mi_rmsnorm: the root-mean-square norm of each row, with a residual added first.
 *
 *   h = x + residual          rounded to `type` (h = x without a residual)
 *   rstd = 1 / sqrt(mean of h^2 over the row + eps)   in FP32: 0, and so y = 0,
 *          where the sum of h^2 passes 2^128 (from |h| = 1.8e19 on)
 *   y = h * rstd * weight     in FP32
 *   q, scale = y in 8 bits, as mi_fp8_quantize with MI_BLOCK_ROW makes it
 *              from y in FP32
 *
 *   type              MI_F32, MI_BF16 or MI_F16: x, residual, h and y.
 *   wtype, weight     `type` or MI_F32; cols values.
 *   residual, ldr     or NULL: none.
 *   h, ldh            or NULL: not wanted. May be x or residual itself (same
 *                     pointer and leading dimension).
 *   y, ldy            y rounded to `type`, or NULL.
 *   ftype, q, ldq, scale, lds   or q NULL.
 *   rstd              `rows` floats for the backward pass, or NULL.
 * One of y and q must be given (MISGEMM_NULL_OUTPUT). rows == 0 or
 * cols == 0: nothing is done.
 */
int mi_rmsnorm(int type, int wtype, int rows, int cols, const void *x, int ldx,
               const void *residual, int ldr, const void *weight, float eps,
               void *h, int ldh, void *y, int ldy,
               int ftype, void *q, int ldq, float *scale, int lds, float *rstd, hipStream_t stream);

/*
 * mi_rmsnorm_backward: gradients of mi_rmsnorm's y = h * rstd * weight.
 *
 *   g = dy * weight, u = h * rstd
 *   dx = rstd * (g - u * mean(g * u)) + dh     (of h, and so of x and of the residual alike)
 *   dweight = sum over rows of dy * u + beta * dweight
 *
 *   type               dy, h, dh and dx; FP32 sums, dx rounded to `type` once.
 *   h, rstd            as mi_rmsnorm left them.
 *   dh, lddh           the gradient that reaches h past the norm, or NULL.
 *                      dx may be dh or dy itself.
 *   dweight            cols floats, or NULL: not wanted. beta == 0: not read.
 * rows == 0: dweight <- beta * dweight. cols == 0: nothing is done. The sum
 * over many rows is split over workgroups whose partial sums go through the
 * stream's workspace (as in mi_sgemm) and are added in a fixed order; for few
 * rows, and where there is no workspace, one workgroup sums all rows of its
 * columns, in the same launch. So dweight's bits are the same for calls alike
 * in rows, cols and whether the stream has a workspace; dx's for the same cols.
 */
int mi_rmsnorm_backward(int type, int wtype, int rows, int cols, const void *dy, int lddy,
                        const void *h, int ldh, const void *weight, const float *rstd,
                        const void *dh, int lddh, void *dx, int lddx,
                        float beta, float *dweight, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MISGEMM_FP8_H */
