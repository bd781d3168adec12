/*
 * misgemm -- the feed-forward block in 16 bits on AMD Instinct MI355X (gfx950), C ABI.
 *
 * Products of BF16 or FP16 matrices with bias, activation and residual in the
 * same kernel; the gated block's two projections, its activation and the
 * product of the two in one kernel; and the backward pass of both, from what
 * the forward pass kept: activations in 16 or 32 bits, or in 8 bits with the
 * scales of misgemm_fp8.h (MI_BLOCK_ROW).
 *
 * The conventions are those of misgemm.h: device pointers owned by the
 * caller, row-major matrices with a leading dimension in elements, work
 * enqueued on `stream` without synchronising, arguments checked in parameter
 * order before any HIP call, thread-safe entry points. Outputs must not
 * overlap inputs or each other, except where an entry point says so. Any
 * pointer alignment that the element type itself allows works, and any leading
 * dimension; 16-byte aligned pointers with rows a multiple of 16 bytes apart
 * are read and written fastest. Types and status codes are those of
 * misgemm_fp8.h.
 */
#ifndef MISGEMM_LINEAR_H
#define MISGEMM_LINEAR_H

#include "misgemm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations f, and their derivatives f'. In FP32. f(-inf) and f(inf) are
 * their limits: 0 and inf (MI_ACT_NONE: -inf and inf); so are f'. NaN stays.
 * f below 2^-119 and f' below 2^-118 may come as 0. */
#define MI_ACT_NONE       0   /* z */
#define MI_ACT_RELU       1   /* max(z, 0); f'(0) = 0 */
#define MI_ACT_SILU       2   /* z / (1 + e^-z) */
#define MI_ACT_GELU       3   /* z / 2 * (1 + erf(z / sqrt 2)) */
#define MI_ACT_GELU_TANH  4   /* z / 2 * (1 + tanh(sqrt(2 / pi) * (z + 0.044715 z^3))) */

/* Status codes beside those of misgemm.h and misgemm_fp8.h. */
#define MISGEMM_BAD_ACT   (-39)   /* none of the activations */

/*
 * mi_linear: C <- f(alpha * op(A) * op(B) + bias) + beta * R
 *
 *   transA, transB    'N' or 'T' (or 'C', as 'T'), as in mi_sgemm: A is M x K or, with 'T',
 *                     K x M; B is K x N or, with 'T', N x K. A layer whose weight
 *                     is kept as outputs x inputs has transB = 'T'.
 *   type              MI_BF16 or MI_F16: A and B.
 *   biastype, bias    `type` or MI_F32; N values, or NULL: none.
 *   act               one of MI_ACT_*.
 *   ctype             `type` or MI_F32: C, R and, unless it has 8 bits, z.
 *   R, ldr            M x N, or NULL: C itself. beta == 0: not read. R may be C
 *                     (same pointer and leading dimension).
 *   ztype, z, ldz     z = alpha * op(A) * op(B) + bias, for the backward pass:
 *                     ctype, or MI_E4M3 or MI_E5M2 with `zscale`, a table
 *                     MI_BLOCK_ROW made as mi_fp8_quantize makes it, from z in
 *                     FP32. z NULL: not wanted.
 * Sums are in FP32; z, f and the sum with beta * R too, and each output is
 * rounded once. K == 0 or alpha == 0: A and B are not read, z = bias.
 * M == 0 or N == 0: nothing is done. The order of the sum is fixed by the
 * shapes, layouts and alignment (of A, B, their leading dimensions), whether
 * z has 8 bits, and, where k is split over workgroups, whether the stream has
 * a workspace (see mi_sgemm): calls alike in these give identical bits. From
 * 2^23 blocks of 64 x 128 outputs on, and where M, N or K passes 2^31 - 257: MISGEMM_TOO_LARGE.
 */
int mi_linear(char transA, char transB, int type, int M, int N, int K, float alpha,
              const void *A, int lda, const void *B, int ldb,
              int biastype, const void *bias, int act, int ctype, float beta, const void *R, int ldr,
              void *C, int ldc, int ztype, void *z, int ldz, float *zscale, int lds, hipStream_t stream);

/*
 * mi_gated: h <- f(g) * u, g = A * G^T + biasG, u = A * U^T + biasU
 *
 *   type              MI_BF16 or MI_F16: A (M x K), G and U (N x K each; they may be
 *                     parts of one matrix).
 *   biastype, biasG, biasU   `type` or MI_F32; N values each, or NULL: none.
 *   htype, h, ldh     `type` or MI_F32, M x N.
 *   ztype             htype, or MI_E4M3 or MI_E5M2: g and u, kept for the backward pass.
 *   g, ldg_, gscale, ldsg   M x N and, in 8 bits, its table as in mi_linear; or g NULL: not wanted.
 *   u, ldu_, uscale, ldsu   likewise; g and u are wanted both or neither (MISGEMM_NULL_OUTPUT).
 * h is formed from g and u in FP32, whatever is kept of them. Sums, their order
 * and sizes as in mi_linear.
 */
int mi_gated(int type, int M, int N, int K, const void *A, int lda, const void *G, int ldg,
             const void *U, int ldu, int biastype, const void *biasG, const void *biasU, int act,
             int htype, void *h, int ldh, int ztype, void *g, int ldg_, float *gscale, int ldsg,
             void *u, int ldu_, float *uscale, int ldsu, hipStream_t stream);

/*
 * mi_act_backward: dz <- dy * f'(z), y <- f(z), dbias <- sum over rows of dz + beta * dbias
 *
 *   type              MI_F32, MI_BF16 or MI_F16: dy, dz and y.
 *   ztype, z, ldz, zscale, lds   `type`, or MI_E4M3 or MI_E5M2 with a table MI_BLOCK_ROW.
 *   dz, lddz          rows x cols. May be dy itself, or z itself where it has `type`.
 *   y, ldy            or NULL: not wanted. May be dy or z as dz may, not dz.
 *   dbias             cols floats, or NULL: not wanted. beta == 0: not read.
 * In FP32, from z as it was kept; dbias is the sum of dz before it is rounded.
 * rows == 0: dbias <- beta * dbias. cols == 0: nothing is done. More than
 * 2^31 - 129 columns: MISGEMM_TOO_LARGE. The sum over
 * many rows is split over workgroups whose partial sums go through the stream's
 * workspace (as in mi_sgemm) and are added in a fixed order; where there is
 * none, one workgroup sums all rows of its columns. Outputs' bits are the same
 * for calls alike in rows, cols and, for dbias, whether the stream has a workspace.
 */
int mi_act_backward(int type, int rows, int cols, const void *dy, int lddy, int act,
                    int ztype, const void *z, int ldz, const float *zscale, int lds,
                    void *dz, int lddz, void *y, int ldy, float beta, float *dbias, hipStream_t stream);

/*
 * mi_gated_backward: gradients of mi_gated's h = f(g) * u
 *
 *   dg <- dh * u * f'(g), du <- dh * f(g), h <- f(g) * u,
 *   dbiasG <- sum over rows of dg + beta * dbiasG, dbiasU likewise of du
 *
 *   type              MI_F32, MI_BF16 or MI_F16: dh, dg, du and h.
 *   ztype             `type`, or MI_E4M3 or MI_E5M2: g and u, with tables MI_BLOCK_ROW in 8 bits.
 *   dg, du            rows x cols each. h, ldh: or NULL: not wanted.
 *                     One of dg, du and h may be dh itself; where g and u have `type`,
 *                     one of them may be g itself, and one u itself.
 *   dbiasG, dbiasU    cols floats each, or NULL: not wanted (each by itself).
 * Sums and their order as in mi_act_backward.
 */
int mi_gated_backward(int type, int rows, int cols, const void *dh, int lddh, int act,
                      int ztype, const void *g, int ldg, const float *gscale, int ldsg,
                      const void *u, int ldu, const float *uscale, int ldsu,
                      void *dg, int lddg, void *du, int lddu, void *h, int ldh,
                      float beta, float *dbiasG, float *dbiasU, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MISGEMM_LINEAR_H */
