// mi_linear and mi_gated: products of BF16 or FP16 matrices with bias,
// activation and residual, and the gated block's two products in one kernel.
//
//   linear   z = alpha op(A) op(B) + bias, C = f(z) + beta R
//   gated    g = A G^T + biasG, u = A U^T + biasU, h = f(g) u
//
// The sums are formed by v_mfma_f32_16x16x32 in FP32, and stay in registers
// until the outputs leave: bias, activation, the product of the two
// projections, the residual and the 8-bit form of what is kept cost no pass
// over memory of their own. The product's first operand is B and its second A:
// a lane then holds outputs of one row of A at neighbouring columns. Which
// values of k a lane group feeds does not matter as long as it is the same for
// both operands.

#include "linear.h"

namespace {

using namespace misgemm_linear;

bool letter(char c, bool &t) {
    t = c == 'T' || c == 't' || c == 'C' || c == 'c';
    return t || c == 'N' || c == 'n';
}
bool too_large(int M, int N, int K) {
    // Tile counts and the launch's threads are 32-bit; sizes are rounded up to tiles.
    return ((M + 63LL) / 64) * ((N + 127LL) / 128) >= 1LL << 23 || N > 0x7fffffff - 256 || M > 0x7fffffff - 256 ||
           K > 0x7fffffff - 256;
}
// Whether 16-byte chunks of a matrix can go to LDS as they are: k runs fastest
// (its last, short block goes another way), or `across` values do.
bool whole(const void *p, long long ld, bool kmajor, int across) {
    return aligned(p, 16) && ld % 8 == 0 && ld < 1 << 23 && (kmajor || across % 8 == 0);
}

int launch(int type, bool gated, bool ta, bool tb, LinArgs &g, hipStream_t stream) {
    return type == MI_BF16 ? launch_tiles_bf16(gated, ta, tb, 0, g, stream)
                           : launch_tiles_f16(gated, ta, tb, 0, g, stream);
}

}  // namespace

extern "C" int mi_linear(char transA, char transB, int type, int M, int N, int K, float alpha, const void *A, int lda,
                         const void *B, int ldb, int biastype, const void *bias, int act, int ctype, float beta,
                         const void *R, int ldr, void *C, int ldc, int ztype, void *z, int ldz, float *zscale, int lds,
                         hipStream_t stream) {
    bool ta, tb;
    if (!letter(transA, ta)) return MISGEMM_BAD_TRANSA;
    if (!letter(transB, tb)) return MISGEMM_BAD_TRANSB;
    if (!is_half(type)) return MISGEMM_BAD_TYPE;
    if (M < 0) return MISGEMM_BAD_M;
    if (N < 0) return MISGEMM_BAD_N;
    if (K < 0) return MISGEMM_BAD_K;
    const bool some = M > 0 && N > 0, reads = some && K > 0 && alpha != 0.0f;
    if (reads && A == nullptr) return MISGEMM_NULL_A;
    if (lda < (ta ? M : K) || lda < 1) return MISGEMM_BAD_LDA;
    if (reads && B == nullptr) return MISGEMM_NULL_B;
    if (ldb < (tb ? K : N) || ldb < 1) return MISGEMM_BAD_LDB;
    if (bias != nullptr && biastype != type && biastype != MI_F32) return MISGEMM_BAD_TYPE;
    if (act < MI_ACT_NONE || act > MI_ACT_GELU_TANH) return MISGEMM_BAD_ACT;
    if (ctype != type && ctype != MI_F32) return MISGEMM_BAD_TYPE;
    if (beta != 0.0f && R != nullptr && ldr < N) return MISGEMM_BAD_LD;
    if (some && C == nullptr) return MISGEMM_NULL_C;
    if (ldc < N || ldc < 1) return MISGEMM_BAD_LDC;
    if (z != nullptr) {
        if (ztype != ctype && !is_f8(ztype)) return MISGEMM_BAD_TYPE;
        if (ldz < N) return MISGEMM_BAD_LD;
        if (is_f8(ztype)) {
            if (some && zscale == nullptr) return MISGEMM_NULL_SCALE;
            if (lds < M) return MISGEMM_BAD_LDS;
        }
    }
    if (too_large(M, N, K)) return MISGEMM_TOO_LARGE;
    if (!some) return MISGEMM_SUCCESS;

    LinArgs g = {};
    g.A = A;
    g.B = B;
    g.bias = bias;
    g.bias32 = biastype == MI_F32;
    g.R = R != nullptr ? R : C;
    g.ldr = R != nullptr ? ldr : ldc;
    g.C = C;
    g.c32 = ctype == MI_F32;
    g.z = z;
    g.zs = z != nullptr && is_f8(ztype) ? zscale : nullptr;
    g.lda = lda;
    g.ldb = ldb;
    g.ldc = ldc;
    g.ldz = ldz;
    g.lds = lds;
    g.M = M;
    g.N = N;
    g.K = reads ? K : 0;
    g.alpha = alpha;
    g.beta = beta;
    g.act = act;
    g.ztype = ztype;
    g.direct = whole(A, lda, !ta, M) && whole(B, ldb, tb, N);
    return launch(type, false, ta, tb, g, stream);
}

extern "C" int mi_gated(int type, int M, int N, int K, const void *A, int lda, const void *G, int ldg, const void *U,
                        int ldu, int biastype, const void *biasG, const void *biasU, int act, int htype, void *h,
                        int ldh, int ztype, void *g, int ldg_, float *gscale, int ldsg, void *u, int ldu_,
                        float *uscale, int ldsu, hipStream_t stream) {
    if (!is_half(type)) return MISGEMM_BAD_TYPE;
    if (M < 0) return MISGEMM_BAD_M;
    if (N < 0) return MISGEMM_BAD_N;
    if (K < 0) return MISGEMM_BAD_K;
    const bool some = M > 0 && N > 0, reads = some && K > 0;
    if (reads && A == nullptr) return MISGEMM_NULL_A;
    if (lda < K || lda < 1) return MISGEMM_BAD_LDA;
    if (reads && G == nullptr) return MISGEMM_NULL_B;
    if (ldg < K || ldg < 1) return MISGEMM_BAD_LDB;
    if (reads && U == nullptr) return MISGEMM_NULL_B;
    if (ldu < K || ldu < 1) return MISGEMM_BAD_LDB;
    if ((biasG != nullptr || biasU != nullptr) && biastype != type && biastype != MI_F32) return MISGEMM_BAD_TYPE;
    if (act < MI_ACT_NONE || act > MI_ACT_GELU_TANH) return MISGEMM_BAD_ACT;
    if (htype != type && htype != MI_F32) return MISGEMM_BAD_TYPE;
    if (some && h == nullptr) return MISGEMM_NULL_C;
    if (ldh < N || ldh < 1) return MISGEMM_BAD_LDC;
    if (g != nullptr || u != nullptr) {
        if (ztype != htype && !is_f8(ztype)) return MISGEMM_BAD_TYPE;
        if (g == nullptr) return MISGEMM_NULL_OUTPUT;
        if (ldg_ < N) return MISGEMM_BAD_LD;
        if (is_f8(ztype) && some && gscale == nullptr) return MISGEMM_NULL_SCALE;
        if (is_f8(ztype) && ldsg < M) return MISGEMM_BAD_LDS;
        if (u == nullptr) return MISGEMM_NULL_OUTPUT;
        if (ldu_ < N) return MISGEMM_BAD_LD;
        if (is_f8(ztype) && some && uscale == nullptr) return MISGEMM_NULL_SCALE;
        if (is_f8(ztype) && ldsu < M) return MISGEMM_BAD_LDS;
    }
    if (too_large(M, N, K)) return MISGEMM_TOO_LARGE;
    if (!some) return MISGEMM_SUCCESS;

    LinArgs a = {};
    a.A = A;
    a.B = G;
    a.U = U;
    a.bias = biasG;
    a.bias_u = biasU;
    a.bias32 = biastype == MI_F32;
    a.C = h;
    a.c32 = htype == MI_F32;
    a.z = g;
    a.zu = u;
    a.zs = g != nullptr && is_f8(ztype) ? gscale : nullptr;
    a.zus = u != nullptr && is_f8(ztype) ? uscale : nullptr;
    a.lda = lda;
    a.ldb = ldg;
    a.ldu = ldu;
    a.ldc = ldh;
    a.ldz = ldg_;
    a.ldzu = ldu_;
    a.lds = ldsg;
    a.ldsu = ldsu;
    a.M = M;
    a.N = N;
    a.K = K;
    a.alpha = 1.0f;
    a.act = act;
    a.ztype = ztype;
    a.direct = whole(A, lda, true, M) && whole(G, ldg, true, N) && whole(U, ldu, true, N);
    return launch(type, true, false, true, a, stream);
}
