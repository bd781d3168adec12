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

// A kernel's time in us is taken to be
//   first + round * (rounds - 1) + step * rounds * steps + share * steps * workgroups / 256
// and, where k is split, split + part * splits more: a round is 256 workgroups
// (one for each CU), a step a block of 64 values of k for each of a workgroup's
// waves that split it. The constants are fitted to the measured times of all
// kernels on 1000 shapes (M, N and K from 1, 64 and 64 to 8192, all layouts and
// alignments), each with one set of operands again and again, which the caches
// hold where it fits. They reproduce these to 5-19%; the kernel picked was 1.6%
// slower than the fastest on average, 9% in one case of twenty, 36% at worst (the
// gated 3460 x 80 x 944: 17.4 us with k split by four, 12.8 in another tile). On
// 200 other shapes, measured alike, 11% in one case of twenty and 22% at worst. On
// 70 of up to 96 rows with operands in rotation, which come from memory, 2.2% on
// average, 10% in one of twenty, 18% at worst.
struct Fit {
    float first, round, step, share;
};
struct Cost {
    int kernel, bm, bn, waves;
    float split, part;
    Fit fit[2];   // below 16: rows 16 bytes aligned; not. From 16 on: both operands with k running fastest; not
};
// 0 to 15 are linear_direct.hip's tile shapes, those from 16 on linear_tile.h's
// (below 24 for any alignment, the others for whole 16 bytes).
constexpr Cost kLinear[] = {
    {0, 16, 16, 16, 0, 0, {{2.93f, 0.41f, 0.43f, 0.24f}, {2.4f, 0.08f, 1.02f, 0.09f}}},
    {1, 16, 32, 8, 0, 0, {{3.11f, 0.26f, 0.37f, 0.1f}, {2.8f, 0, 0.77f, 0.02f}}},
    {2, 32, 32, 8, 0, 0, {{3.07f, 0.37f, 0.54f, 0.05f}, {2.63f, 0, 1.08f, 0.06f}}},
    {3, 48, 16, 8, 0, 0, {{3, 0.08f, 0.55f, 0.06f}, {2.64f, 0, 1.07f, 0}}},
    {4, 64, 32, 4, 0, 0, {{3.43f, 0, 0.51f, 0.1f}, {2.91f, 0, 0.94f, 0}}},
    {16, 128, 128, 1, 1.92f, 0.63f, {{4.45f, 2.22f, 0.47f, 0.31f}, {4.83f, 1.47f, 0.77f, 0}}},
    {17, 64, 128, 1, 1.43f, 0.41f, {{3.71f, 1.03f, 0.36f, 0.19f}, {4.38f, 0.82f, 0.51f, 0}}},
    {18, 256, 128, 1, 3.01f, 1.16f, {{6.13f, 6.81f, 0.78f, 0.5f}, {6.57f, 4.87f, 0.99f, 0.56f}}},
    {24, 64, 128, 1, 1.2f, 0.36f, {{3.88f, 1.21f, 0.26f, 0.2f}, {4.12f, 1.55f, 0.3f, 0.07f}}},
    {25, 128, 128, 1, 1.78f, 0.59f, {{4.53f, 1.47f, 0.35f, 0.57f}, {4.96f, 1.54f, 0.4f, 0.35f}}},
    {26, 128, 128, 1, 1.72f, 0.61f, {{4.96f, 4.56f, 0.37f, 0.3f}, {5.11f, 4.87f, 0.42f, 0.16f}}},
    {27, 128, 256, 1, 2.42f, 1.14f, {{6.5f, 7.02f, 0.6f, 0.64f}, {6.58f, 7.18f, 0.66f, 0.42f}}},
    {28, 256, 256, 1, 0, 0, {{9.28f, 13.97f, 0.98f, 0.98f}, {9.86f, 18.23f, 1.04f, 0.63f}}},
};
constexpr Cost kGated[] = {
    {0, 16, 16, 16, 0, 0, {{2.69f, 0.93f, 0.83f, 0.49f}, {1.84f, 0.55f, 1.82f, 0.07f}}},
    {1, 16, 16, 8, 0, 0, {{3.23f, 0, 0.36f, 0.2f}, {2.91f, 0, 0.77f, 0.02f}}},
    {2, 16, 32, 8, 0, 0, {{2.95f, 0.14f, 0.72f, 0.41f}, {2.24f, 0, 1.56f, 0}}},
    {3, 32, 16, 8, 0, 0, {{3.08f, 0, 0.58f, 0.15f}, {2.61f, 0, 1.11f, 0}}},
    {4, 64, 16, 4, 0, 0, {{3.28f, 0.42f, 0.54f, 0.06f}, {2.86f, 0.09f, 1.01f, 0}}},
    {16, 128, 128, 1, 3.13f, 1.18f, {{5.93f, 7.01f, 0.78f, 0.41f}, {}}},
    {17, 64, 128, 1, 1.96f, 0.65f, {{4.43f, 1.81f, 0.53f, 0.31f}, {}}},
    {24, 64, 128, 1, 1.92f, 0.6f, {{4.43f, 3.81f, 0.45f, 0.34f}, {}}},
    {25, 64, 128, 1, 2, 0.62f, {{4.39f, 0.62f, 0.4f, 0.59f}, {}}},
    {26, 128, 64, 1, 1.81f, 0.63f, {{4.42f, 4.17f, 0.36f, 0.23f}, {}}},
    {27, 128, 64, 1, 1.78f, 0.65f, {{4.15f, 1.19f, 0.35f, 0.39f}, {}}},
    {28, 128, 128, 1, 2.98f, 1.14f, {{5.8f, 6.87f, 0.61f, 0.41f}, {}}},
    {29, 256, 128, 1, 0, 0, {{8.06f, 10, 0.99f, 0.67f}, {}}},
};

// The kernel that is expected to be fastest, and how many workgroups share its k.
int pick(LinArgs &g, bool gated, bool ta, bool tb) {
    const Cost *costs = gated ? kGated : kLinear;
    const int count = gated ? sizeof kGated / sizeof *kGated : sizeof kLinear / sizeof *kLinear;
    const bool kmajor = !ta && tb;
    const bool few = kmajor && g.zs == nullptr && g.K >= 8 && g.lda < 1 << 25 && g.ldb < 1 << 25 && g.ldu < 1 << 25;
    const int kblocks = (g.K + kStep - 1) / kStep;
    int best = 16;
    float least = 3e38f;
    g.splits = 1;
    for (const Cost *c = costs; c < costs + count; ++c) {
        const long long tiles = (g.M + c->bm - 1LL) / c->bm * ((g.N + c->bn - 1LL) / c->bn);
        if (c->kernel < 16 ? !few || tiles * 64 * c->waves >= 1LL << 32 : c->kernel >= 24 ? !g.direct : c->kernel > 16 && !g.near) continue;
        if (gated && g.zs != nullptr && c->bn < kBlock) continue;   // a scale's columns are in one workgroup
        const Fit &f = c->fit[c->kernel < 16 ? !g.direct : !kmajor];
        // At least three blocks of k for each workgroup, three workgroups to a CU at most, and parts that fit the workspace.
        auto shared = [&](int splits) {
            return c->split > 0.0f && splits <= 16 && kblocks / splits >= 3 && tiles * splits <= 3 * kNumCus &&
                   parts_fit(tiles, splits, c->bm * c->bn * (gated ? 2 : 1));
        };
        for (int splits = 1; splits == 1 || shared(splits); splits *= 2) {
            const float groups = (float)(tiles * splits);
            const float rounds = (float)((tiles * splits + kNumCus - 1) / kNumCus);
            const int each = (kblocks + splits - 1) / splits;
            const float steps = (float)((each + c->waves - 1) / c->waves);
            float us = f.first + f.round * (rounds - 1) + f.step * rounds * steps + f.share * steps * groups / kNumCus;
            if (splits > 1) us += c->split + c->part * splits;
            if (us < least) {
                least = us;
                best = c->kernel;
                g.splits = splits;
            }
        }
    }
    return best;
}

int launch(int type, bool gated, bool ta, bool tb, LinArgs &g, hipStream_t stream) {
    const int kernel = pick(g, gated, ta, tb);
    if (kernel < 16) return launch_direct(type, gated, kernel, g, stream);
    return type == MI_BF16 ? launch_tiles_bf16(gated, ta, tb, kernel - 16, g, stream)
                           : launch_tiles_f16(gated, ta, tb, kernel - 16, g, stream);
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
    g.alpha = reads ? alpha : 0.0f;   // without a sum an infinite alpha has no part in z either
    g.beta = beta;
    g.act = act;
    g.ztype = ztype;
    g.direct = whole(A, lda, !ta, M) && whole(B, ldb, tb, N);
    g.near = lda < 1 << 23 && ldb < 1 << 23 && (ta ? M : K) >= 8 && (tb ? K : N) >= 8;
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
    a.near = lda < 1 << 23 && ldg < 1 << 23 && ldu < 1 << 23 && K >= 8;
    return launch(type, true, false, true, a, stream);
}
