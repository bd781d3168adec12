// mi_fp8_gemm: C = alpha * A * B^T + beta * C, A and B in 8-bit floating point
// with a scale for each block of 128.
//
// The sum over one block of k is one v_mfma_f32_16x16x128_f8f6f4 for each 16 x
// 16 outputs, started from zero; its four values per lane are then scaled
// into the FP32 accumulators: acc += (sA * sB) * part. The matrix cores take
// 32 cycles for that product and the vector ALUs 16 for the four FMAs (32
// where B has a scale for each row, whose product with sA differs at every
// output), so the scaling hides behind the products as long as another wave
// has some to issue.
//
// That instruction aligns each eight neighbouring products to the largest of
// them and cuts off what is below 2^-13 of it (measured: a product of 2^-14 of
// its neighbour is lost, one in another eight is not; so in every 8-bit form).
// Against 64 bits, and before C's rounding, sums of normal values are off by
// 0.8e-5 (E5M2 x E5M2) to 1.4e-5 (E4M3 x E4M3) of their typical size, and by
// 1.9e-5 to 3.6e-5 where the columns differ in size (exp of 0.8 times a normal
// value); the rounding to BF16 is off by up to 3.9e-3, that to FP16 by 4.9e-4.
// At worst eight products lose 7 * 2^-13 of their largest. So where C is FP32,
// whose rounding is 6e-8, the operands become BF16 in registers, which holds
// both 8-bit types exactly, and four v_mfma_f32_16x16x32_bf16 make the block's
// sum at half the rate (sums 6e-8 to 9e-8 off).
//
// The product's first operand is B and its second A: a lane then holds
// outputs of one row of A (one sA) at neighbouring columns. Which 32 values of
// k a lane group feeds does not matter as long as it is the same for both
// operands.

#include "fp8_gemm.h"

namespace {

using namespace misgemm_fp8;

// C <- beta * C where nothing is added.
__global__ __launch_bounds__(256) void fp8_scale_c(GemmArgs g) {
    const int n = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (n >= g.N) return;
    for (int m = blockIdx.y; m < g.M; m += gridDim.y) {
        float v[8] = {};
        if (g.ctype == MI_F32)
            put_row<true, 8>(g, m, n, v);
        else
            put_row<false, 8>(g, m, n, v);
    }
}

// K < 16, which the tiles' 16-byte reads would pass: one output per thread,
// the sum of its few products in order of k.
template <int FMT> __device__ __forceinline__ float value(uint8_t v) {
    if constexpr (FMT == MI_E4M3)
        return __builtin_amdgcn_cvt_f32_fp8(v, 0);
    else
        return __builtin_amdgcn_cvt_f32_bf8(v, 0);
}
template <int FA, int FB> __global__ __launch_bounds__(256) void fp8_short(GemmArgs g, bool rows) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= g.N) return;
    const float sb = g.sb[rows ? n : n / kBlock * g.ldsb];
    for (int m = blockIdx.y; m < g.M; m += gridDim.y) {
        float sum = 0.0f;
        for (int k = 0; k < g.K; ++k)
            sum = fmaf(value<FA>(g.A[m * g.lda + k]), value<FB>(g.B[n * g.ldb + k]), sum);
        float v[1] = {g.alpha * (sum * (g.sa[m] * sb))};
        if (g.ctype == MI_F32)
            put_row<true, 1>(g, m, n, v);
        else
            put_row<false, 1>(g, m, n, v);
    }
}

// The kernel that is expected to be fastest: 0 to 5 are fp8_direct.hip's tile
// shapes, 16 to 20 those of fp8_tile.hip.
//
// A product's time in us is taken to be first + round * (rounds - 1) + step *
// rounds * steps, where a round is 256 workgroups (one for each CU) and a step
// is a block of k for each of a workgroup's waves that split k. The constants
// are fitted to the measured times of all kernels on 356 shapes (M, N and K
// from 1, 64 and 64 to 8192, all types of C, kinds of scales and alignments),
// which they reproduce to 8-18%; the kernel picked was 1.8% slower than the
// fastest on average, and 43% at worst (256 x 6232 x 3248, rows 4 bytes aligned).
// They make no difference between the kinds of scales: a scale for each row of B
// costs all tiles alike (8192 x 8192 x 4096 to BF16: 286 us for 244 in tiles of
// 256 x 256, 324 for 292 in tiles of 128 x 128).
struct Cost {
    int kernel, bm, bn, waves;
    struct {
        float first, round, step;
    } fit[2][2];   // C of 16 bits; of 32, with BF16 products. Rows 16 bytes aligned; not
};
constexpr Cost kCosts[] = {
    {0, 16, 16, 16, {{{2.40f, 0.66f, 0.83f}, {1.68f, 0, 1.67f}}, {{2.26f, 0.46f, 1.01f}, {1.65f, 0, 1.69f}}}},
    {1, 16, 32, 8, {{{2.50f, 0.19f, 0.66f}, {2.21f, 0, 1.14f}}, {{2.44f, 0.77f, 0.83f}, {2.00f, 0.24f, 1.34f}}}},
    {2, 32, 32, 8, {{{2.55f, 0.23f, 0.85f}, {2.33f, 0, 1.39f}}, {{2.67f, 0.85f, 1.03f}, {2.14f, 0.37f, 1.76f}}}},
    {3, 64, 32, 8, {{{2.37f, 1.33f, 1.58f}, {2.07f, 0.82f, 2.33f}}, {{2.60f, 1.59f, 1.88f}, {1.97f, 1.29f, 2.82f}}}},
    {4, 64, 32, 4, {{{3.13f, 0.20f, 0.78f}, {3.18f, 0, 1.17f}}, {{3.27f, 0.41f, 0.98f}, {3.27f, 0.42f, 1.38f}}}},
    {5, 64, 64, 8, {{{2.96f, 2.59f, 1.96f}, {2.49f, 1.42f, 2.99f}}, {}}},
    {16, 128, 128, 1, {{{}, {5.21f, 1.55f, 0.98f}}, {{}, {6.53f, 2.46f, 1.31f}}}},
    {17, 64, 128, 1, {{{}, {3.91f, 0.13f, 0.80f}}, {{}, {4.79f, 1.17f, 1.00f}}}},
    {18, 64, 128, 1, {{{4.22f, 0.94f, 0.40f}, {}}, {{4.46f, 0.82f, 0.70f}, {}}}},
    {19, 128, 128, 1, {{{5.36f, 2.31f, 0.56f}, {}}, {{6.06f, 3.20f, 0.89f}, {}}}},
    {20, 256, 256, 1, {{{9.12f, 8.79f, 1.57f}, {}}, {}}},
};
constexpr float kSplitCost = 8.0f;   // exchanging partial tiles

int pick(const GemmArgs &g, bool rows) {
    const bool exact = g.ctype == MI_F32, near = g.lda < 1 << 24 && g.ldb < 1 << 24;
    const bool direct = g.lda < 1 << 26 && g.ldb < 1 << 26;
    int best = 16;
    float least = 3e38f;
    for (const Cost &c : kCosts) {
        const long long tiles = (g.M + c.bm - 1LL) / c.bm * ((g.N + c.bn - 1LL) / c.bn);
        if (c.kernel < 16 && (!direct || tiles * 64 * c.waves >= 1LL << 32)) continue;
        if (c.kernel == 5 && (exact || rows)) continue;   // does not fit the registers
        if (c.kernel == 20 && (exact || g.ldsb >= 1 << 28)) continue;   // nor that; 32-bit offsets of scales
        if (c.kernel >= 16 && (c.kernel > 17) != g.direct) continue;
        if (c.kernel == 17 && !near) continue;
        const int splits = c.kernel == 16 || c.kernel == 19 ? splits_of(tiles, blocks(g.K)) : 1;
        const float rounds = (float)((tiles * splits + kNumCus - 1) / kNumCus);
        const float steps = (float)((blocks(g.K) + c.waves * splits - 1) / (c.waves * splits));
        const auto &f = c.fit[exact][!g.direct];
        const float us = f.first + f.round * (rounds - 1) + f.step * rounds * steps + (splits > 1 ? kSplitCost : 0.0f);
        if (us < least) {
            least = us;
            best = c.kernel;
        }
    }
    return best;
}

}  // namespace

extern "C" int mi_fp8_gemm(int atype, int btype, int block, int ctype, int M, int N, int K, float alpha, const void *A,
                           int lda, const float *scaleA, int ldsa, const void *B, int ldb, const float *scaleB,
                           int ldsb, float beta, void *C, int ldc, hipStream_t stream) {
    if (!is_f8(atype) || !is_f8(btype)) return MISGEMM_BAD_TYPE;
    if (block != MI_BLOCK_ROW && block != MI_BLOCK_TILE) return MISGEMM_BAD_BLOCK;
    if (!is_real(ctype)) return MISGEMM_BAD_TYPE;
    if (M < 0) return MISGEMM_BAD_M;
    if (N < 0) return MISGEMM_BAD_N;
    if (K < 0) return MISGEMM_BAD_K;
    const bool some = M > 0 && N > 0, reads = some && K > 0 && alpha != 0.0f;
    if (reads && A == nullptr) return MISGEMM_NULL_A;
    if (lda < (K > 1 ? K : 1)) return MISGEMM_BAD_LDA;
    if (reads && scaleA == nullptr) return MISGEMM_NULL_SCALE;
    if (ldsa < M) return MISGEMM_BAD_LDS;
    if (reads && B == nullptr) return MISGEMM_NULL_B;
    if (ldb < (K > 1 ? K : 1)) return MISGEMM_BAD_LDB;
    if (reads && scaleB == nullptr) return MISGEMM_NULL_SCALE;
    if (ldsb < (block == MI_BLOCK_ROW ? N : blocks(K))) return MISGEMM_BAD_LDS;
    if (some && C == nullptr) return MISGEMM_NULL_C;
    if (ldc < (N > 1 ? N : 1)) return MISGEMM_BAD_LDC;
    if (!some) return MISGEMM_SUCCESS;
    // Tile counts and the launch's threads are 32-bit; columns are rounded up to tiles.
    if (((M + 127LL) / 128) * ((N + 127LL) / 128) >= 1LL << 23 || N > 0x7fffffff - 256 || M > 0x7fffffff - 256 ||
        K > 0x7fffffff - 256)
        return MISGEMM_TOO_LARGE;

    GemmArgs g;
    g.A = static_cast<const uint8_t *>(A);
    g.B = static_cast<const uint8_t *>(B);
    g.sa = scaleA;
    g.sb = scaleB;
    g.C = C;
    g.ws = nullptr;
    g.counters = nullptr;
    g.lda = lda;
    g.ldb = ldb;
    g.ldsa = ldsa;
    g.ldsb = ldsb;
    g.ldc = ldc;
    g.M = M;
    g.N = N;
    g.K = K;
    g.tiles_m = g.tiles_n = g.splits = g.kb_per_split = 0;
    g.alpha = alpha;
    g.beta = beta;
    g.ctype = ctype;
    g.direct = aligned(A, 16) && lda % 16 == 0 && lda < 1 << 24 && aligned(B, 16) && ldb % 16 == 0 && ldb < 1 << 24;
    if (!reads) {
        if (beta == 1.0f) return MISGEMM_SUCCESS;
        hipLaunchKernelGGL(fp8_scale_c, dim3((unsigned)((N + 2047LL) / 2048), (unsigned)(M < 65535 ? M : 65535)),
                           dim3(256), 0, stream, g);
        return launched();
    }
    const bool rows = block == MI_BLOCK_ROW;
    if (K < 16) {
        const dim3 grid((unsigned)((N + 255LL) / 256), (unsigned)(M < 65535 ? M : 65535));
        const auto kernel = atype == MI_E4M3
                                ? (btype == MI_E4M3 ? fp8_short<MI_E4M3, MI_E4M3> : fp8_short<MI_E4M3, MI_E5M2>)
                                : (btype == MI_E4M3 ? fp8_short<MI_E5M2, MI_E4M3> : fp8_short<MI_E5M2, MI_E5M2>);
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, g, rows);
        return launched();
    }
    const int kernel = pick(g, rows);
    return kernel < 16 ? launch_direct(atype, btype, rows, kernel, g, stream)
                       : launch_tiles(atype, btype, rows, kernel - 16, g, stream);
}
