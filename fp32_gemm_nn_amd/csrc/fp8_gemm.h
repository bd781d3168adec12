// What the kernels of mi_fp8_gemm share: arguments, operands of the matrix
// instructions, the tile order and the output. The mathematics is described
// in fp8_gemm.hip.
#ifndef MISGEMM_FP8_GEMM_H
#define MISGEMM_FP8_GEMM_H

#include "fp8_common.h"
#include "workspace.h"

namespace misgemm_fp8 {

constexpr int kNumCus = 256;
constexpr int kXcds = 8;

struct GemmArgs {
    const uint8_t *A, *B;
    const float *sa, *sb;
    void *C;
    float *ws;
    int *counters;
    long long lda, ldb, ldsa, ldsb, ldc;
    int M, N, K;
    int tiles_m, tiles_n, splits, kb_per_split;
    float alpha, beta;
    int ctype;
    bool direct;   // 16-byte aligned rows, less than 2^24 apart: copied to LDS without registers
};

// Lane values of one operand of a 16 x 16 x 128 product: the 32 bytes as they
// are, or (EXACT) as BF16.
template <bool EXACT> struct Operand {
    i32x8 v;
};
template <> struct Operand<true> {
    bf16x8 v[4];
};

template <int FMT> __device__ __forceinline__ bf16x8 widen(int lo, int hi) {
    bf16x2 w[4];
    if constexpr (FMT == MI_E4M3) {
        w[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
        w[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
        w[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
        w[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    } else {
        w[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
        w[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
        w[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
        w[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
    }
    const bf16x4 a = __builtin_shufflevector(w[0], w[1], 0, 1, 2, 3), b = __builtin_shufflevector(w[2], w[3], 0, 1, 2, 3);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

typedef int words16 __attribute__((ext_vector_type(4), aligned(1)));

// 16 bytes moved down by `over` bytes, zeros after them.
__device__ __forceinline__ i32x4 shifted(i32x4 w, int over) {
    unsigned long long lo = (uint32_t)w[0] | (unsigned long long)(uint32_t)w[1] << 32;
    unsigned long long hi = (uint32_t)w[2] | (unsigned long long)(uint32_t)w[3] << 32;
    if (over >= 8) {
        lo = over < 16 ? hi >> (8 * over - 64) : 0;
        hi = 0;
    } else if (over > 0) {
        lo = lo >> (8 * over) | hi << (64 - 8 * over);
        hi >>= 8 * over;
    }
    return i32x4{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
}

// The builtin's operand selectors: 0 is E4M3, 1 is E5M2.
template <int FA, int FB, bool EXACT>
__device__ __forceinline__ f32x4 product(const Operand<EXACT> &a, const Operand<EXACT> &b) {
    f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (EXACT) {
#pragma unroll
        for (int s = 0; s < 4; ++s) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[s], b.v[s], p, 0, 0, 0);
        return p;
    } else {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, p, FA == MI_E5M2, FB == MI_E5M2, 0, 0, 0, 0);
    }
}

// N neighbouring outputs of row m from column n on.
template <class T, int N> __device__ __forceinline__ void put(const GemmArgs &g, int m, int n, float (&v)[N]) {
    T *c = static_cast<T *>(g.C) + m * g.ldc + n;
    if (g.beta != 0.0f) {
        float old[N];
        load<T, N>(c, g.N - n, old);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = fmaf(g.beta, old[j], v[j]);
    }
    store<T, N>(c, g.N - n, v);
}
template <bool EXACT, int N> __device__ __forceinline__ void put_row(const GemmArgs &g, int m, int n, float (&v)[N]) {
    if (m >= g.M || n >= g.N) return;
    if constexpr (EXACT)
        put<float, N>(g, m, n, v);
    else if (g.ctype == MI_BF16)
        put<bf16, N>(g, m, n, v);
    else
        put<f16, N>(g, m, n, v);
}

// The tile of workgroup `id`. Workgroups go round the XCDs in turn; each XCD
// gets a run of tiles, eight rows of tiles at a time, so that its L2 serves
// panels of A and B to neighbours.
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int total = tiles_m * tiles_n, per = total / kXcds;
    if (id < per * kXcds) id = (id % kXcds) * per + id / kXcds;
    constexpr int GROUP = 8;
    const int band = id / (GROUP * tiles_n), first = band * GROUP, height = min(GROUP, tiles_m - first);
    const int in = id - band * GROUP * tiles_n;
    tm = first + in % height;
    tn = in / height;
}

// Workgroups that share a tile's k, where 128 x 128 tiles leave half of the
// two places on each CU empty: at least four blocks of k for each.
inline int splits_of(long long tiles, int kblocks) {
    long long splits = 2 * kNumCus / tiles;
    if (splits > kblocks / 4) splits = kblocks / 4;
    if (splits <= 1) return 1;
    const int each = (int)((kblocks + splits - 1) / splits);
    return (kblocks + each - 1) / each;
}

// Products of few outputs, without a barrier in their sum (fp8_direct.hip),
// and in tiles that go through LDS (fp8_tile.hip). `shape` names one of their
// tile shapes.
int launch_direct(int atype, int btype, bool rows, int shape, GemmArgs &g, hipStream_t stream);
int launch_tiles(int atype, int btype, bool rows, int shape, GemmArgs &g, hipStream_t stream);

}  // namespace misgemm_fp8

#endif  // MISGEMM_FP8_GEMM_H
