// mi_fp8_quantize: a matrix in 8-bit floating point with a scale for each
// block of 128, the same for its transpose, or both from one pass.
//
// With T the type's largest value and a = max(max |x|, 2^-100) over a block,
// scale = a / T and q = rn(x * (T / a)).
//
// Bound by memory: each value is read once (2 or 4 bytes) and written once or
// twice (1 byte each). 8192 x 4096 in BF16, both ways: 28 us (4.8 TB/s; a large
// copy reaches 5.4); 4096 x 4096 in FP32 with tile blocks, both ways: 19.6 us
// (5.1 TB/s).

#include "fp8_common.h"

namespace {

using namespace misgemm_fp8;

struct QuantArgs {
    const void *x;
    uint8_t *q, *qt;
    float *scale, *scale_t;
    long long ldx, ldq, ldqt, lds, lds_t;
    int rows, cols;
};

// The I-th of eight rows' factors, which lanes 0 to 7 of each 16 hold.
__device__ __forceinline__ void spread(float mine, float (&f)[8]) {
    f[0] = of16<0>(mine);
    f[1] = of16<1>(mine);
    f[2] = of16<2>(mine);
    f[3] = of16<3>(mine);
    f[4] = of16<4>(mine);
    f[5] = of16<5>(mine);
    f[6] = of16<6>(mine);
    f[7] = of16<7>(mine);
}

// One workgroup takes a 128 x 128 block: one scale block in either direction
// and for either kind, so no maximum crosses workgroups. Thread t holds the
// 8 x 8 values at rows 8*(t/16).., columns 8*(t%16)..: 16 lanes read a row's
// 128 values in one wide access each, and the transpose needs no exchange
// but the one that makes its stores whole rows (16 KB of LDS). Each division
// by a maximum is made by one thread, for all that share it.
template <class T, int FMT, bool TILE, bool QT>
__global__ __launch_bounds__(256) void quantize(QuantArgs a) {
    // The transposed block: 8 bytes k of row c at k ^ (c / 8), so that neither
    // the columns that are written nor the rows that are read share banks.
    // Before that the columns' maxima over eight rows each.
    __shared__ union {
        i32x2 block[kBlock][16];
        float colmax[16][kBlock];
    } lds;
    __shared__ float factor_t[kBlock];
    __shared__ float wavemax[4];
    const int tid = threadIdx.x, tc = tid % 16, tr = tid / 16;
    const int rb = blockIdx.y, cb = blockIdx.x;
    const int row0 = rb * kBlock + tr * 8, col0 = cb * kBlock + tc * 8;
    const int nc = min(8, max(0, a.cols - col0));
    const T *x = static_cast<const T *>(a.x);

    // The same for the whole workgroup, and without a branch for each value:
    // reads past an edge are of the last row and the row's last eight values.
    Eight<T, false> v[8];
    if ((cb + 1) * kBlock <= a.cols && (rb + 1) * kBlock <= a.rows) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i].fetch(x + (row0 + i) * a.ldx, col0, a.cols);
    } else if (a.cols >= 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i].fetch(x + min(row0 + i, a.rows - 1) * a.ldx, col0, a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i].settle(row0 + i < a.rows ? col0 : a.cols, a.cols);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i].v[j] = static_cast<T>(0.0f);
                if (row0 + i < a.rows && j < nc) v[i].v[j] = x[(row0 + i) * a.ldx + col0 + j];
            }
    }
    auto value = [&](int i, int j) { return static_cast<float>(v[i].v[j]); };

    float rowf[8];   // T / maximum, of each row
    float tilef = 0.0f;
    if constexpr (TILE) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(value(i, j)));
        m = max_over<64>(m);
        if (tid % 64 == 0) wavemax[tid / 64] = m;
        __syncthreads();
        m = fmaxf(fmaxf(fmaxf(wavemax[0], wavemax[1]), fmaxf(wavemax[2], wavemax[3])), kTiny);
        tilef = top<FMT>() / m;
#pragma unroll
        for (int i = 0; i < 8; ++i) rowf[i] = tilef;
        if (tid == 0) {
            const float scale = m / top<FMT>();
            if (a.q != nullptr) a.scale[rb * a.lds + cb] = scale;
            if constexpr (QT) a.scale_t[cb * a.lds_t + rb] = scale;
        }
    } else {
        if constexpr (QT) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(value(i, j)));
                lds.colmax[tr][tc * 8 + j] = m;
            }
            __syncthreads();
            if (tid < kBlock) {
                float m = kTiny;
#pragma unroll
                for (int r = 0; r < 16; ++r) m = fmaxf(m, lds.colmax[r][tid]);
                factor_t[tid] = top<FMT>() / m;
                if (cb * kBlock + tid < a.cols) a.scale_t[rb * a.lds_t + cb * kBlock + tid] = m / top<FMT>();
            }
        }
        if (a.q != nullptr) {
            float mine = 0.0f;   // the maximum of row tc % 8
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(value(i, j)));
                m = max_over<16>(m);
                if (tc % 8 == i) mine = m;
            }
            mine = fmaxf(mine, kTiny);
            if (tc < 8 && row0 + tc < a.rows) a.scale[cb * a.lds + row0 + tc] = mine / top<FMT>();
            spread(top<FMT>() / mine, rowf);
        }
    }

    if (a.q != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = rowf[i];
            const int w[2] = {pack4<FMT>(value(i, 0) * f, value(i, 1) * f, value(i, 2) * f, value(i, 3) * f),
                              pack4<FMT>(value(i, 4) * f, value(i, 5) * f, value(i, 6) * f, value(i, 7) * f)};
            if (row0 + i < a.rows) store_bytes<8>(a.q + (row0 + i) * a.ldq + col0, nc, w);
        }
    }

    if constexpr (QT) {
        if constexpr (!TILE) __syncthreads();   // the factors are there, the maxima read
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = TILE ? tilef : factor_t[tc * 8 + j];
            i32x2 w;
            w[0] = pack4<FMT>(value(0, j) * f, value(1, j) * f, value(2, j) * f, value(3, j) * f);
            w[1] = pack4<FMT>(value(4, j) * f, value(5, j) * f, value(6, j) * f, value(7, j) * f);
            lds.block[tc * 8 + j][tr ^ tc] = w;
        }
        __syncthreads();
        // Rows of the transpose: 8 lanes write one row's 128 bytes.
        const int n0 = rb * kBlock + (tid % 8) * 16;
        const int n = min(16, max(0, a.rows - n0));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = tid / 8 + 32 * i, s = c / 8, k = (tid % 8) * 2;
            if (cb * kBlock + c >= a.cols) break;
            const i32x2 lo = lds.block[c][k ^ s], hi = lds.block[c][(k + 1) ^ s];
            const int words[4] = {lo[0], lo[1], hi[0], hi[1]};
            store_bytes<16>(a.qt + (cb * kBlock + c) * a.ldqt + n0, n, words);
        }
    }
}

template <class T, int FMT, bool TILE> int launch_qt(const QuantArgs &a, hipStream_t stream) {
    const dim3 grid((unsigned)blocks(a.cols), (unsigned)blocks(a.rows));
    if (a.qt != nullptr)
        hipLaunchKernelGGL((quantize<T, FMT, TILE, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((quantize<T, FMT, TILE, false>), grid, dim3(256), 0, stream, a);
    return launched();
}

template <class T> int launch(int ftype, int block, const QuantArgs &a, hipStream_t stream) {
    if (ftype == MI_E4M3)
        return block == MI_BLOCK_TILE ? launch_qt<T, MI_E4M3, true>(a, stream) : launch_qt<T, MI_E4M3, false>(a, stream);
    return block == MI_BLOCK_TILE ? launch_qt<T, MI_E5M2, true>(a, stream) : launch_qt<T, MI_E5M2, false>(a, stream);
}

}  // namespace

extern "C" int mi_fp8_quantize(int xtype, int rows, int cols, const void *x, int ldx, int ftype, int block, void *q,
                               int ldq, float *scale, int lds, void *qt, int ldqt, float *scale_t, int lds_t,
                               hipStream_t stream) {
    if (!is_real(xtype)) return MISGEMM_BAD_TYPE;
    if (rows < 0) return MISGEMM_BAD_ROWS;
    if (cols < 0) return MISGEMM_BAD_COLS;
    const bool some = rows > 0 && cols > 0;
    if (some && x == nullptr) return MISGEMM_NULL_INPUT;
    if (ldx < cols) return MISGEMM_BAD_LD;
    if (!is_f8(ftype)) return MISGEMM_BAD_TYPE;
    if (block != MI_BLOCK_ROW && block != MI_BLOCK_TILE) return MISGEMM_BAD_BLOCK;
    if (some && q == nullptr && qt == nullptr) return MISGEMM_NULL_OUTPUT;
    const bool tile = block == MI_BLOCK_TILE;
    if (q != nullptr) {
        if (ldq < cols) return MISGEMM_BAD_LD;
        if (some && scale == nullptr) return MISGEMM_NULL_SCALE;
        if (lds < (tile ? blocks(cols) : rows)) return MISGEMM_BAD_LDS;
    }
    if (qt != nullptr) {
        if (ldqt < rows) return MISGEMM_BAD_LD;
        if (some && scale_t == nullptr) return MISGEMM_NULL_SCALE;
        if (lds_t < (tile ? blocks(rows) : cols)) return MISGEMM_BAD_LDS;
    }
    // Row blocks are the grid's y; its x holds less than 2^32 threads.
    if (blocks(rows) > 65535 || blocks(cols) >= 1 << 24) return MISGEMM_TOO_LARGE;
    if (!some) return MISGEMM_SUCCESS;

    QuantArgs a;
    a.x = x;
    a.q = static_cast<uint8_t *>(q);
    a.qt = static_cast<uint8_t *>(qt);
    a.scale = scale;
    a.scale_t = scale_t;
    a.ldx = ldx;
    a.ldq = ldq;
    a.ldqt = ldqt;
    a.lds = lds;
    a.lds_t = lds_t;
    a.rows = rows;
    a.cols = cols;
    if (xtype == MI_F32) return launch<float>(ftype, block, a, stream);
    if (xtype == MI_BF16) return launch<bf16>(ftype, block, a, stream);
    return launch<f16>(ftype, block, a, stream);
}
