// mi_fp8_quantize: a matrix in 8-bit floating point with a scale for each
// block of 128, the same for its transpose, or both from one pass.
//
// With T the type's largest value and a = max(max |x|, 2^-100) over a block,
// scale = a / T and q = rn(x * (T / a)).
//
// Bound by memory: each value is read once (2 or 4 bytes) and written once or
// twice (1 byte each).

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

// One workgroup takes a 128 x 128 block: one scale block in either direction
// and for either kind, so no maximum crosses workgroups. Thread t holds the
// 8 x 8 values at rows 8*(t/16).., columns 8*(t%16)..: 16 lanes read a row's
// 128 values in one wide access each, and the transpose needs no exchange
// but the one that makes its stores whole rows (16 KB of LDS).
template <class T, int FMT, bool TILE, bool QT>
__global__ __launch_bounds__(256) void quantize(QuantArgs a) {
    constexpr int LD = kBlock + 16;   // bytes between rows of the transposed block in LDS
    __shared__ __align__(16) uint8_t block[QT ? kBlock * LD : 16];
    __shared__ float colmax[16][kBlock];
    __shared__ float wavemax[4];
    const int tid = threadIdx.x, tc = tid % 16, tr = tid / 16;
    const int rb = blockIdx.y, cb = blockIdx.x;
    const int row0 = rb * kBlock + tr * 8, col0 = cb * kBlock + tc * 8;
    const int nc = min(8, max(0, a.cols - col0));
    const T *x = static_cast<const T *>(a.x) + row0 * a.ldx + col0;

    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) load8(x + i * a.ldx, row0 + i < a.rows ? nc : 0, v[i]);

    float rowmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        rowmax[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) rowmax[i] = fmaxf(rowmax[i], fabsf(v[i][j]));
    }
    if constexpr (TILE) {
        float m = rowmax[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) m = fmaxf(m, rowmax[i]);
        m = max_over<64>(m);
        if (tid % 64 == 0) wavemax[tid / 64] = m;
        __syncthreads();
        m = fmaxf(fmaxf(fmaxf(wavemax[0], wavemax[1]), fmaxf(wavemax[2], wavemax[3])), kTiny);
#pragma unroll
        for (int i = 0; i < 8; ++i) rowmax[i] = m;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) rowmax[i] = fmaxf(max_over<16>(rowmax[i]), kTiny);
    }

    if (a.q != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = top<FMT>() / rowmax[i];
            const int w[2] = {pack4<FMT>(v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f),
                              pack4<FMT>(v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f)};
            if (row0 + i < a.rows) {
                store_bytes<8>(a.q + (row0 + i) * a.ldq + col0, nc, w);
                if (!TILE && tc == 0) a.scale[cb * a.lds + row0 + i] = rowmax[i] / top<FMT>();
            }
        }
        if (TILE && tid == 0) a.scale[rb * a.lds + cb] = rowmax[0] / top<FMT>();
    }

    if constexpr (QT) {
        float m[8];
        if constexpr (TILE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = rowmax[0];
            if (tid == 0) a.scale_t[cb * a.lds_t + rb] = rowmax[0] / top<FMT>();
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m[j] = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m[j] = fmaxf(m[j], fabsf(v[i][j]));
                colmax[tr][tc * 8 + j] = m[j];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int r = 0; r < 16; ++r) m[j] = fmaxf(m[j], colmax[r][tc * 8 + j]);
                m[j] = fmaxf(m[j], kTiny);
                if (tr == 0 && col0 + j < a.cols) a.scale_t[rb * a.lds_t + col0 + j] = m[j] / top<FMT>();
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = top<FMT>() / m[j];
            i32x2 w;
            w[0] = pack4<FMT>(v[0][j] * f, v[1][j] * f, v[2][j] * f, v[3][j] * f);
            w[1] = pack4<FMT>(v[4][j] * f, v[5][j] * f, v[6][j] * f, v[7][j] * f);
            *reinterpret_cast<i32x2 *>(block + (tc * 8 + j) * LD + tr * 8) = w;
        }
        __syncthreads();
        // Rows of the transpose: 8 lanes write one row's 128 bytes.
        const int n0 = rb * kBlock + (tid % 8) * 16;
        const int n = min(16, max(0, a.rows - n0));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = tid / 8 + 32 * i;
            if (cb * kBlock + j >= a.cols) break;
            const i32x4 w = *reinterpret_cast<const i32x4 *>(block + j * LD + (tid % 8) * 16);
            const int words[4] = {w[0], w[1], w[2], w[3]};
            store_bytes<16>(a.qt + (cb * kBlock + j) * a.ldqt + n0, n, words);
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
