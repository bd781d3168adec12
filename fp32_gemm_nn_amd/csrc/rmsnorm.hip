// mi_rmsnorm and mi_rmsnorm_backward: the root-mean-square norm of each row
// with the residual's addition and an 8-bit output, and its gradients.
//
// Both are bound by memory: every operand is read once and every output
// written once; a row stays in registers between its sum and its use.

#include "fp8_common.h"
#include "workspace.h"

namespace {

using namespace misgemm_fp8;

constexpr int kNumCus = 256;
constexpr int kMaxWaves = 16;

struct NormArgs {
    const void *x, *res, *weight;
    void *h, *y;
    uint8_t *q;
    float *scale, *rstd;
    long long ldx, ldr, ldh, ldy, ldq, lds;
    int rows, cols;
    float eps;
};

// Sum over a workgroup of W waves, in every thread, in a fixed order. `part`
// is not reused before another barrier.
template <int W> __device__ __forceinline__ float block_sum(float v, float *part) {
    v = sum_over<64>(v);
    if constexpr (W == 1) return v;
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w];
    return v;
}

// y of eight values, y and q out. The 16 lanes that hold 128 columns share a scale.
template <class T, int FMT>
__device__ __forceinline__ void norm_out(const NormArgs &a, long long row, int col, int n, const float (&h)[8],
                                         const float (&w)[8], float rstd) {
    float y[8], m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = h[j] * rstd * w[j];
        m = fmaxf(m, fabsf(y[j]));
    }
    if (a.y != nullptr && n > 0) store8(static_cast<T *>(a.y) + row * a.ldy + col, n, y);
    if (a.q == nullptr) return;
    m = fmaxf(max_over<16>(m), kTiny);
    if (n <= 0) return;
    const float f = top<FMT>() / m;
    const int b[2] = {pack4<FMT>(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                      pack4<FMT>(y[4] * f, y[5] * f, y[6] * f, y[7] * f)};
    store_bytes<8>(a.q + row * a.ldq + col, n, b);
    if (col % kBlock == 0) a.scale[(col / kBlock) * a.lds + row] = m / top<FMT>();
}

// h of eight values: x plus the residual, rounded to T as it is kept.
template <class T>
__device__ __forceinline__ void norm_in(const NormArgs &a, long long row, int col, int n, float (&h)[8]) {
    load8(static_cast<const T *>(a.x) + row * a.ldx + col, n, h);
    if (a.res != nullptr) {
        float r[8];
        load8(static_cast<const T *>(a.res) + row * a.ldr + col, n, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = static_cast<float>(static_cast<T>(h[j] + r[j]));
    }
}

// One workgroup of W waves per row; PER eights of columns per thread stay in
// registers. PER == 0: rows too long for that are read again for the output.
template <class T, class TW, int FMT, int W, int PER>
__global__ __launch_bounds__(64 * W) void rmsnorm(NormArgs a) {
    constexpr int NT = 64 * W;
    // Two turns of partial sums: a wave still reading one row's is at most one
    // barrier behind the wave that writes the next row's.
    __shared__ float parts[2][W];
    const int tid = threadIdx.x;
    const TW *weight = static_cast<const TW *>(a.weight);
    int turn = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        float *part = parts[turn];
        T *hout = a.h == nullptr ? nullptr : static_cast<T *>(a.h) + row * a.ldh;
        float sum = 0.0f;
        if constexpr (PER > 0) {
            float h[PER][8], w[PER][8];
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                const int col = (tid + NT * p) * 8;
                norm_in<T>(a, row, col, a.cols - col, h[p]);
                load8(weight + col, a.cols - col, w[p]);
            }
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                const int col = (tid + NT * p) * 8;
                if (hout != nullptr && col < a.cols) store8(hout + col, a.cols - col, h[p]);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fmaf(h[p][j], h[p][j], sum);
            }
            const float rstd = 1.0f / sqrtf(block_sum<W>(sum, part) / a.cols + a.eps);
            if (a.rstd != nullptr && tid == 0) a.rstd[row] = rstd;
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                const int col = (tid + NT * p) * 8;
                norm_out<T, FMT>(a, row, col, a.cols - col, h[p], w[p], rstd);
            }
        } else {
            for (long long c0 = 0; c0 < a.cols; c0 += NT * 8) {
                const long long c = c0 + tid * 8;
                if (c >= a.cols) break;
                const int col = (int)c;
                float h[8];
                norm_in<T>(a, row, col, a.cols - col, h);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fmaf(h[j], h[j], sum);
            }
            const float rstd = 1.0f / sqrtf(block_sum<W>(sum, part) / a.cols + a.eps);
            if (a.rstd != nullptr && tid == 0) a.rstd[row] = rstd;
            // Each thread writes h where it alone reads x and the residual, after
            // it has read them: h may be either.
            for (long long c0 = 0; c0 < a.cols; c0 += NT * 8) {
                // Lanes past the row stay for the maximum over their 16, with nothing.
                const long long c = c0 + tid * 8;
                const int n = c < a.cols ? a.cols - (int)c : 0, col = c < a.cols ? (int)c : a.cols;
                float h[8], w[8];
                norm_in<T>(a, row, col, n, h);
                load8(weight + col, n, w);
                if (hout != nullptr && n > 0) store8(hout + col, n, h);
                norm_out<T, FMT>(a, row, col, n, h, w, rstd);
            }
        }
    }
}

template <class T, class TW, int FMT> int launch_norm(const NormArgs &a, hipStream_t stream) {
    // A grid of 2^20 workgroups stays within the 2^32 threads of a launch.
    const dim3 grid((unsigned)(a.rows < (1 << 20) ? a.rows : 1 << 20));
    if (a.cols <= 512)
        hipLaunchKernelGGL((rmsnorm<T, TW, FMT, 1, 1>), grid, dim3(64), 0, stream, a);
    else if (a.cols <= 2048)
        hipLaunchKernelGGL((rmsnorm<T, TW, FMT, 4, 1>), grid, dim3(256), 0, stream, a);
    else if (a.cols <= 4096)
        hipLaunchKernelGGL((rmsnorm<T, TW, FMT, 4, 2>), grid, dim3(256), 0, stream, a);
    else if (a.cols <= 8192)
        hipLaunchKernelGGL((rmsnorm<T, TW, FMT, 16, 1>), grid, dim3(1024), 0, stream, a);
    else if (a.cols <= 16384)
        hipLaunchKernelGGL((rmsnorm<T, TW, FMT, 16, 2>), grid, dim3(1024), 0, stream, a);
    else
        hipLaunchKernelGGL((rmsnorm<T, TW, FMT, 16, 0>), grid, dim3(1024), 0, stream, a);
    return launched();
}

template <class T, class TW> int launch_norm(int ftype, const NormArgs &a, hipStream_t stream) {
    return ftype == MI_E5M2 ? launch_norm<T, TW, MI_E5M2>(a, stream) : launch_norm<T, TW, MI_E4M3>(a, stream);
}

struct BackArgs {
    const void *dy, *h, *weight, *dh;
    const float *rstd;
    void *dx;
    float *dweight, *partials;
    long long lddy, ldh, lddh, lddx;
    int rows, cols, groups;
    float beta;
};

// dx of eight columns of one row, and their share of the weight's gradient.
template <class T>
__device__ __forceinline__ void back_out(const BackArgs &a, long long row, int col, int n, const float (&dy)[8],
                                         const float (&u)[8], const float (&w)[8], float rstd, float mean,
                                         float (&dw)[8]) {
    float dx[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        dx[j] = rstd * (dy[j] * w[j] - u[j] * mean);
        dw[j] = fmaf(dy[j], u[j], dw[j]);
    }
    if (n <= 0) return;
    if (a.dh != nullptr) {
        float r[8];
        load8(static_cast<const T *>(a.dh) + row * a.lddh + col, n, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[j] += r[j];
    }
    store8(static_cast<T *>(a.dx) + row * a.lddx + col, n, dx);
}

// Workgroup g takes rows g, g + groups, ... and keeps its columns' share of
// the weight's gradient in registers: it writes one row of `partials`.
template <class T, class TW, int W, int PER>
__global__ __launch_bounds__(64 * W) void rmsnorm_back(BackArgs a) {
    constexpr int NT = 64 * W;
    __shared__ float part[2][W];
    const int tid = threadIdx.x;
    float w[PER][8], dw[PER][8];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int col = (tid + NT * p) * 8;
        load8(static_cast<const TW *>(a.weight) + col, a.cols - col, w[p]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[p][j] = 0.0f;
    }
    int turn = 0;
    for (long long row = blockIdx.x; row < a.rows; row += a.groups, turn ^= 1) {
        const float rstd = a.rstd[row];
        float dy[PER][8], u[PER][8], sum = 0.0f;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int col = (tid + NT * p) * 8, n = a.cols - col;
            load8(static_cast<const T *>(a.dy) + row * a.lddy + col, n, dy[p]);
            load8(static_cast<const T *>(a.h) + row * a.ldh + col, n, u[p]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u[p][j] *= rstd;
                sum = fmaf(dy[p][j] * w[p][j], u[p][j], sum);
            }
        }
        // Two turns of `part`: a wave still reading one row's sums is at most
        // one barrier behind the wave that writes the next row's.
        const float mean = block_sum<W>(sum, part[turn]) / a.cols;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int col = (tid + NT * p) * 8;
            back_out<T>(a, row, col, a.cols - col, dy[p], u[p], w[p], rstd, mean, dw[p]);
        }
    }
    if (a.partials != nullptr) {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int col = (tid + NT * p) * 8;
            if (col < a.cols) store8(a.partials + (long long)blockIdx.x * a.cols + col, a.cols - col, dw[p]);
        }
    }
}

// Rows too long for registers: dx alone, each row read twice.
template <class T, class TW>
__global__ __launch_bounds__(64 * kMaxWaves) void rmsnorm_back_long(BackArgs a) {
    constexpr int NT = 64 * kMaxWaves;
    __shared__ float parts[2][kMaxWaves];
    int turn = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const float rstd = a.rstd[row];
        float sum = 0.0f;
        for (long long c = threadIdx.x * 8; c < a.cols; c += NT * 8) {
            const int col = (int)c, n = a.cols - col;
            float dy[8], u[8], w[8];
            load8(static_cast<const T *>(a.dy) + row * a.lddy + col, n, dy);
            load8(static_cast<const T *>(a.h) + row * a.ldh + col, n, u);
            load8(static_cast<const TW *>(a.weight) + col, n, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(dy[j] * w[j], u[j] * rstd, sum);
        }
        const float mean = block_sum<kMaxWaves>(sum, parts[turn]) / a.cols;
        for (long long c = threadIdx.x * 8; c < a.cols; c += NT * 8) {
            const int col = (int)c, n = a.cols - col;
            float dy[8], u[8], w[8], dw[8] = {};
            load8(static_cast<const T *>(a.dy) + row * a.lddy + col, n, dy);
            load8(static_cast<const T *>(a.h) + row * a.ldh + col, n, u);
            load8(static_cast<const TW *>(a.weight) + col, n, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] *= rstd;
            back_out<T>(a, row, col, n, dy, u, w, rstd, mean, dw);
        }
    }
}

// The weight's gradient of 64 columns from dy and h themselves: four waves
// sum every fourth row each. For what has no partial sums.
template <class T>
__global__ __launch_bounds__(256) void weight_grad(BackArgs a) {
    __shared__ float part[4][64];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int col = blockIdx.x * 64 + lane;
    float sum = 0.0f;
    if (col < a.cols)
        for (long long row = wave; row < a.rows; row += 4)
            sum = fmaf(static_cast<float>(static_cast<const T *>(a.dy)[row * a.lddy + col]),
                       static_cast<float>(static_cast<const T *>(a.h)[row * a.ldh + col]) * a.rstd[row], sum);
    part[wave][lane] = sum;
    __syncthreads();
    if (wave == 0 && col < a.cols) {
        sum = ((part[0][lane] + part[1][lane]) + part[2][lane]) + part[3][lane];
        a.dweight[col] = a.beta == 0.0f ? sum : fmaf(a.beta, a.dweight[col], sum);
    }
}

// Partial rows summed: 32 columns per workgroup, 8 threads of each column
// take every eighth row, and one adds theirs.
__global__ __launch_bounds__(256) void sum_partials(BackArgs a) {
    __shared__ float part[8][32];
    const int lane = threadIdx.x % 32, turn = threadIdx.x / 32;
    const int col = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (col < a.cols)
        for (int g = turn; g < a.groups; g += 8) sum += a.partials[(long long)g * a.cols + col];
    part[turn][lane] = sum;
    __syncthreads();
    if (turn == 0 && col < a.cols) {
#pragma unroll
        for (int t = 1; t < 8; ++t) sum += part[t][lane];
        a.dweight[col] = a.beta == 0.0f ? sum : fmaf(a.beta, a.dweight[col], sum);
    }
}

template <class T, class TW> int launch_back(BackArgs a, hipStream_t stream) {
    const bool in_registers = a.cols <= 16384;
    if (a.dweight != nullptr) {
        float *partials = nullptr;
        int *counters = nullptr;
        static_assert(size_t(2) * kNumCus * 16384 <= misgemm_workspace::kFloats, "partial rows fit the workspace");
        if (in_registers && a.rows > 0 && misgemm_workspace::get(stream, &partials, &counters)) {
            a.partials = partials;
        } else {
            // Before dx is written: it may be dy.
            hipLaunchKernelGGL((weight_grad<T>), dim3((unsigned)((a.cols + 63) / 64)), dim3(256), 0, stream, a);
            if (hipGetLastError() != hipSuccess) return MISGEMM_LAUNCH_FAILED;
        }
    }
    if (a.rows == 0) return MISGEMM_SUCCESS;
    if (!in_registers) {
        const dim3 grid((unsigned)(a.rows < (1 << 20) ? a.rows : 1 << 20));
        hipLaunchKernelGGL((rmsnorm_back_long<T, TW>), grid, dim3(64 * kMaxWaves), 0, stream, a);
        return launched();
    }
    a.groups = a.rows < 2 * kNumCus ? a.rows : 2 * kNumCus;
    const dim3 grid((unsigned)a.groups);
    if (a.cols <= 512)
        hipLaunchKernelGGL((rmsnorm_back<T, TW, 1, 1>), grid, dim3(64), 0, stream, a);
    else if (a.cols <= 2048)
        hipLaunchKernelGGL((rmsnorm_back<T, TW, 4, 1>), grid, dim3(256), 0, stream, a);
    else if (a.cols <= 8192)
        hipLaunchKernelGGL((rmsnorm_back<T, TW, 16, 1>), grid, dim3(1024), 0, stream, a);
    else
        hipLaunchKernelGGL((rmsnorm_back<T, TW, 16, 2>), grid, dim3(1024), 0, stream, a);
    if (hipGetLastError() != hipSuccess) return MISGEMM_LAUNCH_FAILED;
    if (a.partials == nullptr) return MISGEMM_SUCCESS;
    hipLaunchKernelGGL(sum_partials, dim3((unsigned)((a.cols + 31) / 32)), dim3(256), 0, stream, a);
    return launched();
}

}  // namespace

extern "C" int mi_rmsnorm(int type, int wtype, int rows, int cols, const void *x, int ldx, const void *residual,
                          int ldr, const void *weight, float eps, void *h, int ldh, void *y, int ldy, int ftype,
                          void *q, int ldq, float *scale, int lds, float *rstd, hipStream_t stream) {
    if (!is_real(type)) return MISGEMM_BAD_TYPE;
    if (wtype != type && wtype != MI_F32) return MISGEMM_BAD_TYPE;
    if (rows < 0) return MISGEMM_BAD_ROWS;
    if (cols < 0) return MISGEMM_BAD_COLS;
    const bool some = rows > 0 && cols > 0;
    if (some && x == nullptr) return MISGEMM_NULL_INPUT;
    if (ldx < cols) return MISGEMM_BAD_LD;
    if (residual != nullptr && ldr < cols) return MISGEMM_BAD_LD;
    if (some && weight == nullptr) return MISGEMM_NULL_INPUT;
    if (h != nullptr && ldh < cols) return MISGEMM_BAD_LD;
    if (y != nullptr && ldy < cols) return MISGEMM_BAD_LD;
    if (some && y == nullptr && q == nullptr) return MISGEMM_NULL_OUTPUT;
    if (q != nullptr) {
        if (!is_f8(ftype)) return MISGEMM_BAD_TYPE;
        if (ldq < cols) return MISGEMM_BAD_LD;
        if (some && scale == nullptr) return MISGEMM_NULL_SCALE;
        if (lds < rows) return MISGEMM_BAD_LDS;
    }
    if (!some) return MISGEMM_SUCCESS;

    NormArgs a;
    a.x = x;
    a.res = residual;
    a.weight = weight;
    a.h = h;
    a.y = y;
    a.q = static_cast<uint8_t *>(q);
    a.scale = scale;
    a.rstd = rstd;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldy = ldy;
    a.ldq = ldq;
    a.lds = lds;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    if (type == MI_F32) return launch_norm<float, float>(ftype, a, stream);
    if (type == MI_BF16)
        return wtype == MI_F32 ? launch_norm<bf16, float>(ftype, a, stream) : launch_norm<bf16, bf16>(ftype, a, stream);
    return wtype == MI_F32 ? launch_norm<f16, float>(ftype, a, stream) : launch_norm<f16, f16>(ftype, a, stream);
}

extern "C" int mi_rmsnorm_backward(int type, int wtype, int rows, int cols, const void *dy, int lddy, const void *h,
                                   int ldh, const void *weight, const float *rstd, const void *dh, int lddh, void *dx,
                                   int lddx, float beta, float *dweight, hipStream_t stream) {
    if (!is_real(type)) return MISGEMM_BAD_TYPE;
    if (wtype != type && wtype != MI_F32) return MISGEMM_BAD_TYPE;
    if (rows < 0) return MISGEMM_BAD_ROWS;
    if (cols < 0) return MISGEMM_BAD_COLS;
    const bool some = rows > 0 && cols > 0;
    if (some && dy == nullptr) return MISGEMM_NULL_INPUT;
    if (lddy < cols) return MISGEMM_BAD_LD;
    if (some && h == nullptr) return MISGEMM_NULL_INPUT;
    if (ldh < cols) return MISGEMM_BAD_LD;
    if (some && (weight == nullptr || rstd == nullptr)) return MISGEMM_NULL_INPUT;
    if (dh != nullptr && lddh < cols) return MISGEMM_BAD_LD;
    if (some && dx == nullptr) return MISGEMM_NULL_OUTPUT;
    if (lddx < cols) return MISGEMM_BAD_LD;
    if (cols == 0) return MISGEMM_SUCCESS;
    if (rows == 0 && (dweight == nullptr || beta == 1.0f)) return MISGEMM_SUCCESS;

    BackArgs a;
    a.dy = dy;
    a.h = h;
    a.weight = weight;
    a.dh = dh;
    a.rstd = rstd;
    a.dx = dx;
    a.dweight = dweight;
    a.partials = nullptr;
    a.lddy = lddy;
    a.ldh = ldh;
    a.lddh = lddh;
    a.lddx = lddx;
    a.rows = rows;
    a.cols = cols;
    a.groups = 0;
    a.beta = beta;
    if (type == MI_F32) return launch_back<float, float>(a, stream);
    if (type == MI_BF16) return wtype == MI_F32 ? launch_back<bf16, float>(a, stream) : launch_back<bf16, bf16>(a, stream);
    return wtype == MI_F32 ? launch_back<f16, float>(a, stream) : launch_back<f16, f16>(a, stream);
}
