// mi_rmsnorm and mi_rmsnorm_backward: the root-mean-square norm of each row
// with the residual's addition and an 8-bit output, and its gradients.
//
// Both are bound by memory: every operand is read once and every output
// written once; a row stays in registers between its sum and its use. 8192 x
// 4096 in BF16: the norm with residual, h, y and 8 bits takes 60 us (5.0 TB/s),
// the gradients 54 us, of which 5 are the second launch for the sum of the
// partial ones (5.0 TB/s; 5.5 without it); a copy of 256 MiB reaches 5.4 TB/s
// here. One row of 4096 takes 3.1 us in a graph, of which a launch is 2 to 3,
// and 3.7 to 4.6 as a call, which is the host's time; 333 x 1300 in FP32 with
// the weight's gradient in the same launch 5.6 us.

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
    int rows, cols, turns;
    float eps;
};

// Sum over the NT threads of a row, in each of them, in a fixed order.
// `part` is not reused before another barrier.
template <int NT> __device__ __forceinline__ float row_sum(float v, float *part) {
    v = sum_over<(NT < 64 ? NT : 64)>(v);
    if constexpr (NT <= 64) {
        return v;
    } else {
        constexpr int W = NT / 64;
        if (threadIdx.x % 64 == 0) part[threadIdx.x / 64 % W] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w];
        return v;
    }
}

// y of eight values, y and q out. The 16 lanes that hold 128 columns share a scale.
template <class T, int FMT, bool EVEN>
__device__ __forceinline__ void norm_out(const NormArgs &a, long long row, int col, int n, const float (&h)[8],
                                         const float (&w)[8], float rstd) {
    float y[8], m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        y[j] = h[j] * rstd * w[j];
        m = fmaxf(m, fabsf(y[j]));
    }
    if (a.y != nullptr && n > 0) store8(static_cast<T *>(a.y) + row * a.ldy + col, EVEN ? 8 : n, y);
    if (a.q == nullptr) return;
    m = fmaxf(max_over<16>(m), kTiny);
    if (n <= 0) return;
    const float f = top<FMT>() / m;
    const int b[2] = {pack4<FMT>(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                      pack4<FMT>(y[4] * f, y[5] * f, y[6] * f, y[7] * f)};
    store_bytes<8>(a.q + row * a.ldq + col, EVEN ? 8 : n, b);
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

// NT threads take a row, PER eights of its columns each in registers, and a
// workgroup G rows at a time, `turns` times. The weight stays in registers
// (read for each row it would be a quarter of what a row moves), and the next
// row's x and residual are on their way while this one is reduced and written.
template <class T, class TW, int FMT, int NT, int G, int PER, bool EVEN>
__global__ __launch_bounds__(NT *G) void rmsnorm(NormArgs a) {
    // Two turns of partial sums: a wave still reading one row's is at most one
    // barrier behind the wave that writes the next row's.
    __shared__ float parts[2][G][NT > 64 ? NT / 64 : 1];
    const int tid = threadIdx.x % NT, group = threadIdx.x / NT;
    Eight<TW, EVEN> w[PER];
    Eight<T, EVEN> x[PER], r[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int col = (tid + NT * p) * 8;
        w[p].fetch(static_cast<const TW *>(a.weight), col, a.cols);
        w[p].settle(col, a.cols);
    }
    auto fetch = [&](long long row) {
        row = row < a.rows ? row : a.rows - 1;   // past the end: not used
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int col = (tid + NT * p) * 8;
            x[p].fetch(static_cast<const T *>(a.x) + row * a.ldx, col, a.cols);
            if (a.res != nullptr) r[p].fetch(static_cast<const T *>(a.res) + row * a.ldr, col, a.cols);
        }
    };
    long long row = blockIdx.x * (long long)G + group;
    fetch(row);
    for (int t = 0; t < a.turns; ++t) {
        float h[PER][8], sum = 0.0f;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            x[p].settle((tid + NT * p) * 8, a.cols);
            if (a.res != nullptr) r[p].settle((tid + NT * p) * 8, a.cols);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[p][j] = static_cast<float>(x[p].v[j]);
                // Rounded to T as it is kept.
                if (a.res != nullptr)
                    h[p][j] = static_cast<float>(static_cast<T>(h[p][j] + static_cast<float>(r[p].v[j])));
                sum = fmaf(h[p][j], h[p][j], sum);
            }
        }
        const long long next = row + (long long)gridDim.x * G;
        if (t + 1 < a.turns) fetch(next);
        const float rstd = 1.0f / sqrtf(row_sum<NT>(sum, parts[t & 1][group]) / a.cols + a.eps);
        if (row < a.rows) {
            if (a.rstd != nullptr && tid == 0) a.rstd[row] = rstd;
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                const int col = (tid + NT * p) * 8;
                if (a.h != nullptr && col < a.cols)
                    store8(static_cast<T *>(a.h) + row * a.ldh + col, EVEN ? 8 : a.cols - col, h[p]);
                float wf[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) wf[j] = static_cast<float>(w[p].v[j]);
                norm_out<T, FMT, EVEN>(a, row, col, a.cols - col, h[p], wf, rstd);
            }
        }
        row = next;
    }
}

// Rows too long for registers (or shorter than eight values): each is read twice.
template <class T, class TW, int FMT>
__global__ __launch_bounds__(64 * kMaxWaves) void rmsnorm_long(NormArgs a) {
    constexpr int NT = 64 * kMaxWaves;
    __shared__ float parts[2][kMaxWaves];
    const int tid = threadIdx.x;
    int turn = 0;
    for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        T *hout = a.h == nullptr ? nullptr : static_cast<T *>(a.h) + row * a.ldh;
        float sum = 0.0f;
        for (long long c = tid * 8; c < a.cols; c += NT * 8) {
            const int col = (int)c;
            float h[8];
            norm_in<T>(a, row, col, a.cols - col, h);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(h[j], h[j], sum);
        }
        const float rstd = 1.0f / sqrtf(row_sum<NT>(sum, parts[turn]) / a.cols + a.eps);
        if (a.rstd != nullptr && tid == 0) a.rstd[row] = rstd;
        // Each thread writes h where it alone reads x and the residual, after
        // it has read them: h may be either.
        for (long long c0 = 0; c0 < a.cols; c0 += NT * 8) {
            // Lanes past the row stay for the maximum over their 16, with nothing.
            const long long c = c0 + tid * 8;
            const int n = c < a.cols ? a.cols - (int)c : 0, col = c < a.cols ? (int)c : a.cols;
            float h[8], w[8];
            norm_in<T>(a, row, col, n, h);
            load8(static_cast<const TW *>(a.weight) + col, n, w);
            if (hout != nullptr && n > 0) store8(hout + col, n, h);
            norm_out<T, FMT, false>(a, row, col, n, h, w, rstd);
        }
    }
}

template <class T, class TW, int FMT, int NT, int G, int PER> int launch_rows(NormArgs a, hipStream_t stream) {
    // As many workgroups as the CUs hold at once (16 waves of them each, 24
    // where a thread has 8 columns), and as even a number of rows for each as
    // that allows.
    constexpr long long kPlaces = kNumCus * ((PER == 2 ? 1024 : 1536) / (NT * G));
    const long long sets = ((long long)a.rows + G - 1) / G;
    a.turns = (int)((sets + kPlaces - 1) / kPlaces);
    const dim3 grid((unsigned)((sets + a.turns - 1) / a.turns));
    if (a.cols % 8 == 0)
        hipLaunchKernelGGL((rmsnorm<T, TW, FMT, NT, G, PER, true>), grid, dim3(NT * G), 0, stream, a);
    else
        hipLaunchKernelGGL((rmsnorm<T, TW, FMT, NT, G, PER, false>), grid, dim3(NT * G), 0, stream, a);
    return launched();
}

template <class T, class TW, int FMT> int launch_norm(const NormArgs &a, hipStream_t stream) {
    if (a.cols >= 8 && a.cols <= 16384) {
        if (a.cols <= 128) return launch_rows<T, TW, FMT, 16, 16, 1>(a, stream);
        if (a.cols <= 256) return launch_rows<T, TW, FMT, 32, 8, 1>(a, stream);
        if (a.cols <= 512) return launch_rows<T, TW, FMT, 64, 4, 1>(a, stream);
        if (a.cols <= 1024) return launch_rows<T, TW, FMT, 128, 2, 1>(a, stream);
        if (a.cols <= 2048) return launch_rows<T, TW, FMT, 256, 1, 1>(a, stream);
        if (a.cols <= 4096) return launch_rows<T, TW, FMT, 256, 1, 2>(a, stream);
        if (a.cols <= 8192) return launch_rows<T, TW, FMT, 512, 1, 2>(a, stream);
        return launch_rows<T, TW, FMT, 1024, 1, 2>(a, stream);
    }
    // A grid of 2^20 workgroups stays within the 2^32 threads of a launch.
    const dim3 grid((unsigned)(a.rows < (1 << 20) ? a.rows : 1 << 20));
    hipLaunchKernelGGL((rmsnorm_long<T, TW, FMT>), grid, dim3(64 * kMaxWaves), 0, stream, a);
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
    int rows, cols, groups, turns;
    float beta;
};

// dx of the `n` columns (eight at most) of one row from `col` on.
template <class T>
__device__ __forceinline__ void back_out(const BackArgs &a, long long row, int col, int n, const float (&dy)[8],
                                         const float (&u)[8], const float (&w)[8], float rstd, float mean) {
    float dx[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dx[j] = rstd * (dy[j] * w[j] - u[j] * mean);
    if (a.dh != nullptr) {
        float r[8];
        load8(static_cast<const T *>(a.dh) + row * a.lddh + col, n, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) dx[j] += r[j];
    }
    store8(static_cast<T *>(a.dx) + row * a.lddx + col, n, dx);
}

// The weight's gradient of 64 columns from dy and h themselves, by NT threads:
// eight columns to a thread, NT / 8 rows at a time, whose sums are added in order.
template <class T, int NT> __device__ __forceinline__ void grad_columns(const BackArgs &a, int block) {
    constexpr int ROWS = NT / 8;
    __shared__ float part[ROWS][64];
    const int lane = threadIdx.x % 8, first = threadIdx.x / 8;
    const int col = block * 64 + lane * 8;
    float sum[8] = {};
    if (a.cols >= 8) {
        // Four rows at once, by every thread alike: past the end the last one's, for nothing.
        for (long long r0 = 0; r0 < a.rows; r0 += 4 * ROWS) {
            Eight<T, false> dy[4], h[4];
            float rstd[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long at = r0 + i * ROWS + first, row = at < a.rows ? at : a.rows - 1;
                dy[i].fetch(static_cast<const T *>(a.dy) + row * a.lddy, col, a.cols);
                h[i].fetch(static_cast<const T *>(a.h) + row * a.ldh, col, a.cols);
                rstd[i] = a.rstd[row];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dy[i].settle(col, a.cols);
                h[i].settle(col, a.cols);
                if (r0 + i * ROWS + first < a.rows) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sum[j] = fmaf(static_cast<float>(dy[i].v[j]), static_cast<float>(h[i].v[j]) * rstd[i], sum[j]);
                }
            }
        }
    } else {
        for (long long row = first; row < a.rows; row += ROWS) {
            float dy[8], h[8];
            load8(static_cast<const T *>(a.dy) + row * a.lddy + col, a.cols - col, dy);
            load8(static_cast<const T *>(a.h) + row * a.ldh + col, a.cols - col, h);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = fmaf(dy[j], h[j] * a.rstd[row], sum[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) part[first][lane * 8 + j] = sum[j];
    __syncthreads();
    // Eight threads add a column's sums of neighbouring rows each, then one theirs.
    const int c = threadIdx.x % 64, eighth = threadIdx.x / 64;
    static_assert(ROWS % (NT / 64) == 0 && NT / 64 >= 1, "");
    constexpr int EACH = ROWS / (NT / 64);
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < EACH; ++r) s += part[eighth * EACH + r][c];
    __syncthreads();
    part[eighth][c] = s;
    __syncthreads();
    if (eighth == 0 && block * 64 + c < a.cols) {
#pragma unroll
        for (int r = 1; r < NT / 64; ++r) s += part[r][c];
        float *dw = a.dweight + block * 64 + c;
        *dw = a.beta == 0.0f ? s : fmaf(a.beta, *dw, s);
    }
}

// NT threads take a row, PER eights of its columns each, and a workgroup G
// rows at a time, `turns` times; the next row's operands are on their way
// while this one is reduced and written. Each thread keeps its columns' share
// of the weight's gradient, and the workgroup writes one row of `partials`.
// AHEAD: there are registers for that.
template <class T, class TW, int NT, int G, int PER, bool EVEN, bool AHEAD>
__global__ __launch_bounds__(NT *G) void rmsnorm_back(BackArgs a) {
    // Workgroups past the rows', where there are some: the weight's gradient.
    if ((int)blockIdx.x >= a.groups) {
        grad_columns<T, NT * G>(a, blockIdx.x - a.groups);
        return;
    }
    // Two turns of sums: a wave still reading one row's is at most one
    // barrier behind the wave that writes the next row's.
    __shared__ float parts[2][G][NT > 64 ? NT / 64 : 1];
    __shared__ float shares[G > 1 ? G - 1 : 1][G > 1 ? NT * PER * 8 : 1];
    const int tid = threadIdx.x % NT, group = threadIdx.x / NT;
    Eight<TW, EVEN> wr[PER];
    Eight<T, EVEN> dyr[PER], hr[PER], dhr[PER];
    float dw[PER][8], rstd = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int col = (tid + NT * p) * 8;
        wr[p].fetch(static_cast<const TW *>(a.weight), col, a.cols);
        wr[p].settle(col, a.cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[p][j] = 0.0f;
    }
    auto fetch = [&](long long row) {
        row = row < a.rows ? row : a.rows - 1;   // past the end: not used
        rstd = a.rstd[row];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int col = (tid + NT * p) * 8;
            dyr[p].fetch(static_cast<const T *>(a.dy) + row * a.lddy, col, a.cols);
            hr[p].fetch(static_cast<const T *>(a.h) + row * a.ldh, col, a.cols);
            if (AHEAD && a.dh != nullptr) dhr[p].fetch(static_cast<const T *>(a.dh) + row * a.lddh, col, a.cols);
        }
    };
    long long row = blockIdx.x * (long long)G + group;
    if (AHEAD) fetch(row);
    for (int t = 0; t < a.turns; ++t) {
        if (!AHEAD) fetch(row);
        const bool live = row < a.rows;
        const float scale = rstd;
        float sum = 0.0f;
        Eight<T, EVEN> dy[PER], h[PER], dh[PER];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            dyr[p].settle((tid + NT * p) * 8, a.cols);
            hr[p].settle((tid + NT * p) * 8, a.cols);
            if (AHEAD && a.dh != nullptr) dhr[p].settle((tid + NT * p) * 8, a.cols);
            dy[p] = dyr[p];
            h[p] = hr[p];
            dh[p] = dhr[p];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sum = fmaf(static_cast<float>(dy[p].v[j]) * static_cast<float>(wr[p].v[j]),
                           static_cast<float>(h[p].v[j]) * scale, sum);
        }
        const long long next = row + (long long)a.groups * G;
        if (AHEAD && t + 1 < a.turns) fetch(next);
        const float mean = row_sum<NT>(sum, parts[t & 1][group]) / a.cols;
        if (live) {
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                const int col = (tid + NT * p) * 8;
                float dx[8];
                dy[p].again();
                if (!AHEAD && sizeof(T) == 4) {   // no registers for it: L2 has it still
                    h[p].fetch(static_cast<const T *>(a.h) + row * a.ldh, col, a.cols);
                    h[p].settle(col, a.cols);
                }
                h[p].again();
                if (!AHEAD && a.dh != nullptr) {
                    dh[p].fetch(static_cast<const T *>(a.dh) + row * a.lddh, col, a.cols);
                    dh[p].settle(col, a.cols);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = static_cast<float>(dy[p].v[j]), u = static_cast<float>(h[p].v[j]) * scale;
                    dx[j] = scale * (d * static_cast<float>(wr[p].v[j]) - u * mean);
                    if (a.dh != nullptr) dx[j] += static_cast<float>(dh[p].v[j]);
                    dw[p][j] = fmaf(d, u, dw[p][j]);
                }
                if (col < a.cols) store8(static_cast<T *>(a.dx) + row * a.lddx + col, EVEN ? 8 : a.cols - col, dx);
                if (!AHEAD) __builtin_amdgcn_sched_barrier(0);
            }
        }
        row = next;
    }
    if (a.partials == nullptr) return;
    if constexpr (G > 1) {
        if (group > 0)
#pragma unroll
            for (int p = 0; p < PER; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) shares[group - 1][(p * 8 + j) * NT + tid] = dw[p][j];
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int o = 0; o < G - 1; ++o)
#pragma unroll
            for (int p = 0; p < PER; ++p)
#pragma unroll
                for (int j = 0; j < 8; ++j) dw[p][j] += shares[o][(p * 8 + j) * NT + tid];
    }
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int col = (tid + NT * p) * 8;
        if (col < a.cols)
            store8(a.partials + (long long)blockIdx.x * a.cols + col, EVEN ? 8 : a.cols - col, dw[p]);
    }
}

// Rows too long for registers (or shorter than eight values): dx alone, each
// row read twice.
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
        const float mean = row_sum<NT>(sum, parts[turn]) / a.cols;
        for (long long c = threadIdx.x * 8; c < a.cols; c += NT * 8) {
            const int col = (int)c, n = a.cols - col;
            float dy[8], u[8], w[8];
            load8(static_cast<const T *>(a.dy) + row * a.lddy + col, n, dy);
            load8(static_cast<const T *>(a.h) + row * a.ldh + col, n, u);
            load8(static_cast<const TW *>(a.weight) + col, n, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] *= rstd;
            back_out<T>(a, row, col, n, dy, u, w, rstd, mean);
        }
    }
}

// The weight's gradient alone.
template <class T, int NT> __global__ __launch_bounds__(NT) void weight_grad(BackArgs a) {
    for (int block = blockIdx.x; block <= (a.cols - 1) / 64; block += gridDim.x) {
        grad_columns<T, NT>(a, block);
        __syncthreads();   // its sums are read before the next block's are written
    }
}

// Partial rows summed: 16 columns per workgroup, four to a thread, of which 64
// take every 64th row each; their sums are added in order.
__global__ __launch_bounds__(256) void sum_partials(BackArgs a) {
    __shared__ f32x4 part[64][4];
    const int lane = threadIdx.x % 4, turn = threadIdx.x / 4;
    const int col = blockIdx.x * 16 + lane * 4, n = a.cols - col;
    float sum[4] = {};
    if (n > 0) {
#pragma unroll 8
        for (int g = turn; g < a.groups; g += 64) {
            float v[4];
            load<float, 4>(a.partials + (long long)g * a.cols + col, n, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += v[j];
        }
    }
    part[turn][lane] = f32x4{sum[0], sum[1], sum[2], sum[3]};
    __syncthreads();
    for (int half = 32; half > 0; half /= 2) {
        if (turn < half) part[turn][lane] += part[turn + half][lane];
        __syncthreads();
    }
    if (turn == 0 && n > 0) {
        float v[4], old[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = part[0][lane][j];
        if (a.beta != 0.0f) {
            load<float, 4>(a.dweight + col, n, old);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = fmaf(a.beta, old[j], v[j]);
        }
        store<float, 4>(a.dweight + col, n, v);
    }
}

constexpr int kGroups = 2 * kNumCus;   // workgroups of the backward pass, and partial rows

// Threads to a row of the backward pass, and rows of a workgroup.
inline int back_threads(int cols) {
    int nt = 16;
    while (nt < 512 && nt * 8 < cols) nt *= 2;
    return cols > 8192 ? 1024 : nt;
}
inline int back_rows(int cols) { return cols > 8192 ? 1 : 512 / back_threads(cols); }

// Whether the weight's gradient is formed from dy and h by workgroups of its
// own, in the same launch, rather than from partial sums in a second one. The
// first costs 4.5 ns a row (its workgroups take all rows one after another),
// the second 2.6 us and the partial sums' way to memory and back at 2.4 TB/s:
// 600 x 4096 in BF16 take 9.1 and 13.9 us, 2000 x 512 take 13.0 and 7.0 us.
inline bool few_rows(const BackArgs &a) {
    const long long sets = ((long long)a.rows + back_rows(a.cols) - 1) / back_rows(a.cols);
    const long long groups = sets < kGroups ? sets : kGroups;
    return 4.5e-3 * a.rows < 2.6 + 8.0 * groups * a.cols / 2.4e6;
}

template <class T, class TW, int NT, int PER> int launch_back_rows(BackArgs a, hipStream_t stream) {
    constexpr int G = NT == 1024 ? 1 : 512 / NT;
    const long long sets = ((long long)a.rows + G - 1) / G;
    a.turns = (int)((sets + kGroups - 1) / kGroups);
    a.groups = (int)((sets + a.turns - 1) / a.turns);
    const bool own = a.dweight != nullptr && a.partials == nullptr;
    const dim3 grid((unsigned)(a.groups + (own ? (a.cols + 63) / 64 : 0)));
    constexpr bool AHEAD = NT * PER < 2048;
    if (a.cols % 8 == 0)
        hipLaunchKernelGGL((rmsnorm_back<T, TW, NT, G, PER, true, AHEAD>), grid, dim3(NT * G), 0, stream, a);
    else
        hipLaunchKernelGGL((rmsnorm_back<T, TW, NT, G, PER, false, AHEAD>), grid, dim3(NT * G), 0, stream, a);
    if (hipGetLastError() != hipSuccess) return MISGEMM_LAUNCH_FAILED;
    if (a.partials == nullptr) return MISGEMM_SUCCESS;
    hipLaunchKernelGGL(sum_partials, dim3((unsigned)((a.cols + 15) / 16)), dim3(256), 0, stream, a);
    return launched();
}

template <class T, class TW> int launch_back(BackArgs a, hipStream_t stream) {
    static_assert(size_t(kGroups) * 16384 <= misgemm_workspace::kFloats, "partial rows fit the workspace");
    const bool in_registers = a.cols >= 8 && a.cols <= 16384 && a.rows > 0;
    if (a.dweight != nullptr) {
        int *counters = nullptr;
        const bool partial = in_registers && !few_rows(a) && misgemm_workspace::get(stream, &a.partials, &counters);
        // Workgroups that read dy for the weight's gradient do not go with
        // others that write dx there: they come first then, with the same sums.
        if (!partial && (!in_registers || a.dx == a.dy)) {
            // As for the rows, at most 2^20 workgroups.
            const int blocks64 = (a.cols - 1) / 64 + 1;
            const dim3 grid((unsigned)(blocks64 < (1 << 20) ? blocks64 : 1 << 20));
            if (a.cols > 8192)
                hipLaunchKernelGGL((weight_grad<T, 1024>), grid, dim3(1024), 0, stream, a);
            else
                hipLaunchKernelGGL((weight_grad<T, 512>), grid, dim3(512), 0, stream, a);
            if (hipGetLastError() != hipSuccess) return MISGEMM_LAUNCH_FAILED;
            a.dweight = nullptr;
        }
    }
    if (a.rows == 0) return MISGEMM_SUCCESS;
    if (!in_registers) {
        const dim3 grid((unsigned)(a.rows < (1 << 20) ? a.rows : 1 << 20));
        hipLaunchKernelGGL((rmsnorm_back_long<T, TW>), grid, dim3(64 * kMaxWaves), 0, stream, a);
        return launched();
    }
    switch (back_threads(a.cols)) {
        case 16: return launch_back_rows<T, TW, 16, 1>(a, stream);
        case 32: return launch_back_rows<T, TW, 32, 1>(a, stream);
        case 64: return launch_back_rows<T, TW, 64, 1>(a, stream);
        case 128: return launch_back_rows<T, TW, 128, 1>(a, stream);
        case 256: return launch_back_rows<T, TW, 256, 1>(a, stream);
        case 512:
            return a.cols <= 4096 ? launch_back_rows<T, TW, 512, 1>(a, stream)
                                  : launch_back_rows<T, TW, 512, 2>(a, stream);
        default: return launch_back_rows<T, TW, 1024, 2>(a, stream);
    }
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
    a.turns = 0;
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
    a.groups = a.turns = 0;
    a.beta = beta;
    if (type == MI_F32) return launch_back<float, float>(a, stream);
    if (type == MI_BF16) return wtype == MI_F32 ? launch_back<bf16, float>(a, stream) : launch_back<bf16, bf16>(a, stream);
    return wtype == MI_F32 ? launch_back<f16, float>(a, stream) : launch_back<f16, f16>(a, stream);
}
