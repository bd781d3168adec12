// mi_rmsnorm and mi_rmsnorm_backward: the root-mean-square norm of each row
// with the residual's addition and an 8-bit output, and its gradients.
//
// Both are bound by memory: every operand is read once and every output
// written once; a row stays in registers between its sum and its use. 8192 x
// 4096 in BF16: the norm with residual, h, y and 8 bits takes 59 us (5.1 TB/s),
// the gradients 50 us (5.4 TB/s) and 5 us for the sum of the partial ones; a
// copy of 256 MiB reaches 5.4 TB/s here. One row of 4096 takes 3.6 us, of
// which a launch is 2 to 3.

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

// Eight values of T as they lie in memory, fetched a row ahead of their use.
// EVEN: the row's length is a multiple of 8, so that there are eight or none.
template <class T, bool EVEN> struct Raw {
    typename Values<T, 8>::type v;
    // Has the values made into floats anew from here on, not kept as such.
    __device__ __forceinline__ void again() {
        typedef int words __attribute__((ext_vector_type(2 * sizeof(T))));
        words w = __builtin_bit_cast(words, v);
        asm("" : "+v"(w));
        v = __builtin_bit_cast(typename Values<T, 8>::type, w);
    }
    __device__ __forceinline__ void fetch(const T *p, int n) {
        if (EVEN ? n > 0 : n >= 8) {
            v = *reinterpret_cast<const typename Values<T, 8>::type *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = static_cast<T>(0.0f);
                if constexpr (!EVEN)
                    if (i < n) v[i] = p[i];
            }
        }
    }
};

// Sum over the W waves of a row, in each of its threads, in a fixed order.
// `part` is not reused before another barrier.
template <int W> __device__ __forceinline__ float row_sum(float v, float *part) {
    v = sum_over64(v);
    if constexpr (W == 1) return v;
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64 % W] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w];
    return v;
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

// W waves take a row, PER eights of its columns per thread in registers, and a
// workgroup G rows at a time, `turns` times. The weight stays in registers
// (read for each row it would be a quarter of what a row moves), and the next
// row's x and residual are on their way while this one is reduced and written.
template <class T, class TW, int FMT, int W, int G, int PER, bool EVEN>
__global__ __launch_bounds__(64 * W * G) void rmsnorm(NormArgs a) {
    constexpr int NT = 64 * W;
    // Two turns of partial sums: a wave still reading one row's is at most one
    // barrier behind the wave that writes the next row's.
    __shared__ float parts[2][G][W];
    const int tid = threadIdx.x % NT, group = threadIdx.x / NT;
    Raw<TW, EVEN> w[PER];
    Raw<T, EVEN> x[PER], r[PER];
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int col = (tid + NT * p) * 8;
        w[p].fetch(static_cast<const TW *>(a.weight) + col, a.cols - col);
    }
    auto fetch = [&](long long row) {
        row = row < a.rows ? row : a.rows - 1;   // past the end: not used
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int col = (tid + NT * p) * 8;
            x[p].fetch(static_cast<const T *>(a.x) + row * a.ldx + col, a.cols - col);
            if (a.res != nullptr) r[p].fetch(static_cast<const T *>(a.res) + row * a.ldr + col, a.cols - col);
        }
    };
    long long row = blockIdx.x * (long long)G + group;
    fetch(row);
    for (int t = 0; t < a.turns; ++t) {
        float h[PER][8], sum = 0.0f;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[p][j] = static_cast<float>(x[p].v[j]);
                // Rounded to T as it is kept.
                if (a.res != nullptr) h[p][j] = static_cast<float>(static_cast<T>(h[p][j] + static_cast<float>(r[p].v[j])));
                sum = fmaf(h[p][j], h[p][j], sum);
            }
        }
        const long long next = row + (long long)gridDim.x * G;
        if (t + 1 < a.turns) fetch(next);
        const float rstd = 1.0f / sqrtf(row_sum<W>(sum, parts[t & 1][group]) / a.cols + a.eps);
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

// Rows too long for registers: each is read twice.
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
        const float rstd = 1.0f / sqrtf(row_sum<kMaxWaves>(sum, parts[turn]) / a.cols + a.eps);
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

template <class T, class TW, int FMT, int W, int G, int PER> int launch_rows(NormArgs a, hipStream_t stream) {
    // As many workgroups as the CUs hold at once (16 waves of them each, 24
    // where a thread has 8 columns), and as even a number of rows for each as
    // that allows.
    constexpr long long kPlaces = kNumCus * ((PER == 2 ? 16 : 24) / (W * G));
    const long long sets = ((long long)a.rows + G - 1) / G;
    a.turns = (int)((sets + kPlaces - 1) / kPlaces);
    const dim3 grid((unsigned)((sets + a.turns - 1) / a.turns));
    if (a.cols % 8 == 0)
        hipLaunchKernelGGL((rmsnorm<T, TW, FMT, W, G, PER, true>), grid, dim3(64 * W * G), 0, stream, a);
    else
        hipLaunchKernelGGL((rmsnorm<T, TW, FMT, W, G, PER, false>), grid, dim3(64 * W * G), 0, stream, a);
    return launched();
}

template <class T, class TW, int FMT> int launch_norm(const NormArgs &a, hipStream_t stream) {
    if (a.cols <= 512) return launch_rows<T, TW, FMT, 1, 4, 1>(a, stream);
    if (a.cols <= 1024) return launch_rows<T, TW, FMT, 2, 2, 1>(a, stream);
    if (a.cols <= 2048) return launch_rows<T, TW, FMT, 4, 1, 1>(a, stream);
    if (a.cols <= 4096) return launch_rows<T, TW, FMT, 4, 1, 2>(a, stream);
    if (a.cols <= 8192) return launch_rows<T, TW, FMT, 8, 1, 2>(a, stream);
    if (a.cols <= 16384) return launch_rows<T, TW, FMT, 16, 1, 2>(a, stream);
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

// W waves take a row, PER eights of its columns per thread, and a workgroup G
// rows at a time, `turns` times; the next row's operands are on their way
// while this one is reduced and written. Each thread keeps its columns' share
// of the weight's gradient, and the workgroup writes one row of `partials`.
// AHEAD: there are registers for that.
template <class T, class TW, int W, int G, int PER, bool EVEN, bool AHEAD>
__global__ __launch_bounds__(64 * W * G) void rmsnorm_back(BackArgs a) {
    constexpr int NT = 64 * W;
    // Two turns of sums: a wave still reading one row's is at most one
    // barrier behind the wave that writes the next row's.
    __shared__ float parts[2][G][W];
    __shared__ float shares[G > 1 ? G - 1 : 1][G > 1 ? NT * PER * 8 : 1];
    const int tid = threadIdx.x % NT, group = threadIdx.x / NT;
    Raw<TW, EVEN> wr[PER];
    Raw<T, EVEN> dyr[PER], hr[PER], dhr[PER];
    float dw[PER][8], rstd = 0.0f;
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int col = (tid + NT * p) * 8;
        wr[p].fetch(static_cast<const TW *>(a.weight) + col, a.cols - col);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[p][j] = 0.0f;
    }
    auto fetch = [&](long long row) {
        row = row < a.rows ? row : a.rows - 1;   // past the end: not used
        rstd = a.rstd[row];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int col = (tid + NT * p) * 8, n = a.cols - col;
            dyr[p].fetch(static_cast<const T *>(a.dy) + row * a.lddy + col, n);
            hr[p].fetch(static_cast<const T *>(a.h) + row * a.ldh + col, n);
            if (AHEAD && a.dh != nullptr) dhr[p].fetch(static_cast<const T *>(a.dh) + row * a.lddh + col, n);
        }
    };
    long long row = blockIdx.x * (long long)G + group;
    if (AHEAD) fetch(row);
    for (int t = 0; t < a.turns; ++t) {
        if (!AHEAD) fetch(row);
        const bool live = row < a.rows;
        const float scale = rstd;
        float sum = 0.0f;
        Raw<T, EVEN> dy[PER], h[PER], dh[PER];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
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
        const float mean = row_sum<W>(sum, parts[t & 1][group]) / a.cols;
        if (live) {
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                const int col = (tid + NT * p) * 8;
                float dx[8];
                dy[p].again();
                if (!AHEAD && sizeof(T) == 4)   // no registers for it: L2 has it still
                    h[p].fetch(static_cast<const T *>(a.h) + row * a.ldh + col, a.cols - col);
                h[p].again();
                if (!AHEAD && a.dh != nullptr)
                    dh[p].fetch(static_cast<const T *>(a.dh) + row * a.lddh + col, a.cols - col);
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
        const float mean = row_sum<kMaxWaves>(sum, parts[turn]) / a.cols;
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

template <class T, class TW, int W, int G, int PER> int launch_back_rows(BackArgs a, hipStream_t stream) {
    const long long sets = ((long long)a.rows + G - 1) / G;
    a.turns = (int)((sets + kGroups - 1) / kGroups);
    a.groups = (int)((sets + a.turns - 1) / a.turns);
    if (a.cols % 8 == 0)
        hipLaunchKernelGGL((rmsnorm_back<T, TW, W, G, PER, true, W * PER < 32>), dim3(a.groups), dim3(64 * W * G), 0, stream, a);
    else
        hipLaunchKernelGGL((rmsnorm_back<T, TW, W, G, PER, false, W * PER < 32>), dim3(a.groups), dim3(64 * W * G), 0, stream, a);
    if (hipGetLastError() != hipSuccess) return MISGEMM_LAUNCH_FAILED;
    if (a.partials == nullptr) return MISGEMM_SUCCESS;
    hipLaunchKernelGGL(sum_partials, dim3((unsigned)((a.cols + 15) / 16)), dim3(256), 0, stream, a);
    return launched();
}

template <class T, class TW> int launch_back(BackArgs a, hipStream_t stream) {
    const bool in_registers = a.cols <= 16384;
    if (a.dweight != nullptr) {
        float *partials = nullptr;
        int *counters = nullptr;
        static_assert(size_t(kGroups) * 16384 <= misgemm_workspace::kFloats, "partial rows fit the workspace");
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
    if (a.cols <= 512) return launch_back_rows<T, TW, 1, 8, 1>(a, stream);
    if (a.cols <= 1024) return launch_back_rows<T, TW, 2, 4, 1>(a, stream);
    if (a.cols <= 2048) return launch_back_rows<T, TW, 4, 2, 1>(a, stream);
    if (a.cols <= 4096) return launch_back_rows<T, TW, 8, 1, 1>(a, stream);
    if (a.cols <= 8192) return launch_back_rows<T, TW, 8, 1, 2>(a, stream);
    return launch_back_rows<T, TW, 16, 1, 2>(a, stream);
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
