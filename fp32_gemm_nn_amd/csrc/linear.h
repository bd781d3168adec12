// What the kernels of the 16-bit feed-forward block share: arguments,
// activations, and the way from sums to outputs. The mathematics is described
// in linear.hip.
#ifndef MISGEMM_LINEAR_KERNELS_H
#define MISGEMM_LINEAR_KERNELS_H

#include "fp8_gemm.h"
#include "misgemm_linear.h"

namespace misgemm_linear {

using namespace misgemm_fp8;

constexpr int kStep = 64;   // values of k to a block: 128 bytes

template <class T> struct Vec {
    typedef T x8 __attribute__((ext_vector_type(8)));
};

struct LinArgs {
    const void *A, *B, *U;        // U: the gated block's second weight, beside B
    const void *bias, *bias_u, *R;
    void *C, *z, *zu;             // z: NULL where it is not kept
    float *zs, *zus, *ws;
    int *counters;
    long long lda, ldb, ldu, ldr, ldc, ldz, ldzu, lds, ldsu;
    int M, N, K;
    int tiles_m, tiles_n, splits, kb_per_split;
    float alpha, beta;
    int act, ztype;
    bool bias32, c32;             // FP32 rather than the operands' type
    bool direct;                  // whole aligned 16 bytes everywhere: copied to LDS without registers
    bool near;                    // 32-bit offsets inside a tile, and rows of eight values at least
};

// f in few instructions: an epilogue forms 128 of them a lane while the matrix
// cores wait, and v_exp_f32 and v_rcp_f32 take as long as four others. Their
// steps of a result's last place are the least error there is; e^x as 2^(x / ln 2)
// is off by |x| of them at most. Where z is infinite a factor that would make
// NaN of the other's 0 is held at 104, beyond which f and f' are at their limits
// (v_med3_f32 drops NaN, so the other factor has to carry it).
constexpr float kLog2E = 1.44269504f;
__device__ __forceinline__ float above(float z) { return __builtin_amdgcn_fmed3f(z, -104.0f, __builtin_inff()); }
__device__ __forceinline__ float within(float z) { return __builtin_amdgcn_fmed3f(z, -104.0f, 104.0f); }

// 1 / (1 + e^-z).
__device__ __forceinline__ float sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -kLog2E));
}
// gelu_tanh is z * sigmoid(p), p = 2 sqrt(2/pi) (z + 0.044715 z^3): (1 + tanh x) / 2 without its cancellation.
constexpr float kGelu1 = 1.59576912f, kGelu3 = 0.0713548163f;
__device__ __forceinline__ float gelu_sigmoid(float z) {
    const float t = z * fmaf(-kGelu3 * kLog2E, z * z, -kGelu1 * kLog2E);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}
// The normal distribution's integral up to -|z|, and its density without the
// factor 1 / sqrt(2 pi): e^(-z^2/2) times a polynomial in t = 1 / (1 + 0.34 |z|),
// fitted to least relative error over |z| <= 14.5 (6.0e-8, at 0, as FP32 holds
// the coefficients). In FP32 it is off by 5 steps of 2^-24 below |z| = 1, by 10
// at 3, 32 at 6 and 126 at 13, where the rounding of z^2 counts. 1 + erf would
// cancel; erfcf takes five times as long.
__device__ __forceinline__ float tail(float z, float &density) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.34f, fabsf(z), 1.0f));
    density = __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2E));
    float p = -0.02587636187672615f;
    p = fmaf(p, t, 0.1383567452430725f);
    p = fmaf(p, t, -0.2708704173564911f);
    p = fmaf(p, t, 0.1997169554233551f);
    p = fmaf(p, t, -0.043105896562337875f);
    p = fmaf(p, t, 0.11471346020698547f);
    p = fmaf(p, t, 0.11535173654556274f);
    p = fmaf(p, t, 0.13609223067760468f);
    p = fmaf(p, t, 0.135621577501297f);
    return p * t * density;
}

// f(z).
template <int ACT> __device__ __forceinline__ float act_of(float z) {
    if constexpr (ACT == MI_ACT_RELU) return z <= 0.0f ? 0.0f : z;
    if constexpr (ACT == MI_ACT_SILU) return above(z) * sigmoid(z);
    if constexpr (ACT == MI_ACT_GELU) {
        // z (1 - tail) above 0 and z tail below it.
        float density;
        const float h = tail(z, density);
        return fmaf(-fminf(fabsf(z), 104.0f), h, fmaxf(z, 0.0f));
    }
    if constexpr (ACT == MI_ACT_GELU_TANH) return above(z) * gelu_sigmoid(z);
    return z;
}
// f(z) and f'(z).
template <int ACT> __device__ __forceinline__ void act_both(float z, float &f, float &df) {
    if constexpr (ACT == MI_ACT_RELU) {
        f = act_of<ACT>(z);
        df = z <= 0.0f ? 0.0f : z > 0.0f ? 1.0f : z;
    } else if constexpr (ACT == MI_ACT_SILU) {
        const float s = sigmoid(z);
        f = above(z) * s;
        df = s * fmaf(within(z), 1.0f - s, 1.0f);
    } else if constexpr (ACT == MI_ACT_GELU) {
        float density;
        const float h = tail(z, density), c = within(z);
        f = fmaf(-fabsf(c), h, fmaxf(z, 0.0f));
        df = fmaf(c * 0.398942280f, density, z > 0.0f ? 1.0f - h : h);
    } else if constexpr (ACT == MI_ACT_GELU_TANH) {
        const float c = within(z), s = gelu_sigmoid(z);
        f = above(z) * s;
        df = fmaf(c * fmaf(3.0f * kGelu3, c * c, kGelu1), s * (1.0f - s), s);
    } else {
        f = z;
        df = 1.0f;
    }
}
// v <- f(v), the activation chosen once for all N.
template <int N> __device__ __forceinline__ void activate(int act, float (&v)[N]) {
    auto all = [&](auto f) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = f(v[j]);
    };
    switch (act) {
        case MI_ACT_RELU: return all([](float z) { return act_of<MI_ACT_RELU>(z); });
        case MI_ACT_SILU: return all([](float z) { return act_of<MI_ACT_SILU>(z); });
        case MI_ACT_GELU: return all([](float z) { return act_of<MI_ACT_GELU>(z); });
        case MI_ACT_GELU_TANH: return all([](float z) { return act_of<MI_ACT_GELU_TANH>(z); });
        default: return;
    }
}

// N neighbouring values of the bias, zero without one and past the row.
template <class T, int N> __device__ __forceinline__ void bias_at(const void *bias, bool f32, int n, int left, float (&v)[N]) {
    if (bias == nullptr) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = 0.0f;
    } else if (f32) {
        load<float, N>(static_cast<const float *>(bias) + n, left, v);
    } else {
        load<T, N>(static_cast<const T *>(bias) + n, left, v);
    }
}

// N values or bytes to memory, past L2 where they STREAM: a large product's
// outputs would push out operands that neighbours read (8192 x 8192 x 4096 with
// an 8-bit checkpoint 430 us, 445 through L2; gated with two 834 and 860, but 915
// where the checkpoints' pieces of 32 bytes pass it too: those L2 has to join).
template <class CT, int N, bool STREAM> __device__ __forceinline__ void put(CT *p, int left, const float (&v)[N]) {
    if (STREAM && left >= N) {
        typedef typename Values<CT, N>::type type;
        type w;
#pragma unroll
        for (int j = 0; j < N; ++j) w[j] = static_cast<CT>(v[j]);
        __builtin_nontemporal_store(w, reinterpret_cast<type *>(p));
    } else {
        store<CT, N>(p, left, v);
    }
}
// `apart`: the second four bytes go 32 columns on.
template <bool STREAM> __device__ __forceinline__ void put_bytes(uint8_t *p, int left, const int (&w)[2], bool apart) {
    typedef int words __attribute__((ext_vector_type(2), aligned(1)));
    if (apart) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k % 4 + 32 * (k / 4) < left)
                p[k % 4 + 32 * (k / 4)] = static_cast<uint8_t>(static_cast<unsigned>(w[k / 4]) >> (8 * (k % 4)));
        return;
    }
    if (STREAM && left >= 8)
        __builtin_nontemporal_store(words{w[0], w[1]}, reinterpret_cast<words *>(p));
    else
        store_bytes<8>(p, left, w);
}

// R rows, `step` apart from row m on, of PER pieces of N neighbouring values
// each, 32 columns apart from column n on (n < N): z (unless it has 8 bits), then
// f(z) + beta R. R may be C: a value is read by the thread that writes it. WHOLE:
// all of them are in the matrix.
template <class CT, int R, int PER, int N, bool WHOLE, bool STREAM>
__device__ __forceinline__ void put_linear(const LinArgs &g, int m, int step, int n, float (&v)[R * PER * N]) {
    auto each = [&](void *base, long long ld, auto f) {
        CT *p = static_cast<CT *>(base) + m * ld + n;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int left = WHOLE ? N : g.N - n - 32 * k;
                if (WHOLE || (m + r * step < g.M && left > 0))
                    f(p + r * (step * ld) + 32 * k, left, *reinterpret_cast<float(*)[N]>(v + (r * PER + k) * N));
            }
    };
    auto write = [&](CT *p, int left, float (&x)[N]) { put<CT, N, STREAM>(p, left, x); };
    if (g.z != nullptr && g.zs == nullptr) each(g.z, g.ldz, write);
    activate<R * PER * N>(g.act, v);
    if (g.beta != 0.0f)
        each(const_cast<void *>(g.R), g.ldr, [&](const CT *p, int left, float (&x)[N]) {
            float old[N];
            load<CT, N>(p, left, old);
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = fmaf(g.beta, old[j], x[j]);
        });
    each(g.C, g.ldc, write);
}
// The gated block's: v is g and then h, u is u.
template <class CT, int R, int N, bool WHOLE, bool STREAM>
__device__ __forceinline__ void put_gated(const LinArgs &g, int m, int step, int n, float (&v)[R * N],
                                          float (&u)[R * N]) {
    const int left = WHOLE ? N : g.N - n;
    auto write = [&](void *base, long long ld, float (&x)[R * N]) {
        CT *p = static_cast<CT *>(base) + m * ld + n;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (WHOLE || m + r * step < g.M)
                put<CT, N, STREAM>(p + r * (step * ld), left, *reinterpret_cast<float(*)[N]>(x + r * N));
    };
    if (g.z != nullptr && g.zs == nullptr) {
        write(g.z, g.ldz, v);
        write(g.zu, g.ldzu, u);
    }
    activate<R * N>(g.act, v);
#pragma unroll
    for (int j = 0; j < R * N; ++j) v[j] *= u[j];
    write(g.C, g.ldc, v);
}
// PIECES: of FP32 (and not gated) each eight values are two pieces of four.
template <class T, bool GATED, int R, int N, bool WHOLE, bool STREAM, bool PIECES>
__device__ __forceinline__ void put_out(const LinArgs &g, int m, int step, int n, float (&v)[R * N],
                                        float (&u)[R * N]) {
    if constexpr (GATED) {
        if (g.c32)
            put_gated<float, R, N, WHOLE, STREAM>(g, m, step, n, v, u);
        else
            put_gated<T, R, N, WHOLE, STREAM>(g, m, step, n, v, u);
    } else {
        constexpr int PER = PIECES ? 2 : 1;
        if (g.c32)
            put_linear<float, R, PER, N / PER, WHOLE, STREAM>(g, m, step, n, v);
        else
            put_linear<T, R, 1, N, WHOLE, STREAM>(g, m, step, n, v);
    }
}

// Whether a stream's workspace has room for `parts` parts of each of `tiles`
// tiles of `floats` sums. Asked before a plan is chosen, not after: a plan that
// is then run whole is another than the one that was weighed (448 x 4288 x 16384
// with rows 2 bytes aligned: 293 us in 68 tiles of 256 x 128, 151 as it is chosen).
inline bool parts_fit(long long tiles, int parts, int floats) {
    return tiles <= misgemm_workspace::kCounters && tiles * parts * floats <= (long long)misgemm_workspace::kFloats;
}

inline bool is_half(int t) { return t == MI_BF16 || t == MI_F16; }

// Tiles that go through LDS (linear_tile.h, a file for each type), and
// products of few rows without a barrier in their sum (linear_direct.hip).
// `shape` names one of their tile shapes.
int launch_tiles_bf16(bool gated, bool ta, bool tb, int shape, LinArgs &g, hipStream_t stream);
int launch_tiles_f16(bool gated, bool ta, bool tb, int shape, LinArgs &g, hipStream_t stream);
int launch_direct(int type, bool gated, int shape, LinArgs &g, hipStream_t stream);

}  // namespace misgemm_linear

#endif  // MISGEMM_LINEAR_KERNELS_H
