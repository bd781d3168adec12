// What the kernels of the 8-bit linear layer share: element types, eight
// values at a time in and out of memory, block scales, reductions over lanes.
#ifndef MISGEMM_FP8_COMMON_H
#define MISGEMM_FP8_COMMON_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "misgemm_fp8.h"

namespace misgemm_fp8 {

using bf16 = __bf16;
using f16 = _Float16;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 128;                  // values that share a scale
constexpr float kTiny = 0x1p-100f;           // the least maximum a scale is made for

__host__ __device__ constexpr int blocks(int n) { return n / kBlock + (n % kBlock != 0); }

// The largest finite value of an 8-bit type.
template <int FMT> __device__ constexpr float top() { return FMT == MI_E4M3 ? 448.0f : 57344.0f; }

// N values of T as floats, or back, in accesses of up to 16 bytes at any
// alignment of T: gfx950 reads and writes wide words at any byte address.
// Values from `n` on are zero, and neither read nor written.
template <class T, int N> struct Values {
    typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};
template <class T, int N> __device__ __forceinline__ void load(const T *p, int n, float (&v)[N]) {
    if (n >= N) {
        const typename Values<T, N>::type w = *reinterpret_cast<const typename Values<T, N>::type *>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = static_cast<float>(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < n ? static_cast<float>(p[i]) : 0.0f;
    }
}
template <class T, int N> __device__ __forceinline__ void store(T *p, int n, const float (&v)[N]) {
    if (n >= N) {
        typename Values<T, N>::type w;
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = static_cast<T>(v[i]);
        *reinterpret_cast<typename Values<T, N>::type *>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = static_cast<T>(v[i]);
    }
}
template <class T> __device__ __forceinline__ void load8(const T *p, int n, float (&v)[8]) { load<T, 8>(p, n, v); }
template <class T> __device__ __forceinline__ void store8(T *p, int n, const float (&v)[8]) { store<T, 8>(p, n, v); }

// Eight values of T as they lie in memory, of which the first `n` of a row of
// `cols` values are wanted (others zero; n may be negative): one wide read
// without a branch, so that reads ahead of their use stay so. Where fewer than
// eight are left, the row's last eight are read and moved. `col` is where in
// the row; cols >= 8. EVEN: cols is a multiple of 8, so that n is 8 or none.
template <class T, bool EVEN> struct Eight {
    typedef typename Values<T, 8>::type type;
    typedef int words __attribute__((ext_vector_type(2 * sizeof(T))));
    type v;
    __device__ __forceinline__ void fetch(const T *row, int col, int cols) {
        v = *reinterpret_cast<const type *>(row + min(col, cols - 8));
    }
    // Down by BY values, where `over` has that bit.
    template <int BY> static __device__ __forceinline__ words moved(words w, int over) {
        constexpr int N = 2 * sizeof(T), STEP = BY * (int)sizeof(T) / 4;
        words m;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (STEP > 0)
                m[i] = i + STEP < N ? w[i + STEP < N ? i + STEP : 0] : 0;
            else
                m[i] = (int)((uint32_t)w[i] >> 16 | (i + 1 < N ? (uint32_t)w[i + 1 < N ? i + 1 : 0] << 16 : 0u));
        }
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = (over & BY) ? m[i] : w[i];
        return w;
    }
    // After `fetch`, at the first use.
    __device__ __forceinline__ void settle(int col, int cols) {
        const int over = max(col - (cols - 8), 0);   // col + 8 may pass 2^31
        words w = __builtin_bit_cast(words, v);
        if constexpr (EVEN) {
#pragma unroll
            for (unsigned i = 0; i < 2 * sizeof(T); ++i) w[i] = over > 0 ? 0 : w[i];
        } else {
            // No branch here either.
            w = moved<4>(w, over);
            w = moved<2>(w, over);
            w = moved<1>(w, over);
#pragma unroll
            for (unsigned i = 0; i < 2 * sizeof(T); ++i) w[i] = over >= 8 ? 0 : w[i];
        }
        v = __builtin_bit_cast(type, w);
    }
    // Has the values made into floats anew from here on, not kept as such.
    __device__ __forceinline__ void again() {
        words w = __builtin_bit_cast(words, v);
        asm("" : "+v"(w));
        v = __builtin_bit_cast(type, w);
    }
};

// Four floats to four 8-bit values, to nearest with ties to even. The values
// are at most the type's largest by their scale (x * (T/a) exceeds T by two
// roundings at most, which round back to T), so nothing saturates here.
template <int FMT> __device__ __forceinline__ int pack4(float a, float b, float c, float d) {
    int r = 0;
    if constexpr (FMT == MI_E4M3) {
        r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
        r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    } else {
        r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
        r = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
    }
    return r;
}

// N (8 or 16) bytes to memory at any address, the first `n` of them.
template <int N> __device__ __forceinline__ void store_bytes(uint8_t *p, int n, const int (&w)[N / 4]) {
    typedef int words __attribute__((ext_vector_type(N / 4), aligned(1)));
    if (n >= N) {
        words v;
#pragma unroll
        for (int i = 0; i < N / 4; ++i) v[i] = w[i];
        *reinterpret_cast<words *>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) p[i] = static_cast<uint8_t>(static_cast<unsigned>(w[i / 4]) >> (8 * (i % 4)));
    }
}

// Reductions over groups of 16, 32 or 64 neighbouring lanes, in every lane. In 16
// the partners come by rotations in the same instruction.
template <int BY> __device__ __forceinline__ float rotated16(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x120 + BY, 0xf, 0xf, false));
}
template <int WIDTH> __device__ __forceinline__ float max_over(float v) {
    static_assert(WIDTH == 16 || WIDTH == 64, "");
    v = fmaxf(v, rotated16<8>(v));
    v = fmaxf(v, rotated16<4>(v));
    v = fmaxf(v, rotated16<2>(v));
    v = fmaxf(v, rotated16<1>(v));
    if constexpr (WIDTH == 64) {
        v = fmaxf(v, __shfl_xor(v, 16));
        v = fmaxf(v, __shfl_xor(v, 32));
    }
    return v;
}
template <int WIDTH> __device__ __forceinline__ float sum_over(float v) {
    static_assert(WIDTH == 16 || WIDTH == 32 || WIDTH == 64, "");
    v += rotated16<8>(v);
    v += rotated16<4>(v);
    v += rotated16<2>(v);
    v += rotated16<1>(v);
    if constexpr (WIDTH >= 32) v += __shfl_xor(v, 16);
    if constexpr (WIDTH >= 64) v += __shfl_xor(v, 32);
    return v;
}
// The value of lane I of each 16.
template <int I> __device__ __forceinline__ float of16(float v) {
    return __builtin_bit_cast(float,
                              __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x150 + I, 0xf, 0xf, true));
}

inline bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline bool is_real(int t) { return t == MI_F32 || t == MI_BF16 || t == MI_F16; }
inline bool is_f8(int t) { return t == MI_E4M3 || t == MI_E5M2; }
inline int launched() { return hipGetLastError() == hipSuccess ? MISGEMM_SUCCESS : MISGEMM_LAUNCH_FAILED; }

}  // namespace misgemm_fp8

#endif  // MISGEMM_FP8_COMMON_H
