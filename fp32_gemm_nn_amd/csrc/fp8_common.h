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

// Reductions over groups of 16 or 64 neighbouring lanes, in every lane. In 16
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
__device__ __forceinline__ float sum_over64(float v) {
    v += rotated16<8>(v);
    v += rotated16<4>(v);
    v += rotated16<2>(v);
    v += rotated16<1>(v);
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
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
