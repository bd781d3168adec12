// Products of few rows in 16 bits, both operands with k running fastest,
// without a barrier in the sum: z = alpha A B^T + bias and what follows it.
//
// Bound by memory and its latency: B is read once and used for little
// arithmetic. A workgroup makes 16 MB x 16 NB outputs; its W waves take every
// W-th block of 64 values of k each and meet at one barrier, after which their
// sums are added in order of wave. A wave has D blocks of k on their way in
// registers. It reads them as whole rows of 128 bytes, eight to a load, and
// turns them into the matrix cores' operands (lane i of 16 holds row i) through
// LDS of its own, which needs no barrier. 1 x 4096 x 8192 takes 11.6 us (5.8
// TB/s) where 64 x 128 tiles take 17.2 with k in eight parts, 33 x 4096 x 4096 9.2
// us and 13.8, the gated 1 x 8192 x 4096 21.2 us (6.3 TB/s) and 26.8; with weights
// that the last level of cache does not hold, 13.4, 12.0 and 26.6 us.

#include <type_traits>

#include "linear.h"

namespace {

using namespace misgemm_linear;

template <class T> __device__ __forceinline__ f32x4 product(typename Vec<T>::x8 a, typename Vec<T>::x8 b, f32x4 c) {
    if constexpr (std::is_same<T, bf16>::value)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ i32x4 at(const void *base, uint32_t offset) {
    typedef int words __attribute__((ext_vector_type(4), aligned(2)));
    return *reinterpret_cast<const words *>(static_cast<const uint8_t *>(base) + offset);
}

// For K >= 8 and leading dimensions below 2^25 (32-bit offsets inside a tile).
// GATED: half of the NB sixteens are the first weight's rows and half the
// second's, of the same columns.
template <class T, int MB, int NB, int W, int D, bool GATED>
__global__ __launch_bounds__(64 * W) void lin_direct(LinArgs g) {
    constexpr int NH = GATED ? NB / 2 : NB, BM = 16 * MB, BN = 16 * NH, FRAGS = MB * NB;
    constexpr int LOADS = 2 * (MB + NB);   // eight rows each: A's, then B's
    static_assert(D == 1 || D == 2, "a wave that has fewer blocks takes them one at a time");
    static_assert(LOADS >= FRAGS, "a wave's sums fit its LDS");
    // A wave's rows of one block of k: chunk c of row r at position c ^ (r & 7),
    // so that the 16 rows an operand's read touches spread over all banks.
    __shared__ i32x4 lds[W][LOADS * 64];
    // The wave's number is the same in its lanes: known as such, its addresses
    // are a scalar base and 32-bit offsets.
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int i = lane % 16, grp = lane / 16;
    int tm, tn;
    tile_of(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN, ncol = n0 + grp * 4 * NH;

    // Rows past a matrix repeat its last one: their outputs are not stored.
    // Row 16 b + i of B's is column (i/4)*4*NH + 4*b + i%4, so that a lane's
    // outputs lie side by side.
    uint32_t at_row[LOADS];
    const uint8_t *A0 = static_cast<const uint8_t *>(g.A) + m0 * g.lda * 2;
    const uint8_t *B0 = static_cast<const uint8_t *>(g.B) + n0 * g.ldb * 2;
    const uint8_t *U0 = GATED ? static_cast<const uint8_t *>(g.U) + n0 * g.ldu * 2 : nullptr;
#pragma unroll
    for (int l = 0; l < 2 * MB; ++l) at_row[l] = min(8 * l + lane / 8, g.M - 1 - m0) * (uint32_t)g.lda * 2;
#pragma unroll
    for (int l = 0; l < 2 * NB; ++l) {
        const int r = 8 * (l % 2) + lane / 8, b = l / 2 % NH;
        at_row[2 * MB + l] = min((r / 4) * 4 * NH + 4 * b + r % 4, g.N - 1 - n0) *
                             (uint32_t)(l / 2 >= NH ? g.ldu : g.ldb) * 2;
    }
    const int c16 = 16 * ((lane % 8) ^ (lane / 8));   // this lane's chunk of its rows
    const long long bytes = 2LL * g.K;

    struct Block {
        i32x4 w[LOADS];
    };
    auto fetch = [&](Block &s, int kb) {
        // Hides that kb counts a loop: known as such, each load would get a
        // pointer of its own that runs with it, two registers a piece.
        asm("" : "+s"(kb));
        // A chunk that passes K is read as the last 16 bytes before K, and
        // moved when it is used. (The base is 16 bytes low to keep offsets positive.)
        const long long k = (long long)kb * 128 - 16;
        const uint32_t off = 16 + (uint32_t)min((long long)c16, bytes - 16 - kb * 128LL);
#pragma unroll
        for (int l = 0; l < LOADS; ++l)
            s.w[l] = at((l < 2 * MB ? A0 : l < 2 * (MB + NH) ? B0 : U0) + k, at_row[l] + off);
    };
    f32x4 acc[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto put = [&](Block &s, int kb) {
        if ((kb + 1) * 128LL > bytes) {
            const int over = (int)(kb * 128LL + c16 + 16 - bytes);
#pragma unroll
            for (int l = 0; l < LOADS; ++l) s.w[l] = shifted(s.w[l], over);
        }
#pragma unroll
        for (int l = 0; l < LOADS; ++l) lds[wave][64 * l + lane] = s.w[l];
        asm volatile("" ::: "memory");
    };
    auto add = [&] {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            using x8 = typename Vec<T>::x8;
            const i32x4 *from = lds[wave] + i * 8 + ((grp + 4 * s) ^ (i & 7));
            x8 fb[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) fb[b] = __builtin_bit_cast(x8, from[(MB + b) * 128]);
#pragma unroll
            for (int a = 0; a < MB; ++a) {
                const x8 fa = __builtin_bit_cast(x8, from[a * 128]);
#pragma unroll
                for (int b = 0; b < NB; ++b) acc[a][b] = product<T>(fb[b], fa, acc[a][b]);
            }
        }
        asm volatile("" ::: "memory");
    };

    // This wave's blocks are wave, wave + W, ...: n of them, at least DD.
    const int kblocks = (g.K + kStep - 1) / kStep, n = (kblocks - wave + W - 1) / W;
    // The loop's loads hang on no condition: where they do, the compiler has
    // to wait for all of them before it uses the first.
    auto run = [&](auto depth) {
        constexpr int DD = decltype(depth)::value;
        Block set[DD];
        auto step = [&](int d, int t, bool more) {
            put(set[d], wave + W * (t + d));
            if (more) fetch(set[d], wave + W * (t + DD + d));
            add();
        };
#pragma unroll
        for (int d = 0; d < DD; ++d) fetch(set[d], wave + W * d);
        int t = 0;
#pragma unroll 1
        for (; t + 2 * DD <= n; t += DD)
#pragma unroll
            for (int d = 0; d < DD; ++d) step(d, t, true);
#pragma unroll
        for (int d = 0; d < DD; ++d) step(d, t, t + DD + d < n);
        t += DD;
#pragma unroll
        for (int d = 0; d < DD - 1; ++d)
            if (t + d < n) step(d, t, false);
    };
    if (D >= 2 && n >= 2)
        run(std::integral_constant<int, D>{});
    else if (n >= 1)
        run(std::integral_constant<int, 1>{});

    f32x4 *sums = reinterpret_cast<f32x4 *>(lds[wave]);
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) sums[64 * (a * NB + b) + lane] = acc[a][b];
    __syncthreads();
    auto total = [&](int f, float (&v)[4], const void *bias, int n) {
        f32x4 sum = reinterpret_cast<const f32x4 *>(lds[0])[64 * f + lane];
#pragma unroll 5
        for (int w = 1; w < W; ++w) sum += reinterpret_cast<const f32x4 *>(lds[w])[64 * f + lane];
        float more[4];
        bias_at<T, 4>(bias, g.bias32, n, g.N - n, more);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(g.alpha, sum[j], more[j]);
    };
#pragma unroll
    for (int f0 = 0; f0 < MB * NH; f0 += W) {
        const int f = f0 + wave;
        if (MB * NH % W != 0 && f >= MB * NH) break;
        const int a = f / NH, b = f % NH, col = ncol + 4 * b;
        float v[4], u[4] = {};
        total(a * NB + b, v, g.bias, col);
        if constexpr (GATED) total(a * NB + NH + b, u, g.bias_u, col);
        const int m = m0 + 16 * a + i;
        if (m < g.M && col < g.N) put_out<T, GATED, 1, 4, false, false, false>(g, m, 0, col, v, u);
    }
}

template <class T, int MB, int NB, int W, int D, bool GATED> int launch_shape(LinArgs &g, hipStream_t stream) {
    constexpr int COLS = 16 * (GATED ? NB / 2 : NB);
    g.tiles_m = (g.M + 16 * MB - 1) / (16 * MB);
    g.tiles_n = (g.N + COLS - 1) / COLS;
    hipLaunchKernelGGL((lin_direct<T, MB, NB, W, D, GATED>), dim3((unsigned)(g.tiles_m * g.tiles_n)), dim3(64 * W), 0,
                       stream, g);
    return launched();
}

template <class T> int launch(bool gated, int shape, LinArgs &g, hipStream_t stream) {
    if (gated) {
        switch (shape) {
            case 0: return launch_shape<T, 1, 2, 16, 1, true>(g, stream);
            case 1: return launch_shape<T, 1, 2, 8, 2, true>(g, stream);
            case 2: return launch_shape<T, 1, 4, 8, 2, true>(g, stream);
            case 3: return launch_shape<T, 2, 2, 8, 2, true>(g, stream);
            default: return launch_shape<T, 4, 2, 4, 2, true>(g, stream);
        }
    }
    switch (shape) {
        case 0: return launch_shape<T, 1, 1, 16, 2, false>(g, stream);
        case 1: return launch_shape<T, 1, 2, 8, 2, false>(g, stream);
        case 2: return launch_shape<T, 2, 2, 8, 1, false>(g, stream);
        case 3: return launch_shape<T, 3, 1, 8, 2, false>(g, stream);
        default: return launch_shape<T, 4, 2, 4, 1, false>(g, stream);
    }
}

}  // namespace

int misgemm_linear::launch_direct(int type, bool gated, int shape, LinArgs &g, hipStream_t stream) {
    return type == MI_BF16 ? launch<bf16>(gated, shape, g, stream) : launch<f16>(gated, shape, g, stream);
}
