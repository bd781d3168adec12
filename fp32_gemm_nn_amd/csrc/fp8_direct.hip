// Products of few outputs: C = alpha * A * B^T + beta * C as in fp8_gemm.hip,
// without a barrier in the sum.
//
// Bound by memory and its latency: where A has few rows, B is read once and
// used for little arithmetic. A workgroup makes 16 MB x 16 NB outputs; its W
// waves take every W-th block of k each and meet at one barrier, after which
// their sums are added in order of wave. A wave has D blocks of k on their way
// in registers. It reads them as whole rows of 128 bytes, eight to a load, and
// turns them into the matrix cores' operands (lane i of 16 holds row i) through
// LDS of its own, which needs no barrier. (Loads straight into operands have
// neighbouring lanes in different rows, and brought 13 bytes per clock and CU
// where these bring up to 38.) 1 x 4096 x 4096 takes 5.3 us, 8192 x 8192 with
// one row 11.5 us (5.8 TB/s); 64 x 4096 x 4096 6.4 us, 512 x 2048 x 2048 8.2 us,
// where 128 x 128 tiles through LDS take 16.7, 24, 17.7 and 14.1 us (calls one
// after another; in a graph each is 0.1 to 0.6 us longer).

#include <type_traits>

#include "fp8_gemm.h"

namespace {

using namespace misgemm_fp8;

template <class T> __device__ __forceinline__ T at(const void *base, uint32_t offset) {
    return *reinterpret_cast<const T *>(static_cast<const uint8_t *>(base) + offset);
}

template <int FMT, bool EXACT> __device__ __forceinline__ Operand<EXACT> operand(i32x4 lo, i32x4 hi) {
    Operand<EXACT> o;
    if constexpr (EXACT) {
        o.v[0] = widen<FMT>(lo[0], lo[1]);
        o.v[1] = widen<FMT>(lo[2], lo[3]);
        o.v[2] = widen<FMT>(hi[0], hi[1]);
        o.v[3] = widen<FMT>(hi[2], hi[3]);
    } else {
        o.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return o;
}

// For K >= 16 and leading dimensions below 2^26 (32-bit offsets inside a tile).
template <int MB, int NB, int W, int D, int FA, int FB, bool ROWB, bool EXACT>
__global__ __launch_bounds__(64 * W) void fp8_direct(GemmArgs g) {
    constexpr int BM = 16 * MB, BN = 16 * NB, FRAGS = MB * NB;
    constexpr int SB = ROWB ? 4 * NB : 1;
    constexpr int LOADS = 2 * (MB + NB);   // eight rows each: A's, then B's
    static_assert(D == 1 || D == 2, "a wave that has fewer blocks takes them one at a time");
    static_assert(kBlock % BN == 0, "a tile's columns share a block");
    static_assert(LOADS >= FRAGS, "a wave's sums fit its LDS");
    // A wave's rows of one block of k: chunk c of row r at position c ^ (r & 7),
    // so that the 16 rows a fragment read touches spread over all banks.
    __shared__ i32x4 lds[W][LOADS * 64];
    // The wave's number is the same in its lanes: known as such, its addresses
    // are a scalar base and 32-bit offsets.
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int i = lane % 16, grp = lane / 16;
    int tm, tn;
    tile_of(blockIdx.x, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN, ncol = n0 + grp * 4 * NB;

    // Rows past a matrix repeat its last one: their outputs are not stored.
    // Row 16 b + i of B's is column (i/4)*4*NB + 4*b + i%4, so that a lane's
    // outputs lie side by side.
    uint32_t at_row[LOADS], at_sa[MB], at_sb[SB];
    const uint8_t *A0 = g.A + m0 * g.lda, *B0 = g.B + n0 * g.ldb;
#pragma unroll
    for (int l = 0; l < 2 * MB; ++l) at_row[l] = min(8 * l + lane / 8, g.M - 1 - m0) * (uint32_t)g.lda;
#pragma unroll
    for (int l = 0; l < 2 * NB; ++l) {
        const int r = 8 * (l % 2) + lane / 8;
        at_row[2 * MB + l] = min((r / 4) * 4 * NB + 4 * (l / 2) + r % 4, g.N - 1 - n0) * (uint32_t)g.ldb;
    }
#pragma unroll
    for (int a = 0; a < MB; ++a) at_sa[a] = 4 * min(16 * a + i, g.M - 1 - m0);
#pragma unroll
    for (int b = 0; b < SB; ++b) at_sb[b] = ROWB ? 4 * min(grp * 4 * NB + b, g.N - 1 - n0) : 0;
    const int c16 = 16 * ((lane % 8) ^ (lane / 8));   // this lane's chunk of its rows

    struct Block {
        i32x4 w[LOADS];
        float fa[MB], fb[SB];
    };
    auto fetch = [&](Block &s, int kb) {
        // Hides that kb counts a loop: known as such, each load would get a
        // pointer of its own that runs with it, two registers a piece.
        asm("" : "+s"(kb));
        // A chunk that passes K is read as the last 16 bytes before K, and
        // moved when it is used. (The base is 16 bytes low to keep offsets positive.)
        const long long k = (long long)kb * kBlock - 16;
        const uint32_t off = 16 + min(c16, g.K - 16 - kb * kBlock);
#pragma unroll
        for (int l = 0; l < LOADS; ++l) s.w[l] = at<words16>((l < 2 * MB ? A0 : B0) + k, at_row[l] + off);
        const float *sa = g.sa + kb * g.ldsa + m0;
        const float *sb = ROWB ? g.sb + kb * g.ldsb + n0 : g.sb + n0 / kBlock * g.ldsb + kb;
#pragma unroll
        for (int a = 0; a < MB; ++a) s.fa[a] = at<float>(sa, at_sa[a]);
#pragma unroll
        for (int b = 0; b < SB; ++b) s.fb[b] = at<float>(sb, at_sb[b]);
    };
    f32x4 acc[MB][NB];
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto put = [&](Block &s, int kb) {
        if ((kb + 1) * kBlock > g.K) {
            const int over = kb * kBlock + c16 + 16 - g.K;
#pragma unroll
            for (int l = 0; l < LOADS; ++l) s.w[l] = shifted(s.w[l], over);
        }
#pragma unroll
        for (int l = 0; l < LOADS; ++l) lds[wave][64 * l + lane] = s.w[l];
        asm volatile("" ::: "memory");
    };
    auto add = [&](const float (&sa)[MB], const float (&sb)[SB]) {
        const i32x4 *from = lds[wave] + i * 8 + (grp ^ (i & 7));
        const i32x4 *with = lds[wave] + i * 8 + (grp ^ 4 ^ (i & 7));
        Operand<EXACT> fb[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
            fb[b] = operand<FB, EXACT>(from[(MB + b) * 128], with[(MB + b) * 128]);
#pragma unroll
        for (int a = 0; a < MB; ++a) {
            // Without it the scheduler widens several rows ahead, beyond the registers.
            if constexpr (EXACT) __builtin_amdgcn_sched_barrier(0);
            const Operand<EXACT> fa = operand<FA, EXACT>(from[a * 128], with[a * 128]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const f32x4 p = product<FB, FA, EXACT>(fb[b], fa);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[a][b][j] = fmaf(p[j], sa[a] * sb[ROWB ? 4 * b + j : 0], acc[a][b][j]);
            }
        }
        asm volatile("" ::: "memory");
    };

    // This wave's blocks are wave, wave + W, ...: n of them, at least DD.
    const int kblocks = blocks(g.K), n = (kblocks - wave + W - 1) / W;
    // The loop's loads hang on no condition: where they do, the compiler has
    // to wait for all of them before it uses the first.
    auto run = [&](auto depth) {
        constexpr int DD = decltype(depth)::value;
        Block set[DD];
        auto step = [&](int d, int t, bool more) {
            Block &s = set[d];
            put(s, wave + W * (t + d));
            float sa[MB], sb[SB];
#pragma unroll
            for (int a = 0; a < MB; ++a) sa[a] = s.fa[a];
#pragma unroll
            for (int b = 0; b < SB; ++b) sb[b] = s.fb[b];
            if (more) fetch(s, wave + W * (t + DD + d));
            add(sa, sb);
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
#pragma unroll
    for (int f0 = 0; f0 < FRAGS; f0 += W) {
        const int f = f0 + wave;
        if (FRAGS % W != 0 && f >= FRAGS) break;
        f32x4 sum = reinterpret_cast<const f32x4 *>(lds[0])[64 * f + lane];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += reinterpret_cast<const f32x4 *>(lds[w])[64 * f + lane];
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = g.alpha * sum[j];
        put_row<EXACT, 4>(g, m0 + 16 * (f / NB) + i, ncol + 4 * (f % NB), v);
    }
}

template <int MB, int NB, int W, int D, int FA, int FB, bool ROWB, bool EXACT>
int launch_shape(GemmArgs &g, hipStream_t stream) {
    g.tiles_m = (g.M + 16 * MB - 1) / (16 * MB);
    g.tiles_n = (g.N + 16 * NB - 1) / (16 * NB);
    hipLaunchKernelGGL((fp8_direct<MB, NB, W, D, FA, FB, ROWB, EXACT>), dim3((unsigned)(g.tiles_m * g.tiles_n)),
                       dim3(64 * W), 0, stream, g);
    return launched();
}

template <int FA, int FB, bool ROWB, bool EXACT> int launch(int shape, GemmArgs &g, hipStream_t stream) {
    switch (shape) {
        case 0: return launch_shape<1, 1, 16, 2, FA, FB, ROWB, EXACT>(g, stream);
        case 1: return launch_shape<1, 2, 8, 2, FA, FB, ROWB, EXACT>(g, stream);
        case 2: return launch_shape<2, 2, 8, 1, FA, FB, ROWB, EXACT>(g, stream);
        case 3: return launch_shape<4, 2, 8, 1, FA, FB, ROWB, EXACT>(g, stream);
        case 4: return launch_shape<4, 2, 4, 1, FA, FB, ROWB, EXACT>(g, stream);
        default:
            // Widened operands, or a scale for each column, do not fit the registers there.
            if constexpr (!EXACT && !ROWB) return launch_shape<4, 4, 8, 1, FA, FB, ROWB, EXACT>(g, stream);
            return MISGEMM_LAUNCH_FAILED;
    }
}

template <int FA, int FB> int launch(bool rows, int shape, GemmArgs &g, hipStream_t stream) {
    if (g.ctype == MI_F32)
        return rows ? launch<FA, FB, true, true>(shape, g, stream) : launch<FA, FB, false, true>(shape, g, stream);
    return rows ? launch<FA, FB, true, false>(shape, g, stream) : launch<FA, FB, false, false>(shape, g, stream);
}

}  // namespace

int misgemm_fp8::launch_direct(int atype, int btype, bool rows, int shape, GemmArgs &g, hipStream_t stream) {
    if (atype == MI_E4M3)
        return btype == MI_E4M3 ? launch<MI_E4M3, MI_E4M3>(rows, shape, g, stream)
                                : launch<MI_E4M3, MI_E5M2>(rows, shape, g, stream);
    return btype == MI_E4M3 ? launch<MI_E5M2, MI_E4M3>(rows, shape, g, stream)
                            : launch<MI_E5M2, MI_E5M2>(rows, shape, g, stream);
}
