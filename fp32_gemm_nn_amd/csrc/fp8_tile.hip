// Products of many outputs: C = alpha * A * B^T + beta * C as in fp8_gemm.hip,
// in tiles of BM x BN outputs whose operands go through LDS.
//
// Two buffers hold a block of k each. While the products of one are formed the
// other fills, by loads that go to LDS without registers; the waves meet once
// a block, one row of products before its end, when what they read of it is in
// registers: the next block's operands and the loads of the one after it start
// behind those products. B's operands of a block stay in registers, A's pass
// by, and each product is scaled into the sums while the next ones run.
//
// 256 x 256 tiles on eight waves (128 x 64 each, 128 registers of sums) halve
// what 128 x 128 tiles read from L2 and LDS: 8192 x 8192 x 4096 to BF16 takes
// 244 us (2.25 PFLOP/s) in the former and 292 us in the latter, two workgroups
// of which share a CU; with a scale for each row of B, whose product with A's
// differs at every output, 286 and 324 us. Below 256 tiles of 256 x 256 CUs
// stay empty, and the smaller ones win (2048 x 4096 x 1024: 14.5 us and 19.7
// us); 64 x 128 tiles fill the gap to fp8_direct.hip (331 x 5752 x 352 with row
// scales: 6.7 us, 7.3 in tiles of 128 x 128, 10.2 there). Both sides of these
// are calls one after another on one card; cards and runs differ by 6%. What
// bounds the large one: the matrix cores are busy 52 to 57% of the time; the
// operands' way from L2 to LDS alone took 220 us (measured with the products
// left out), the products alone 217 us, where the whole took 241. FP32 results
// (BF16 products, half the rate) are nearer to the matrix cores: 4096 x 4096 x
// 8192 takes 248 us (1.11 PFLOP/s) with a scale for each block of B and 267 us
// with one for each row.

#include "fp8_gemm.h"

namespace {

using namespace misgemm_fp8;

// BYTES (16 or 4) a lane from base + offset to LDS, 64 lanes' side by side
// from `lds` on. In assembly, since the compiler would have every later read
// of LDS wait for it: the reads here are of another buffer until `meet`. It
// writes no register.
template <int BYTES> __device__ __forceinline__ void load_lds(const void *base, uint32_t offset, const uint8_t *lds) {
    const uint32_t to =
        (uint32_t)reinterpret_cast<size_t>((const __attribute__((address_space(3))) uint8_t *)lds);
    if constexpr (BYTES == 16)
        asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" :: "{m0}"(to), "v"(offset), "s"(base) : "memory");
    else
        asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, %2" :: "{m0}"(to), "v"(offset), "s"(base) : "memory");
}

// One operand's 128 bytes of k for ROWS rows in LDS: rows of eight 16-byte
// chunks, chunk c of row r at position c ^ swz(r), so that the 16 rows a
// fragment read touches spread over all banks. Rows past the matrix repeat its
// last one: their outputs are not stored.
template <int ROWS, int NT> struct Stage {
    static constexpr int PER = ROWS * 8 / NT;
    static_assert(PER * NT == ROWS * 8 && NT % 64 == 0, "whole chunks per thread");
    static __device__ __forceinline__ int swz(int r) { return r & 7; }
    static __device__ __forceinline__ int row(int tid, int j) { return tid / 8 + NT / 8 * j; }
    static __device__ __forceinline__ int chunk(int tid, int j) { return tid % 8 ^ swz(row(tid, j)); }

    // Offsets of a thread's chunks in a block of k, for leading dimensions below 2^24.
    static __device__ __forceinline__ void offsets(uint32_t (&at)[PER], int ld, int rows, int tid) {
#pragma unroll
        for (int j = 0; j < PER; ++j) at[j] = min(row(tid, j), rows - 1) * (uint32_t)ld + 16 * chunk(tid, j);
    }
    // A whole block of k of 16-byte aligned rows, without registers; `lds` is where the wave's first 1024 bytes go.
    static __device__ __forceinline__ void copy(const uint8_t *src, const uint32_t (&at)[PER], uint8_t *lds) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            load_lds<16>(src, at[j], lds + 16 * NT * j);
    }
    // The same of any block and alignment, in two steps, for leading dimensions
    // below 2^24. A chunk that passes K (K >= 16) is read as the 16 bytes before
    // K and moved on its way to LDS. `at` are offsets of whole rows; `src` is 16
    // bytes low, to keep offsets positive.
    static __device__ __forceinline__ void rows_at(uint32_t (&at)[PER], int ld, int rows, int tid) {
#pragma unroll
        for (int j = 0; j < PER; ++j) at[j] = min(row(tid, j), rows - 1) * (uint32_t)ld;
    }
    static __device__ __forceinline__ void fetch_near(i32x4 (&w)[PER], const uint8_t *src, const uint32_t (&at)[PER],
                                                      int left, int tid) {
        static_assert(NT / 8 % 8 == 0, "a thread's chunks are in one place of their rows");
        const uint32_t off = 16 + min(16 * chunk(tid, 0), left - 16);
#pragma unroll
        for (int j = 0; j < PER; ++j)
            w[j] = *reinterpret_cast<const words16 *>(src - 16 + (at[j] + off));
    }
    // The same for any leading dimension. A chunk that passes K (K >= 16) is
    // read as the 16 bytes before K and moved on its way to LDS.
    static __device__ __forceinline__ void fetch(i32x4 (&w)[PER], const uint8_t *src, long long ld, int rows, int k0,
                                                 int K, int tid) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            w[j] = *reinterpret_cast<const words16 *>(src + min(row(tid, j), rows - 1) * ld +
                                                      min(k0 + 16 * chunk(tid, j), K - 16));
    }
    static __device__ __forceinline__ void settle(i32x4 (&w)[PER], int k0, int K, int tid) {
        if (k0 + kBlock > K) {
#pragma unroll
            for (int j = 0; j < PER; ++j) w[j] = shifted(w[j], k0 + 16 * chunk(tid, j) + 16 - K);
        }
    }
    static __device__ __forceinline__ void write(const i32x4 (&w)[PER], int tid, uint8_t *lds) {
#pragma unroll
        for (int j = 0; j < PER; ++j) *reinterpret_cast<i32x4 *>(lds + 16 * (tid + NT * j)) = w[j];
    }
};

// The 16-byte chunks at `at` and four chunks further of a row in LDS.
__device__ __forceinline__ i32x8 raw(const uint8_t *lds, int at) {
    const i32x4 lo = *reinterpret_cast<const i32x4 *>(lds + at);
    const i32x4 hi = *reinterpret_cast<const i32x4 *>(lds + (at ^ 64));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int FMT, bool EXACT> __device__ __forceinline__ Operand<EXACT> operand(i32x8 w) {
    Operand<EXACT> o;
    if constexpr (EXACT) {
#pragma unroll
        for (int s = 0; s < 4; ++s) o.v[s] = widen<FMT>(w[2 * s], w[2 * s + 1]);
    } else {
        o.v = w;
    }
    return o;
}

// The waves of a workgroup meet, with all they have read and written in LDS
// done, and all they load to LDS landed.
__device__ __forceinline__ void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

enum Way { DIRECT, STAGED, FAR };   // operands to LDS: without registers, through them, with any leading dimension

template <int BM, int BN, int WM, int WN, int FA, int FB, bool ROWB, bool EXACT, Way WAY>
__global__ __launch_bounds__(64 * WM * WN, WAY == FAR && EXACT && ROWB ? 1 : 2) void fp8_tile(GemmArgs g) {
    constexpr bool ANY = WAY != DIRECT;
    constexpr int NT = 64 * WM * WN, TM = BM / WM, TN = BN / WN, MI = TM / 16, NI = TN / 16;
    constexpr int ROWS = MI < 4 ? MI : 4;   // sixteens of rows that leave at a time
    static_assert(TN == 64 && MI % ROWS == 0, "a wave's columns share a block, and leave as whole rows");
    using StageA = Stage<BM, NT>;
    using StageB = Stage<BN, NT>;
    constexpr int OPERANDS = (BM + BN) * kBlock, SB = ROWB ? 4 * NI : 1;
    // Behind the operands A's scales and B's: of each row, or of each block of 128.
    constexpr int BYTES = OPERANDS + 4 * (BM + (ROWB ? BN : 64));
    __shared__ __align__(16) uint8_t lds[2][BYTES];
    __shared__ int is_last;
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int i = lane % 16, grp = lane / 16;
    const int wm = wave / WN, wn = wave % WN;

    int tm, tn;
    const int tiles = g.tiles_m * g.tiles_n;
    const int split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles;
    tile_of(tile, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int kb0 = split * g.kb_per_split, kb1 = min(blocks(g.K), kb0 + g.kb_per_split);
    const uint8_t *A0 = g.A + m0 * g.lda, *B0 = g.B + n0 * g.ldb;

    const int row_a = wm * TM + i, row_b = wn * TN + i;
    const int at_a = row_a * kBlock + 16 * (grp ^ StageA::swz(row_a));
    const int at_b = BM * kBlock + row_b * kBlock + 16 * (grp ^ StageB::swz(row_b));
    const int at_sa = OPERANDS + 4 * row_a;
    const int at_sb = OPERANDS + 4 * BM + (ROWB ? 4 * (wn * TN + 4 * grp) : 4 * (wn * TN / kBlock));

    // Scales to LDS, 64 to a wave.
    constexpr int PARTS = BM / 64 + (ROWB ? BN / 64 : 1);
    uint32_t at_scale[(PARTS + WM * WN - 1) / (WM * WN)];
#pragma unroll
    for (int p0 = 0; p0 < PARTS; p0 += WM * WN) {
        const int p = p0 + wave, r = 64 * p + lane;
        at_scale[p0 / (WM * WN)] =
            p < BM / 64 ? 4 * min(r, g.M - 1 - m0)
            : ROWB      ? 4 * min(r - BM, g.N - 1 - n0)
                        : 4 * (uint32_t)g.ldsb * min(lane % ((BN + kBlock - 1) / kBlock), (g.N - 1 - n0) / kBlock);
    }
    auto copy_scales = [&](int kb, uint8_t *to) {
        const float *sa = g.sa + kb * g.ldsa + m0;
        const float *sb = ROWB ? g.sb + kb * g.ldsb + n0 : g.sb + n0 / kBlock * g.ldsb + kb;
#pragma unroll
        for (int p0 = 0; p0 < PARTS; p0 += WM * WN) {
            const int p = p0 + wave;
            if (p < PARTS)
                load_lds<4>(p < BM / 64 ? sa : sb, at_scale[p0 / (WM * WN)], to + OPERANDS + 256 * p);
        }
    };

    uint32_t from_a[StageA::PER], from_b[StageB::PER];
    if constexpr (WAY == DIRECT) {
        StageA::offsets(from_a, (int)g.lda, g.M - m0, tid);
        StageB::offsets(from_b, (int)g.ldb, g.N - n0, tid);
    } else if constexpr (WAY == STAGED) {
        StageA::rows_at(from_a, (int)g.lda, g.M - m0, tid);
        StageB::rows_at(from_b, (int)g.ldb, g.N - n0, tid);
    }
    auto copy = [&](int kb, int buf) {
        // Hides that kb counts a loop: known as such, each load would get a
        // pointer of its own that runs with it, two registers a piece.
        asm("" : "+s"(kb));
        StageA::copy(A0 + (long long)kb * kBlock, from_a, lds[buf] + 1024 * wave);
        StageB::copy(B0 + (long long)kb * kBlock, from_b, lds[buf] + BM * kBlock + 1024 * wave);
        copy_scales(kb, lds[buf]);
    };
    struct Chunks {
        i32x4 a[StageA::PER], b[StageB::PER];
    };
    auto fetch = [&](Chunks &w, int kb) {
        asm("" : "+s"(kb));
        if constexpr (WAY == STAGED) {
            StageA::fetch_near(w.a, A0 + (long long)kb * kBlock, from_a, g.K - kb * kBlock, tid);
            StageB::fetch_near(w.b, B0 + (long long)kb * kBlock, from_b, g.K - kb * kBlock, tid);
            return;
        }
        StageA::fetch(w.a, A0, g.lda, g.M - m0, kb * kBlock, g.K, tid);
        StageB::fetch(w.b, B0, g.ldb, g.N - n0, kb * kBlock, g.K, tid);
    };
    auto write = [&](Chunks &w, int kb, int buf) {
        StageA::settle(w.a, kb * kBlock, g.K, tid);
        StageB::settle(w.b, kb * kBlock, g.K, tid);
        StageA::write(w.a, tid, lds[buf]);
        StageB::write(w.b, tid, lds[buf] + BM * kBlock);
        copy_scales(kb, lds[buf]);
    };

    f32x4 acc[MI][NI];
#pragma unroll
    for (int a = 0; a < MI; ++a)
#pragma unroll
        for (int b = 0; b < NI; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    Operand<EXACT> fb[NI];
    float sb[SB], sa;
    i32x8 wa;
    auto read_fb = [&](int buf, int b) { fb[b] = operand<FB, EXACT>(raw(lds[buf], at_b + b * 16 * kBlock)); };
    auto read_sb = [&](int buf) {
#pragma unroll
        for (int b = 0; b < NI; ++b) {
            if constexpr (ROWB) {
                const f32x4 s = *reinterpret_cast<const f32x4 *>(lds[buf] + at_sb + 64 * b);
#pragma unroll
                for (int j = 0; j < 4; ++j) sb[4 * b + j] = s[j];
            }
        }
        if constexpr (!ROWB) sb[0] = *reinterpret_cast<const float *>(lds[buf] + at_sb);
    };
    auto read_a = [&](int buf, int a) {
        wa = raw(lds[buf], at_a + a * 16 * kBlock);
        sa = *reinterpret_cast<const float *>(lds[buf] + at_sa + 64 * a);
    };
    // The products of one block of k. `turn` comes when all that this wave
    // reads of the block is in registers, with a row of products left to hide
    // what it does. A product is scaled and added after the next row's are
    // issued, one by one in its place: the matrix cores have its result by then.
    auto multiply = [&](int buf, bool more, auto turn) {
        f32x4 p[NI];
        float f = 0.0f;
#pragma unroll
        for (int a = 0; a <= MI; ++a) {
            Operand<EXACT> fa;
            const float s = sa;
            if (a < MI) fa = operand<FA, EXACT>(wa);
            if (a + 1 < MI)
                read_a(buf, a + 1);
            else if (a + 1 == MI)
                turn();
#pragma unroll
            for (int b = 0; b < NI; ++b) {
                if (a > 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[a - 1][b][j] = fmaf(p[b][j], ROWB ? f * sb[4 * b + j] : f, acc[a - 1][b][j]);
                    // Keeps the sums here: moved past the branches of `turn`, they
                    // would leave a block's products waiting in registers.
                    asm volatile("" : "+v"(acc[a - 1][b]));
                }
                if (a < MI) p[b] = product<FB, FA, EXACT>(fb[b], fa);
                // Their last use (not so where they would be widened here and now).
                if (a + 1 == MI && more && !EXACT) read_fb(buf ^ 1, b);
                __builtin_amdgcn_sched_barrier(0);
            }
            f = ROWB ? s : s * sb[0];
        }
        if (more) {
            read_sb(buf ^ 1);
#pragma unroll
            for (int b = 0; b < NI && EXACT; ++b) read_fb(buf ^ 1, b);
        }
    };
    auto begin = [&] {
        read_sb(0);
#pragma unroll
        for (int b = 0; b < NI; ++b) read_fb(0, b);
        read_a(0, 0);
    };

    const int last = ANY ? kb1 : min(kb1, g.K / kBlock);   // the blocks that the loop takes
    if (kb0 < last) {
        Chunks w;
        if constexpr (ANY) {
            fetch(w, kb0);
            write(w, kb0, 0);
            if (kb0 + 1 < last) fetch(w, kb0 + 1);
        } else {
            copy(kb0, 0);
        }
        meet();
        if constexpr (ANY) {
            if (kb0 + 1 < last) write(w, kb0 + 1, 1);
        } else {
            if (kb0 + 1 < last) copy(kb0 + 1, 1);
        }
        begin();
#pragma unroll 1
        for (int kb = kb0; kb < last; ++kb) {
            const int buf = (kb - kb0) & 1;
            if constexpr (ANY) {
                if (kb + 2 < last) fetch(w, kb + 2);
            }
            // The next block's operands come from the buffer that `meet` opens
            // (after the last block they are not used).
            multiply(buf, true, [&] {
                meet();
                if constexpr (ANY) {
                    if (kb + 2 < last) write(w, kb + 2, buf);
                } else {
                    if (kb + 2 < last) copy(kb + 2, buf);
                }
                read_a(buf ^ 1, 0);
            });
        }
    }
    if constexpr (!ANY) {
        if (last < kb1) {   // the last block of k, where it is short
            Chunks w;
            fetch(w, last);
            meet();
            write(w, last, 0);
            meet();
            begin();
            multiply(0, false, [] {});
        }
    }

    if (g.splits > 1) {
        // Partial tiles go to the workspace, written and read past the XCDs'
        // own caches; the last workgroup of a tile adds them in split order.
        constexpr int PART = BM * BN;
        float *part = g.ws + ((size_t)tile * g.splits) * PART + (size_t)wave * (MI * NI * 4 * 64) + lane;
#pragma unroll
        for (int a = 0; a < MI; ++a)
#pragma unroll
            for (int b = 0; b < NI; ++b)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    __hip_atomic_store(part + (size_t)split * PART + ((a * NI + b) * 4 + j) * 64, acc[a][b][j],
                                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (tid == 0)
            is_last = __hip_atomic_fetch_add(&g.counters[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                      g.splits - 1;
        __syncthreads();
        if (!is_last) return;
        if (tid == 0) __hip_atomic_store(&g.counters[tile], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int a = 0; a < MI; ++a)
#pragma unroll
            for (int b = 0; b < NI; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < g.splits; ++s)
#pragma unroll
            for (int a = 0; a < MI; ++a)
#pragma unroll
                for (int b = 0; b < NI; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[a][b][j] += __hip_atomic_load(part + (size_t)s * PART + ((a * NI + b) * 4 + j) * 64,
                                                          __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }

    // A lane holds four neighbouring outputs of a row; stored like that, 16
    // rows at once, they would leave in pieces of 16 bytes. So up to 64 x 64
    // outputs at a time turn in LDS, each wave's in its own, and leave as whole rows.
    // Chunk c of row r is at c ^ (r & 15).
    meet();
    f32x4 *own = reinterpret_cast<f32x4 *>(lds) + wave * ROWS * 256;
    const int m1 = m0 + wm * TM, n1 = n0 + wn * TN;
#pragma unroll
    for (int a0 = 0; a0 < MI; a0 += ROWS) {
#pragma unroll
        for (int a = 0; a < ROWS; ++a)
#pragma unroll
            for (int b = 0; b < NI; ++b) own[(16 * a + i) * 16 + ((4 * b + grp) ^ i)] = acc[a0 + a][b];
        asm volatile("" ::: "memory");
        constexpr int N = EXACT ? 4 : 8, LANES = 64 / N;   // outputs of a lane, lanes of a row
#pragma unroll 4
        for (int r0 = 0; r0 < 16 * ROWS; r0 += 64 / LANES) {
            const int r = r0 + lane / LANES, c = lane % LANES * (N / 4);
            float v[N];
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                const f32x4 w = own[r * 16 + ((c + h) ^ (r & 15))];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * h + j] = g.alpha * w[j];
            }
            put_row<EXACT, N>(g, m1 + 16 * a0 + r, n1 + 4 * c, v);
        }
        asm volatile("" ::: "memory");
    }
}

template <int BM, int BN, int WM, int WN, int FA, int FB, bool ROWB, bool EXACT, Way WAY>
int launch_tile(GemmArgs &g, bool split, hipStream_t stream) {
    g.tiles_m = (g.M + BM - 1) / BM;
    g.tiles_n = (g.N + BN - 1) / BN;
    const int kblocks = blocks(g.K);
    const long long tiles = (long long)g.tiles_m * g.tiles_n;
    g.splits = split ? splits_of(tiles, kblocks) : 1;
    static_assert((size_t)2 * kNumCus * 128 * 128 <= misgemm_workspace::kFloats &&
                  2 * kNumCus <= misgemm_workspace::kCounters, "partial tiles fit the workspace");
    if (g.splits > 1 && !misgemm_workspace::get(stream, &g.ws, &g.counters)) g.splits = 1;
    g.kb_per_split = (kblocks + g.splits - 1) / g.splits;
    hipLaunchKernelGGL((fp8_tile<BM, BN, WM, WN, FA, FB, ROWB, EXACT, WAY>), dim3((unsigned)(tiles * g.splits)),
                       dim3(64 * WM * WN), 0, stream, g);
    return launched();
}

template <int FA, int FB, bool ROWB, bool EXACT> int launch(int shape, GemmArgs &g, hipStream_t stream) {
    const bool near = g.lda < 1 << 24 && g.ldb < 1 << 24;
    switch (shape) {
        case 0:
            if (near) return launch_tile<128, 128, 2, 2, FA, FB, ROWB, EXACT, STAGED>(g, true, stream);
            return launch_tile<128, 128, 2, 2, FA, FB, ROWB, EXACT, FAR>(g, true, stream);
        case 1: return launch_tile<64, 128, 2, 2, FA, FB, ROWB, EXACT, STAGED>(g, false, stream);
        case 2: return launch_tile<64, 128, 2, 2, FA, FB, ROWB, EXACT, DIRECT>(g, false, stream);
        case 3: return launch_tile<128, 128, 2, 2, FA, FB, ROWB, EXACT, DIRECT>(g, true, stream);
        default:
            // Widened operands of 128 x 64 outputs do not fit a wave's registers.
            if constexpr (!EXACT) return launch_tile<256, 256, 2, 4, FA, FB, ROWB, EXACT, DIRECT>(g, false, stream);
            return MISGEMM_LAUNCH_FAILED;
    }
}

template <int FA, int FB> int launch(bool rows, int shape, GemmArgs &g, hipStream_t stream) {
    if (g.ctype == MI_F32)
        return rows ? launch<FA, FB, true, true>(shape, g, stream) : launch<FA, FB, false, true>(shape, g, stream);
    return rows ? launch<FA, FB, true, false>(shape, g, stream) : launch<FA, FB, false, false>(shape, g, stream);
}

}  // namespace

int misgemm_fp8::launch_tiles(int atype, int btype, bool rows, int shape, GemmArgs &g, hipStream_t stream) {
    if (atype == MI_E4M3)
        return btype == MI_E4M3 ? launch<MI_E4M3, MI_E4M3>(rows, shape, g, stream)
                                : launch<MI_E4M3, MI_E5M2>(rows, shape, g, stream);
    return btype == MI_E4M3 ? launch<MI_E5M2, MI_E4M3>(rows, shape, g, stream)
                            : launch<MI_E5M2, MI_E5M2>(rows, shape, g, stream);
}
