// Products of many outputs in 16 bits, in tiles of BM x BN whose operands go
// through LDS. One translation unit for each type includes this.
//
// LDS holds BUFS blocks of 64 values of k; whole 16-byte chunks come to it
// without registers (DIRECT), others through them (STAGED, FAR). A wave forms
// the products of one half of a block while it reads the operands of the other
// from LDS, and the waves meet once a block, between the halves: by then all of
// the block is in registers, so its place takes the block BUFS further, whose
// loads go between the rows of products. What is on its way to later places
// stays so at the meeting. Operands in either layout: with k running fastest as
// they lie, otherwise by LDS's transposing reads, so no layout costs a pass.
//
// 256 x 256 outputs on eight waves (64 x 128 each, 128 registers of sums) read
// the least from L2: 8192 x 8192 x 4096 takes 376 to 414 us by the card (1.33 to
// 1.46 PFLOP/s; 128 x 256 468, 128 x 128 460 on a card where it took 377), 8192 x
// 4096 x 8192 with B's outputs running fastest 365 to 410, 4096 x 4096 x 8192
// with both across 196 to 207. What bounds them is power: the clock falls to 1.7
// to 1.9 GHz of 2.4, with the matrix cores busy 62 to 68% of the time, and
// operands of zeros take 296 us instead of 391. So what saves energy counts, not
// what fills gaps: raised wave priority and other orders of reads and loads
// changed it by 1%, v_mfma_f32_32x32x16 (413 us for 378) by its reads of sums.
// Below a round of 256 such tiles the smaller ones win: 128 x 256 outputs or 128
// x 128 on eight waves, of these two workgroups to a CU (2048 x 4096 x 1024: 19.8
// us in both, 24.3 in 256 x 256) or one with four blocks in LDS (2048 x 2048 x
// 4096: 34.5 to 37.5 us, 43 with two), and 64 x 128 (512 x 2048 x 2048: 12.1 us, k
// shared by two, 15 in 128 x 128). Four waves on 128 x 128 outputs take longer
// (20.0 us for 19.2; 46 for 37).
//
// The gated tile takes as many rows of both weights, each wave of the same
// columns, so that f(g) u needs no exchange: 8192 x 8192 x 4096 takes 744 to 776
// us (1.42 to 1.48 PFLOP/s), with both projections kept in 8 bits 823 to 840.
// What is kept costs its bytes, which all CUs write at once at a tile's end.
//
// Rows without whole chunks cost registers and addresses: 4096 x 4096 x 4096 with
// rows 8 bytes aligned takes 142 to 150 us in tiles of 256 x 128, 98 in aligned ones.
#ifndef MISGEMM_LINEAR_TILE_H
#define MISGEMM_LINEAR_TILE_H

#include "linear.h"

namespace misgemm_linear {
namespace {

// 16 bytes a lane from base + offset to LDS, 64 lanes' side by side from `lds`
// on. In assembly, since the compiler would have every later read of LDS wait
// for it: the reads here are of another buffer until `meet`. It writes no register.
__device__ __forceinline__ void load_lds(const void *base, uint32_t offset, const uint8_t *lds) {
    const uint32_t to =
        (uint32_t)reinterpret_cast<size_t>((const __attribute__((address_space(3))) uint8_t *)lds);
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(to), "v"(offset), "s"(base) : "memory");
}

// The waves of a workgroup meet, with all they have read and written in LDS
// done, and all they load to LDS landed.
__device__ __forceinline__ void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
// The same with loads to registers left on their way.
__device__ __forceinline__ void meet_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);   // LDS's counter alone
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}
// The same with each wave's last N loads to LDS left on their way.
template <int N> __device__ __forceinline__ void meet_but() {
    static_assert(N >= 0 && N < 64, "the counter's range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | N >> 4 << 14 | 7 << 4);   // none of the others
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <class T> __device__ __forceinline__ f32x4 product(typename Vec<T>::x8 a, typename Vec<T>::x8 b, f32x4 c) {
    if constexpr (std::is_same<T, bf16>::value)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// One operand's block of 64 values of k for ROWS rows of outputs, in LDS in
// 16-byte chunks, chunk q of thread q % NT. KMAJOR: memory has k running
// fastest; LDS holds rows of eight chunks, chunk c of row r at c ^ (r & 7).
// Otherwise memory has the outputs' rows running fastest; LDS holds 64 rows of
// k, whose pairs of chunks (16 values) are moved by turn(k), and the matrix
// cores' operands come through the transposing read: lane l of 16 names four
// values of row k = l / 4, and gets the l-th of each of four rows. Either way
// the lanes that read at once touch all banks.
template <class T, int ROWS, int NT, bool KMAJOR> struct Panel {
    static constexpr int PER = ROWS * 8 / NT, CHUNKS = KMAJOR ? 8 : ROWS / 8;
    static_assert(PER * NT == ROWS * 8 && NT % 64 == 0 && ROWS >= 64, "whole chunks per thread");
    static __device__ __forceinline__ int turn(int k) {
        if constexpr (ROWS >= 128) return (k & 3) | (k >> 1 & 4);
        return (k >> 1 & 1) | (k >> 2 & 2);
    }
    // Of chunk q = tid + NT * j: its row in LDS, and its chunk in memory's row.
    static __device__ __forceinline__ int row(int tid, int j) { return (tid + NT * j) / CHUNKS; }
    static __device__ __forceinline__ int chunk(int tid, int j) {
        const int r = row(tid, j);
        return (tid + NT * j) % CHUNKS ^ (KMAJOR ? r & 7 : 2 * turn(r));
    }
    // Where this lane reads 16 rows of outputs from `first` on.
    static __device__ __forceinline__ uint32_t at(int first, int lane) {
        const int i = lane % 16, grp = lane / 16;
        if constexpr (KMAJOR)
            return (first + i) * 128 + 16 * (grp ^ (i & 7));
        else
            return (8 * grp + i / 4) * (2 * ROWS) + 32 * (first / 16 ^ turn(8 * grp + i / 4)) + 8 * (i % 4);
    }
    // The operand of k values 32 s .. 32 s + 31 of the a-th 16 rows from there,
    // of at most eight (four where ROWS is 64), whose first is a multiple of as many.
    static __device__ __forceinline__ typename Vec<T>::x8 read(const uint8_t *lds, uint32_t at, int a, int s) {
        typedef short short4v __attribute__((ext_vector_type(4)));
        typedef short short8v __attribute__((ext_vector_type(8)));
        if constexpr (KMAJOR) {
            return *reinterpret_cast<const typename Vec<T>::x8 *>(lds + (at ^ 64 * s) + 2048 * a);
        } else {
            typedef __attribute__((address_space(3))) short4v lds4;
            lds4 *p = (lds4 *)(lds + (at ^ 32 * a) + 32 * s * (2 * ROWS));
            const short4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
            const short4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p + ROWS);   // four rows of k on
            const short8v v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
            return __builtin_bit_cast(typename Vec<T>::x8, v);
        }
    }
};

// Eight values of a row of `cols` from column col on, zeros past its end, in
// two steps: as they are read, and once they have come. `live`: the row is one.
template <class T> struct Chunk {
    i32x4 w;
    typedef int words __attribute__((ext_vector_type(4), aligned(2)));
    __device__ __forceinline__ void fetch(const T *row, int col, int cols) {
        if (cols >= 8) {
            w = *reinterpret_cast<const words *>(row + min(col, cols - 8));
        } else {
            uint32_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[j] = col + j < cols ? reinterpret_cast<const uint16_t *>(row)[col + j] : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = (int)(v[2 * j] | v[2 * j + 1] << 16);
        }
    }
    __device__ __forceinline__ void settle(int col, int cols, bool live) {
        if (cols >= 8) w = shifted(w, 2 * max(col - (cols - 8), 0));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = live ? w[j] : 0;
    }
};

// Operands to LDS: without registers; through them at any alignment, for leading
// dimensions below 2^23 and rows of eight values at least; the same for any.
enum Way { DIRECT, STAGED, FAR };

// BUFS blocks of k have room in LDS: one that is read, the others on their way.
template <class T, int BM, int BN, int WM, int WN, int BUFS, bool KA, bool KB, bool GATED, Way WAY>
__global__ __launch_bounds__(64 * WM * WN, WM * WN / 4 * (2 * BUFS * (BM + BN) * 128 <= 160 * 1024 ? 2 : 1)) void lin_tile(
    LinArgs g) {
    constexpr int NT = 64 * WM * WN, TM = BM / WM, TN = BN / WN, MI = TM / 16, NI = TN / 16;
    static_assert(!GATED || (KB && BN <= 256), "a tile has up to 128 columns of both projections");
    static_assert(TN == 64 || TN == 128, "");
    using PanelA = Panel<T, BM, NT, KA>;
    using PanelB = Panel<T, BN, NT, KB>;
    using x8 = typename Vec<T>::x8;
    constexpr int BYTES = (BM + BN) * 128;
    // After the sums: 16 * ROWS rows of 64 outputs of each wave, and rows' maxima.
    constexpr int ROWS = MI < 4 ? MI : 4, TURN = WM * WN * ROWS * 16 * 64 * 4, MAXES = 4 * BM * WN * (GATED ? 2 : 1);
    constexpr int LDS = BUFS * BYTES > TURN + MAXES ? BUFS * BYTES : TURN + MAXES;
    __shared__ __align__(1024) uint8_t lds[LDS];
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int i = lane % 16, grp = lane / 16;
    const int wm = wave / WN, wn = wave % WN;

    int tm, tn;
    const int tiles = g.tiles_m * g.tiles_n;
    const int split = blockIdx.x / tiles, tile = blockIdx.x - split * tiles;
    tile_of(tile, g.tiles_m, g.tiles_n, tm, tn);
    constexpr int COLS = GATED ? BN / 2 : BN;   // of outputs
    const int m0 = tm * BM, n0 = tn * COLS;
    const int kblocks = (g.K + kStep - 1) / kStep;
    const int kb0 = split * g.kb_per_split, kb1 = min(kblocks, kb0 + g.kb_per_split);
    const T *A = static_cast<const T *>(g.A), *B = static_cast<const T *>(g.B), *U = static_cast<const T *>(g.U);

    // The gated tile's rows of B: each wave has TN / 2 of the first weight's and as many of the second's, of the same columns.
    auto second = [](int r) { return GATED && r % TN >= TN / 2; };
    auto column = [](int r) { return GATED ? r / TN * (TN / 2) + r % (TN / 2) : r; };

    uint32_t from_a[PanelA::PER], from_b[PanelB::PER];
    if constexpr (WAY == DIRECT) {
        // Rows and chunks past the matrix repeat its last ones: their outputs are not stored.
#pragma unroll
        for (int j = 0; j < PanelA::PER; ++j) {
            const int r = PanelA::row(tid, j), c = PanelA::chunk(tid, j);
            from_a[j] = KA ? min(r, g.M - 1 - m0) * (uint32_t)g.lda * 2 + 16 * c
                           : r * (uint32_t)g.lda * 2 + 16 * min(c, (g.M - m0) / 8 - 1);
        }
#pragma unroll
        for (int j = 0; j < PanelB::PER; ++j) {
            const int r = PanelB::row(tid, j), c = PanelB::chunk(tid, j);
            const uint32_t ld = second(r) ? (uint32_t)g.ldu : (uint32_t)g.ldb;
            from_b[j] = KB ? min(column(r), g.N - 1 - n0) * ld * 2 + 16 * c
                           : r * ld * 2 + 16 * min(c, (g.N - n0) / 8 - 1);
        }
    }
    if constexpr (WAY == STAGED) {
        // Offsets of whole rows of a block of k, 16 bytes high to keep them
        // positive; across k (or, where k is across, along the outputs) they go
        // back to the row's last 16 bytes where it ends.
#pragma unroll
        for (int j = 0; j < PanelA::PER; ++j) {
            const int r = PanelA::row(tid, j), c = 16 * PanelA::chunk(tid, j);
            from_a[j] = (KA ? min(r, g.M - 1 - m0) : r) * (uint32_t)g.lda * 2 + 16 + (KA ? 0 : min(c, 2 * (g.M - m0) - 16));
        }
#pragma unroll
        for (int j = 0; j < PanelB::PER; ++j) {
            const int r = PanelB::row(tid, j), c = 16 * PanelB::chunk(tid, j);
            from_b[j] = (KB ? min(column(r), g.N - 1 - n0) : r) * (uint32_t)(second(r) ? g.ldu : g.ldb) * 2 + 16 +
                        (KB ? 0 : min(c, 2 * (g.N - n0) - 16));
        }
    }
    auto copy_a = [&](int kb, int buf, int j) {
        const T *src = KA ? A + m0 * g.lda + (long long)kb * kStep : A + (long long)kb * kStep * g.lda + m0;
        load_lds(src, from_a[j], lds + buf * BYTES + 1024 * wave + 16 * NT * j);
    };
    auto copy_b = [&](int kb, int buf, int j) {
        // A wave's 64 chunks are eight rows, of one weight.
        const T *src;
        if constexpr (KB) {
            const bool u = second(8 * wave + NT / 8 * j);
            src = (u ? U + n0 * g.ldu : B + n0 * g.ldb) + (long long)kb * kStep;
        } else {
            src = B + (long long)kb * kStep * g.ldb + n0;
        }
        load_lds(src, from_b[j], lds + buf * BYTES + BM * 128 + 1024 * wave + 16 * NT * j);
    };
    auto copy = [&](int kb, int buf) {
#pragma unroll
        for (int j = 0; j < PanelA::PER; ++j) copy_a(kb, buf, j);
#pragma unroll
        for (int j = 0; j < PanelB::PER; ++j) copy_b(kb, buf, j);
    };
    struct Chunks {
        Chunk<T> a[PanelA::PER], b[PanelB::PER];
    };
    // A block's 16 bytes of each of a thread's chunks, by offsets from its beginning.
    auto fetch_near = [&](Chunks &w, int kb) {
        asm("" : "+s"(kb));   // hides that kb counts a loop: each load would get a pointer of its own
        const int left = g.K - kb * kStep;
        auto get = [](const T *base, uint32_t offset) {
            return *reinterpret_cast<const typename Chunk<T>::words *>(reinterpret_cast<const uint8_t *>(base) - 16 + offset);
        };
        // Rows of k past its end: the last one's, to be cleared.
        auto across = [&](uint32_t from, int r, long long ld) {
            return left >= kStep ? from : from - max(r - (left - 1), 0) * (uint32_t)ld * 2;
        };
#pragma unroll
        for (int j = 0; j < PanelA::PER; ++j) {
            const int c = 16 * PanelA::chunk(tid, j);
            if (KA)
                w.a[j].w = get(A + m0 * g.lda + (long long)kb * kStep, from_a[j] + min(c, 2 * left - 16));
            else
                w.a[j].w = get(A + (long long)kb * kStep * g.lda + m0, across(from_a[j], PanelA::row(tid, j), g.lda));
        }
#pragma unroll
        for (int j = 0; j < PanelB::PER; ++j) {
            const int c = 16 * PanelB::chunk(tid, j);
            if (KB) {
                const bool u = second(8 * wave + NT / 8 * j);   // eight rows of a wave are of one weight
                w.b[j].w = get((u ? U + n0 * g.ldu : B + n0 * g.ldb) + (long long)kb * kStep, from_b[j] + min(c, 2 * left - 16));
            } else {
                w.b[j].w = get(B + (long long)kb * kStep * g.ldb + n0, across(from_b[j], PanelB::row(tid, j), g.ldb));
            }
        }
    };
    auto fetch = [&](Chunks &w, int kb) {
        if constexpr (WAY == STAGED) {
            fetch_near(w, kb);
            return;
        }
        const int k0 = kb * kStep;
#pragma unroll
        for (int j = 0; j < PanelA::PER; ++j) {
            const int r = PanelA::row(tid, j), c = 8 * PanelA::chunk(tid, j);
            if (KA)
                w.a[j].fetch(A + min(m0 + r, g.M - 1) * g.lda, k0 + c, g.K);
            else
                w.a[j].fetch(A + min(k0 + r, g.K - 1) * g.lda, m0 + c, g.M);
        }
#pragma unroll
        for (int j = 0; j < PanelB::PER; ++j) {
            const int r = PanelB::row(tid, j), c = 8 * PanelB::chunk(tid, j);
            if (KB)
                w.b[j].fetch((second(r) ? U : B) + min(n0 + column(r), g.N - 1) * (second(r) ? g.ldu : g.ldb), k0 + c, g.K);
            else
                w.b[j].fetch(B + min(k0 + r, g.K - 1) * g.ldb, n0 + c, g.N);
        }
    };
    auto write = [&](Chunks &w, int kb, int buf) {
        const int k0 = kb * kStep;
        const bool edge = k0 + kStep > g.K;
        if (edge || (!KA && m0 + BM > g.M)) {
#pragma unroll
            for (int j = 0; j < PanelA::PER; ++j) {
                const int r = PanelA::row(tid, j), c = 8 * PanelA::chunk(tid, j);
                w.a[j].settle((KA ? k0 : m0) + c, KA ? g.K : g.M, KA || k0 + r < g.K);
            }
        }
        if (edge || (!KB && n0 + BN > g.N)) {
#pragma unroll
            for (int j = 0; j < PanelB::PER; ++j) {
                const int r = PanelB::row(tid, j), c = 8 * PanelB::chunk(tid, j);
                w.b[j].settle((KB ? k0 : n0) + c, KB ? g.K : g.N, KB || k0 + r < g.K);
            }
        }
#pragma unroll
        for (int j = 0; j < PanelA::PER; ++j)
            *reinterpret_cast<i32x4 *>(lds + buf * BYTES + 16 * (tid + NT * j)) = w.a[j].w;
#pragma unroll
        for (int j = 0; j < PanelB::PER; ++j)
            *reinterpret_cast<i32x4 *>(lds + buf * BYTES + BM * 128 + 16 * (tid + NT * j)) = w.b[j].w;
    };

    f32x4 acc[MI][NI];
#pragma unroll
    for (int a = 0; a < MI; ++a)
#pragma unroll
        for (int b = 0; b < NI; ++b) acc[a][b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // Operands of half a block each: one half's products run while the other's are read.
    struct Half {
        x8 a[MI], b[NI];
    };
    Half half[2];
    const uint32_t at_a = PanelA::at(wm * TM, lane), at_b = PanelB::at(wn * TN, lane);
    auto read = [&](int buf, int s, int p) {
        Half &h = half[s];
        if (p < NI)
            h.b[p] = PanelB::read(lds + buf * BYTES + BM * 128, at_b, p, s);
        else
            h.a[p - NI] = PanelA::read(lds + buf * BYTES, at_a, p - NI, s);
    };
    constexpr int READS = MI + NI;
    // The products of one half; before each row of them some of the next half's
    // reads, and of `more`. Transposing reads are twice as many and spread over
    // all rows, others over three quarters of them (each the faster, by 1 to 3%).
    // Every other row goes backwards: one operand stays from product to product.
    auto upto = [](int a) { return min(READS, KA && KB ? READS * a * 4 / (3 * MI) : READS * a / MI); };
    auto multiply = [&](int s, int next_buf, auto more) __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < MI; ++a) {
#pragma unroll
            for (int p = upto(a); p < upto(a + 1); ++p) read(next_buf, s ^ 1, p);
            more(a);
#pragma unroll
            for (int b0 = 0; b0 < NI; ++b0) {
                const int b = a & 1 ? NI - 1 - b0 : b0;
                acc[a][b] = product<T>(half[s].b[b], half[s].a[a], acc[a][b]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto nothing = [](int) {};

    const int last = WAY != DIRECT ? kb1 : min(kb1, g.K / kStep);   // the blocks that the loop takes
    if (kb0 < last) {
        constexpr int PER = PanelA::PER + PanelB::PER, AHEAD = BUFS - 1;
        if constexpr (WAY != DIRECT) {
            // Two blocks in LDS, and the next ones on their way to registers:
            // two (8% faster than one, 4096 x 4096 x 4096 with 128 x 128 outputs),
            // but one where two workgroups to a CU have no registers for more.
            static_assert(BUFS == 2, "");
            constexpr int SETS = 2 * LDS <= 160 * 1024 && BM * BN >= 128 * 128 ? 1 : 2;
            Chunks w[SETS];
            fetch(w[0], kb0);
            if (SETS == 2 && kb0 + 1 < last) fetch(w[SETS - 1], kb0 + 1);
            write(w[0], kb0, 0);
            if (kb0 + SETS < last) fetch(w[0], kb0 + SETS);
            meet_lds();
            if (kb0 + 1 < last) write(w[SETS - 1], kb0 + 1, 1);
            if (kb0 + 1 + SETS < last) fetch(w[SETS - 1], kb0 + 1 + SETS);
#pragma unroll
            for (int p = 0; p < READS; ++p) read(0, 0, p);
            auto block = [&](int kb, auto buf_) {
                constexpr int buf = decltype(buf_)::value;
                multiply(0, buf, nothing);
                // All of this block is in registers, and the next one is written.
                meet_lds();
                if (kb + 2 < last) write(w[buf % SETS], kb + 2, buf);
                if (kb + 2 + SETS < last) fetch(w[buf % SETS], kb + 2 + SETS);
                multiply(1, buf ^ 1, nothing);
            };
#pragma unroll 1
            for (int kb = kb0; kb < last; kb += 2) {
                block(kb, std::integral_constant<int, 0>{});
                if (kb + 1 < last) block(kb + 1, std::integral_constant<int, 1>{});
            }
        } else {
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (kb0 + k < last) copy(kb0 + k, k);
            if (kb0 + AHEAD <= last)
                meet_but<PER *(AHEAD - 1)>();
            else
                meet();
            if (kb0 + AHEAD < last) copy(kb0 + AHEAD, AHEAD);
#pragma unroll
            for (int p = 0; p < READS; ++p) read(0, 0, p);
            int buf = 0;
#pragma unroll 1
            for (int kb = kb0; kb < last; ++kb) {
                const int next = buf + 1 == BUFS ? 0 : buf + 1;
                multiply(0, buf, nothing);
                // All of this block is in registers, and the next one has landed.
                if (BUFS > 2 && kb + BUFS <= last)
                    meet_but<PER *(BUFS - 2)>();
                else
                    meet();
                // The block that this one's place is for, a part before each row of products.
                const bool more = kb + BUFS < last;
                multiply(1, next, [&](int a) {
                    if (!more) return;
#pragma unroll
                    for (int j = PER * a / MI; j < PER * (a + 1) / MI; ++j) {
                        if (j < PanelA::PER)
                            copy_a(kb + BUFS, buf, j);
                        else
                            copy_b(kb + BUFS, buf, j - PanelA::PER);
                    }
                });
                buf = next;
            }
        }
    }
    if constexpr (WAY == DIRECT) {
        if (last < kb1) {   // the last block of k, where it is short
            Chunks w;
            fetch(w, last);
            meet();
            write(w, last, 0);
            meet();
#pragma unroll
            for (int p = 0; p < READS; ++p) read(0, 0, p);
            multiply(0, 0, nothing);
            multiply(1, 0, nothing);
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
        int *is_last = reinterpret_cast<int *>(lds);   // of the operands' memory, which is read no more
        if (tid == 0)
            *is_last = __hip_atomic_fetch_add(&g.counters[tile], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                      g.splits - 1;
        __syncthreads();
        if (!*is_last) return;
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

    // z: a lane holds row 16 a + i and columns 16 b + 4 grp + 0..3 of its wave's.
    meet();
    const int m1 = m0 + wm * TM, n1 = n0 + wn * (GATED ? TN / 2 : TN);
    constexpr int NH = GATED ? NI / 2 : NI;   // sixteens of columns of outputs
    if (g.alpha != 1.0f || g.bias != nullptr || (GATED && g.bias_u != nullptr))
#pragma unroll
    for (int b = 0; b < NI; ++b) {
        const int n = n1 + 16 * (b % NH) + 4 * grp;
        float bias[4];
        bias_at<T, 4>(b < NH ? g.bias : g.bias_u, g.bias32, n, g.N - n, bias);
#pragma unroll
        for (int a = 0; a < MI; ++a)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[a][b][j] = fmaf(g.alpha, acc[a][b][j], bias[j]);
    }
    // Largest |z| of each row and 128 columns, which SHARE waves have.
    constexpr int SHARE = GATED ? WN : 128 / TN;
    float *maxes = reinterpret_cast<float *>(lds + TURN);
    const bool in8 = g.zs != nullptr;
    auto row_maxes = [&](auto edge_) {
        constexpr bool edge = decltype(edge_)::value;   // columns past the matrix do not count
#pragma unroll
        for (int half = 0; half < (GATED ? 2 : 1); ++half)
#pragma unroll
            for (int a = 0; a < MI; ++a) {
                float m = 0.0f;
#pragma unroll
                for (int b = half * NH; b < (half + 1) * NH; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        m = fmaxf(m, edge && n1 + 16 * (b - half * NH) + 4 * grp + j >= g.N ? 0.0f : fabsf(acc[a][b][j]));
                m = fmaxf(m, __shfl_xor(m, 16));
                m = fmaxf(m, __shfl_xor(m, 32));
                if (grp == 0) maxes[(half * WN + wn) * BM + wm * TM + 16 * a + i] = m;
            }
    };
    if (in8) {
        if (n0 + COLS > g.N)
            row_maxes(std::true_type{});
        else
            row_maxes(std::false_type{});
        __syncthreads();
        // The tables, and what values are multiplied by in the maxima's place.
        constexpr int EACH = WN / SHARE;   // blocks of 128 columns, or weights, times rows
        const float most = g.ztype == MI_E4M3 ? top<MI_E4M3>() : top<MI_E5M2>();
        for (int t = tid; t < (GATED ? 2 : EACH) * BM; t += NT) {
            const int part = t / BM, r = t % BM, m = m0 + r, n = GATED ? n0 : n0 + kBlock * part;
            float a = kTiny;
#pragma unroll
            for (int w = 0; w < SHARE; ++w) a = fmaxf(a, maxes[(part * SHARE + w) * BM + r]);
            maxes[part * SHARE * BM + r] = most / a;
            if (m < g.M && n < g.N) {
                float *table = GATED && part == 1 ? g.zus : g.zs;
                table[n / kBlock * (GATED && part == 1 ? g.ldsu : g.lds) + m] = a / most;
            }
        }
        __syncthreads();
    }
    // Outputs turn in LDS, each wave's in its own, and leave as whole rows:
    // 64 columns at a time, or 32 and 32 of the two projections. Chunk c (four
    // values) of row r is at c ^ (r & 15). A lane takes eight columns of up to
    // four rows at once, so that their reads and the choices on the way (the
    // activation, types, what is kept) are shared; where the tile ends inside
    // the matrix, without a bound to check.
    f32x4 *own = reinterpret_cast<f32x4 *>(lds) + wave * ROWS * 256;
    constexpr int LANES = GATED ? 4 : 8, STEP = 64 / LANES;   // of a row; rows at a time
    constexpr int SETS = 16 * ROWS / STEP, R = SETS < 4 ? SETS : 4;
    constexpr bool STREAM = BM * BN == 256 * 256;
    auto leave = [&](auto whole_) __attribute__((always_inline)) {
        constexpr bool WHOLE = decltype(whole_)::value;
#pragma unroll
        for (int p = 0; p < NI / 4; ++p)
#pragma unroll
            for (int a0 = 0; a0 < MI; a0 += ROWS) {
#pragma unroll
                for (int a = 0; a < ROWS; ++a)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        own[(16 * a + i) * 16 + ((4 * b + grp) ^ i)] =
                            acc[a0 + a][GATED ? (b < 2 ? 2 * p + b : NH + 2 * p + b - 2) : 4 * p + b];
                asm volatile("" ::: "memory");
#pragma unroll 1
                for (int s0 = 0; s0 < SETS; s0 += R) {
                    // Chunk c and the next one, or (FP32: a lane's 16 bytes beside its neighbours') the eighth from it.
                    const bool apart = !GATED && g.c32;
                    const int r0 = s0 * STEP + lane / LANES, c = lane % LANES * (apart ? 1 : 2);
                    const int m = m1 + 16 * a0 + r0, n = n1 + (GATED ? 32 : 64) * p + 4 * c;
                    float v[8 * R], u[8 * R];
#pragma unroll
                    for (int s = 0; s < R; ++s)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int r = r0 + s * STEP;
                            const f32x4 x = own[r * 16 + ((c + (apart ? 8 * h : h)) ^ (r & 15))];
                            f32x4 y = {};
                            if constexpr (GATED) y = own[r * 16 + ((8 + c + h) ^ (r & 15))];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                v[8 * s + 4 * h + j] = x[j];
                                u[8 * s + 4 * h + j] = y[j];
                            }
                        }
                    if (!WHOLE && n >= g.N) continue;
                    if (in8) {
                        auto keep = [&](const float *z, int part, void *q, long long ldq) {
                            uint8_t *to = static_cast<uint8_t *>(q) + m * ldq + n;
#pragma unroll
                            for (int s = 0; s < R; ++s, z += 8) {
                                const float f = maxes[part * SHARE * BM + wm * TM + 16 * a0 + r0 + s * STEP];
                                int w[2];
                                if (g.ztype == MI_E4M3) {
                                    w[0] = pack4<MI_E4M3>(z[0] * f, z[1] * f, z[2] * f, z[3] * f);
                                    w[1] = pack4<MI_E4M3>(z[4] * f, z[5] * f, z[6] * f, z[7] * f);
                                } else {
                                    w[0] = pack4<MI_E5M2>(z[0] * f, z[1] * f, z[2] * f, z[3] * f);
                                    w[1] = pack4<MI_E5M2>(z[4] * f, z[5] * f, z[6] * f, z[7] * f);
                                }
                                if (WHOLE || m + s * STEP < g.M)
                                    put_bytes<STREAM && !GATED>(to + s * (STEP * ldq), WHOLE ? 64 : g.N - n, w, apart);
                            }
                        };
                        keep(v, GATED ? 0 : wn / SHARE, g.z, g.ldz);
                        if constexpr (GATED) keep(u, 1, g.zu, g.ldzu);
                    }
                    put_out<T, GATED, R, 8, WHOLE, STREAM, true>(g, m, STEP, n, v, u);
                }
                asm volatile("" ::: "memory");
            }
    };
    if (m0 + BM <= g.M && n0 + COLS <= g.N)
        leave(std::true_type{});
    else
        leave(std::false_type{});
}

template <class T, int BM, int BN, int WM, int WN, int BUFS, bool KA, bool KB, bool GATED, Way WAY>
int launch_tile(LinArgs &g, hipStream_t stream) {
    constexpr int COLS = GATED ? BN / 2 : BN;
    g.tiles_m = (g.M + BM - 1) / BM;
    g.tiles_n = (g.N + COLS - 1) / COLS;
    const int kblocks = (g.K + kStep - 1) / kStep;
    const long long tiles = (long long)g.tiles_m * g.tiles_n;
    // What was chosen (its parts fit), where the stream has a workspace.
    if (g.splits > 1 && !misgemm_workspace::get(stream, &g.ws, &g.counters)) g.splits = 1;
    g.kb_per_split = (kblocks + g.splits - 1) / g.splits;
    if (g.splits > 1) g.splits = (kblocks + g.kb_per_split - 1) / g.kb_per_split;
    hipLaunchKernelGGL((lin_tile<T, BM, BN, WM, WN, BUFS, KA, KB, GATED, WAY>), dim3((unsigned)(tiles * g.splits)),
                       dim3(64 * WM * WN), 0, stream, g);
    return launched();
}

template <class T, bool KA, bool KB> int launch_linear(int shape, LinArgs &g, hipStream_t stream) {
    switch (shape) {
        case 0:
            if (!g.near) return launch_tile<T, 128, 128, 4, 2, 2, KA, KB, false, FAR>(g, stream);
            return launch_tile<T, 128, 128, 4, 2, 2, KA, KB, false, STAGED>(g, stream);
        case 1: return launch_tile<T, 64, 128, 4, 2, 2, KA, KB, false, STAGED>(g, stream);
        case 2: return launch_tile<T, 256, 128, 4, 2, 2, KA, KB, false, STAGED>(g, stream);
        case 8: return launch_tile<T, 64, 128, 4, 2, 3, KA, KB, false, DIRECT>(g, stream);
        case 9: return launch_tile<T, 128, 128, 4, 2, 2, KA, KB, false, DIRECT>(g, stream);
        case 10: return launch_tile<T, 128, 128, 4, 2, 4, KA, KB, false, DIRECT>(g, stream);
        case 11: return launch_tile<T, 128, 256, 2, 4, 3, KA, KB, false, DIRECT>(g, stream);
        case 12:
            // Waves of 64 x 128 outputs, but of 128 x 64 where B alone comes by transposing reads.
            if constexpr (KA && !KB)
                return launch_tile<T, 256, 256, 2, 4, 2, KA, KB, false, DIRECT>(g, stream);
            else
                return launch_tile<T, 256, 256, 4, 2, 2, KA, KB, false, DIRECT>(g, stream);
        default: return MISGEMM_LAUNCH_FAILED;
    }
}
template <class T> int launch_gated(int shape, LinArgs &g, hipStream_t stream) {
    switch (shape) {
        case 0:
            if (!g.near) return launch_tile<T, 128, 256, 2, 4, 2, true, true, true, FAR>(g, stream);
            return launch_tile<T, 128, 256, 2, 4, 2, true, true, true, STAGED>(g, stream);
        case 1: return launch_tile<T, 64, 256, 2, 4, 2, true, true, true, STAGED>(g, stream);
        case 8: return launch_tile<T, 64, 256, 2, 4, 3, true, true, true, DIRECT>(g, stream);
        case 9: return launch_tile<T, 64, 256, 2, 4, 2, true, true, true, DIRECT>(g, stream);
        case 10: return launch_tile<T, 128, 128, 4, 2, 4, true, true, true, DIRECT>(g, stream);
        case 11: return launch_tile<T, 128, 128, 4, 2, 2, true, true, true, DIRECT>(g, stream);
        case 12: return launch_tile<T, 128, 256, 2, 4, 3, true, true, true, DIRECT>(g, stream);
        case 13: return launch_tile<T, 256, 256, 4, 2, 2, true, true, true, DIRECT>(g, stream);
        default: return MISGEMM_LAUNCH_FAILED;
    }
}

// ta, tb: A is K x M, B is N x K in memory.
template <class T> int launch_tiles(bool gated, bool ta, bool tb, int shape, LinArgs &g, hipStream_t stream) {
    if (gated) return launch_gated<T>(shape, g, stream);
    if (ta)
        return tb ? launch_linear<T, false, true>(shape, g, stream) : launch_linear<T, false, false>(shape, g, stream);
    return tb ? launch_linear<T, true, true>(shape, g, stream) : launch_linear<T, true, false>(shape, g, stream);
}

}  // namespace
}  // namespace misgemm_linear

#endif  // MISGEMM_LINEAR_TILE_H
