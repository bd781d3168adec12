// mi_act_backward and mi_gated_backward: from the gradient of f(z), or of
// f(g) u, and z or g and u as they were kept (in 8 bits with scales, or as
// matrices), their gradients, f(z) or f(g) u again, and the sums over rows
// that are the biases' gradients.
//
// Bound by memory: 8192 x 8192 gated in BF16 from E4M3, with h, reads 4 and
// writes 6 bytes a value: 132 us (5.1 TB/s; a large copy reaches 5.4). A
// workgroup takes 128 columns, which share a scale, of a run of rows; 512 columns
// at a time took 4% longer, and more rows' reads at once as much more without the
// gate (66 us for one, 73 for two). The sums cost 4 us there: each workgroup's go
// through the workspace, and the last of a strip of columns adds them, sixteen
// reads at once (one by one that took 25 us). 777 x 1300 in FP16 with its sums
// takes 7.9 us, 64 x 4096 gated with both 5.7: a launch and three memory latencies.

#include <type_traits>

#include "linear.h"

namespace {

using namespace misgemm_linear;

struct BackArgs {
    const void *dy, *z, *u;
    const float *zs, *us;
    void *dz, *du, *y;
    float *dbz, *dbu, *partials;
    int *counters;
    long long lddy, ldz, ldu, lds, ldsu, lddz, lddu, ldy;
    int rows, cols, chunks, chunk_rows;
    float beta;
};

constexpr int kNone = 0;   // Z: a matrix of the gradients' type, not an 8-bit one

// Eight 8-bit values as Eight has them of other types: one read without a
// branch, of the row's last eight where it ends, moved to their place.
struct Eight8 {
    i32x2 v;
    __device__ __forceinline__ void fetch(const uint8_t *row, int col, int cols) {
        typedef int words __attribute__((ext_vector_type(2), aligned(1)));
        v = *reinterpret_cast<const words *>(row + min(col, cols - 8));
    }
    __device__ __forceinline__ void settle(int col, int cols) {
        const int over = max(col - (cols - 8), 0);
        unsigned long long w = (uint32_t)v[0] | (unsigned long long)(uint32_t)v[1] << 32;
        w = over < 8 ? w >> (8 * over) : 0;
        v = i32x2{(int)w, (int)(w >> 32)};
    }
};

// Eight values of a row of `cols` from column col on, in T or (FMT) in 8 bits.
template <class T, int FMT> struct Row8 {
    typename std::conditional<FMT == kNone, Eight<T, false>, Eight8>::type w;
    using Memory = typename std::conditional<FMT == kNone, T, uint8_t>::type;
    __device__ __forceinline__ void fetch(const void *base, long long row, int col, int cols) {
        const Memory *p = static_cast<const Memory *>(base) + row;
        if (cols >= 8) {
            w.fetch(p, col, cols);
        } else if constexpr (FMT == kNone) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w.v[j] = j < cols ? p[j] : static_cast<T>(0.0f);
        } else {
            w.v = i32x2{0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < cols) w.v[j / 4] |= (int)((uint32_t)p[j] << (8 * (j % 4)));
        }
    }
    __device__ __forceinline__ void values(int col, int cols, float scale, float (&v)[8]) {
        if (cols >= 8 && col > cols - 8) w.settle(col, cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if constexpr (FMT == kNone) v[j] = static_cast<float>(w.v[j]);
        }
        if constexpr (FMT == MI_E4M3 || FMT == MI_E5M2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v[4 * h] = value<0>(w.v[h]) * scale;
                v[4 * h + 1] = value<1>(w.v[h]) * scale;
                v[4 * h + 2] = value<2>(w.v[h]) * scale;
                v[4 * h + 3] = value<3>(w.v[h]) * scale;
            }
        }
    }
    template <int I> static __device__ __forceinline__ float value(int w) {
        if constexpr (FMT == MI_E4M3)
            return __builtin_amdgcn_cvt_f32_fp8(w, I);
        else
            return __builtin_amdgcn_cvt_f32_bf8(w, I);
    }
};

constexpr int kLanes = 16, kRows = 16, kCols = kLanes * 8;   // of a workgroup: threads of a row, rows, columns

template <class T, int FMT, int ACT, bool GATED> __global__ __launch_bounds__(256) void act_backward(BackArgs a) {
    const int tx = threadIdx.x % kLanes, ty = threadIdx.x / kLanes;
    const int strip = blockIdx.x, chunk = blockIdx.y;
    const int col = strip * kCols + tx * 8, n = a.cols - col;
    const long long r0 = (long long)chunk * a.chunk_rows;
    const int end = (int)(r0 + a.chunk_rows < a.rows ? r0 + a.chunk_rows : a.rows);
    constexpr int AHEAD = GATED ? 2 : 1;
    float sz[8] = {}, su[8] = {};
    if (n > 0) {
        // AHEAD rows' reads on their way at once; past the end the last one's, for nothing.
        for (long long first = r0 + ty; first < end; first += kRows * AHEAD) {
            Row8<T, kNone> dyr[AHEAD];
            Row8<T, FMT> zr[AHEAD], ur[AHEAD];
            float zs[AHEAD], us[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const long long at = first + i * kRows, row = at < end ? at : end - 1;
                dyr[i].fetch(a.dy, row * a.lddy, col, a.cols);
                zr[i].fetch(a.z, row * a.ldz, col, a.cols);
                if constexpr (GATED) ur[i].fetch(a.u, row * a.ldu, col, a.cols);
                zs[i] = FMT == kNone ? 1.0f : a.zs[strip * a.lds + row];
                us[i] = FMT == kNone || !GATED ? 1.0f : a.us[strip * a.ldsu + row];
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const long long row = first + i * kRows;
                if (row >= end) break;
                float dy[8], z[8], u[8], f[8], dz[8], du[8];
                dyr[i].values(col, a.cols, 1.0f, dy);
                zr[i].values(col, a.cols, zs[i], z);
                if constexpr (GATED) ur[i].values(col, a.cols, us[i], u);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float df;
                    act_both<ACT>(z[j], f[j], df);
                    if constexpr (GATED) {
                        du[j] = dy[j] * f[j];
                        dz[j] = dy[j] * u[j] * df;
                        f[j] *= u[j];
                        su[j] += du[j];
                    } else {
                        dz[j] = dy[j] * df;
                    }
                    sz[j] += dz[j];
                }
                store8(static_cast<T *>(a.dz) + row * a.lddz + col, n, dz);
                if constexpr (GATED) store8(static_cast<T *>(a.du) + row * a.lddu + col, n, du);
                if (a.y != nullptr) store8(static_cast<T *>(a.y) + row * a.ldy + col, n, f);
            }
        }
    }
    if (a.dbz == nullptr && a.dbu == nullptr) return;

    // Sums of the workgroup's rows, in order of ty; then those of the chunks,
    // in their order, by the workgroup that comes last.
    constexpr int SETS = GATED ? 2 : 1;
    __shared__ float part[SETS][kRows][kCols];
    __shared__ int is_last;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        part[0][ty][tx * 8 + j] = sz[j];
        if constexpr (GATED) part[SETS - 1][ty][tx * 8 + j] = su[j];
    }
    __syncthreads();
    const int set = threadIdx.x / kCols, c = threadIdx.x % kCols, at = strip * kCols + c;
    float *out = set == 0 ? a.dbz : a.dbu;
    const bool mine = set < SETS && out != nullptr && at < a.cols;
    float sum = 0.0f;
    if (mine) {
#pragma unroll
        for (int r = 0; r < kRows; ++r) sum += part[set][r][c];
    }
    if (a.chunks > 1) {
        // Partial sums are written and read past the XCDs' own caches.
        float *mid = a.partials + (long long)set * a.chunks * a.cols + at;
        if (mine)
            __hip_atomic_store(mid + (long long)chunk * a.cols, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        if (threadIdx.x == 0)
            is_last = __hip_atomic_fetch_add(&a.counters[strip], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                      a.chunks - 1;
        __syncthreads();
        if (!is_last) return;
        if (threadIdx.x == 0) __hip_atomic_store(&a.counters[strip], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (mine) {
            // Sixteen reads on their way at once; those past the last are not added.
            sum = 0.0f;
            for (int k0 = 0; k0 < a.chunks; k0 += 16) {
                float v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    v[k] = __hip_atomic_load(mid + (long long)min(k0 + k, a.chunks - 1) * a.cols, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                for (int k = 0; k < 16; ++k) sum += k0 + k < a.chunks ? v[k] : 0.0f;
            }
        }
    }
    if (mine) out[at] = a.beta == 0.0f ? sum : fmaf(a.beta, out[at], sum);
}

template <class T, int FMT, int ACT, bool GATED> int launch_one(BackArgs &a, hipStream_t stream) {
    const int strips = (a.cols - 1) / kCols + 1;
    const bool sums = a.dbz != nullptr || a.dbu != nullptr;
    long long chunks = ((long long)a.rows + 4 * kRows - 1) / (4 * kRows);
    // 64 parts, but where those leave CUs without one (up to 384 columns) as many
    // as make eight workgroups to a CU: 1,000,000 x 64 in BF16 with f(z) takes 119
    // us, in 64 parts 864. With sums, which the last workgroup adds, two to a CU, of
    // 512 rows at least: 141 us for 769 (four to a CU 116, but at 128 columns 184
    // for 175; without the 512 rows 20,000 x 128 takes 17.5 us for 14.5).
    long long most = 64;
    if (strips < kNumCus / 64) {
        most = (sums ? 2 : 8) * kNumCus / strips;
        if (sums && most > a.rows / 512) most = a.rows / 512;
        if (most < 64) most = 64;
    }
    if (chunks > most) chunks = most;
    while (sums && 2 * chunks * a.cols > (long long)misgemm_workspace::kFloats) chunks /= 2;
    if (chunks < 1 || (sums && strips > misgemm_workspace::kCounters)) chunks = 1;
    if (sums && chunks > 1 && !misgemm_workspace::get(stream, &a.partials, &a.counters)) chunks = 1;
    a.chunk_rows = (int)(((long long)a.rows + chunks - 1) / chunks);
    a.chunks = a.rows == 0 ? 1 : (a.rows - 1) / a.chunk_rows + 1;
    hipLaunchKernelGGL((act_backward<T, FMT, ACT, GATED>), dim3((unsigned)strips, (unsigned)a.chunks), dim3(256), 0, stream, a);
    return launched();
}
template <class T, int FMT, bool GATED> int launch_act(int act, BackArgs &a, hipStream_t stream) {
    switch (act) {
        case MI_ACT_RELU: return launch_one<T, FMT, MI_ACT_RELU, GATED>(a, stream);
        case MI_ACT_SILU: return launch_one<T, FMT, MI_ACT_SILU, GATED>(a, stream);
        case MI_ACT_GELU: return launch_one<T, FMT, MI_ACT_GELU, GATED>(a, stream);
        case MI_ACT_GELU_TANH: return launch_one<T, FMT, MI_ACT_GELU_TANH, GATED>(a, stream);
        default: return launch_one<T, FMT, MI_ACT_NONE, GATED>(a, stream);
    }
}
template <class T, bool GATED> int launch_kept(int ztype, int act, BackArgs &a, hipStream_t stream) {
    if (ztype == MI_E4M3) return launch_act<T, MI_E4M3, GATED>(act, a, stream);
    if (ztype == MI_E5M2) return launch_act<T, MI_E5M2, GATED>(act, a, stream);
    return launch_act<T, kNone, GATED>(act, a, stream);
}
template <bool GATED> int launch_back(int type, int ztype, int act, BackArgs &a, hipStream_t stream) {
    if (type == MI_F32) return launch_kept<float, GATED>(ztype, act, a, stream);
    if (type == MI_BF16) return launch_kept<bf16, GATED>(ztype, act, a, stream);
    return launch_kept<f16, GATED>(ztype, act, a, stream);
}

// What there is to do of rows x cols: nothing, or (without rows) only sums that change.
bool idle(int rows, int cols, float beta, bool sums) { return cols == 0 || (rows == 0 && (!sums || beta == 1.0f)); }

}  // namespace

extern "C" int mi_act_backward(int type, int rows, int cols, const void *dy, int lddy, int act, int ztype,
                               const void *z, int ldz, const float *zscale, int lds, void *dz, int lddz, void *y,
                               int ldy, float beta, float *dbias, hipStream_t stream) {
    if (!is_real(type)) return MISGEMM_BAD_TYPE;
    if (rows < 0) return MISGEMM_BAD_ROWS;
    if (cols < 0) return MISGEMM_BAD_COLS;
    const bool some = rows > 0 && cols > 0;
    if (some && dy == nullptr) return MISGEMM_NULL_INPUT;
    if (lddy < cols) return MISGEMM_BAD_LD;
    if (act < MI_ACT_NONE || act > MI_ACT_GELU_TANH) return MISGEMM_BAD_ACT;
    if (ztype != type && !is_f8(ztype)) return MISGEMM_BAD_TYPE;
    if (some && z == nullptr) return MISGEMM_NULL_INPUT;
    if (ldz < cols) return MISGEMM_BAD_LD;
    if (is_f8(ztype)) {
        if (some && zscale == nullptr) return MISGEMM_NULL_SCALE;
        if (lds < rows) return MISGEMM_BAD_LDS;
    }
    if (some && dz == nullptr) return MISGEMM_NULL_OUTPUT;
    if (lddz < cols) return MISGEMM_BAD_LD;
    if (y != nullptr && ldy < cols) return MISGEMM_BAD_LD;
    if (cols > 0x7fffffff - kCols) return MISGEMM_TOO_LARGE;
    if (idle(rows, cols, beta, dbias != nullptr)) return MISGEMM_SUCCESS;

    BackArgs a = {};
    a.dy = dy;
    a.lddy = lddy;
    a.z = z;
    a.ldz = ldz;
    a.zs = zscale;
    a.lds = lds;
    a.dz = dz;
    a.lddz = lddz;
    a.y = y;
    a.ldy = ldy;
    a.dbz = dbias;
    a.rows = rows;
    a.cols = cols;
    a.beta = beta;
    return launch_back<false>(type, ztype, act, a, stream);
}

extern "C" int mi_gated_backward(int type, int rows, int cols, const void *dh, int lddh, int act, int ztype,
                                 const void *g, int ldg, const float *gscale, int ldsg, const void *u, int ldu,
                                 const float *uscale, int ldsu, void *dg, int lddg, void *du, int lddu, void *h,
                                 int ldh, float beta, float *dbiasG, float *dbiasU, hipStream_t stream) {
    if (!is_real(type)) return MISGEMM_BAD_TYPE;
    if (rows < 0) return MISGEMM_BAD_ROWS;
    if (cols < 0) return MISGEMM_BAD_COLS;
    const bool some = rows > 0 && cols > 0;
    if (some && dh == nullptr) return MISGEMM_NULL_INPUT;
    if (lddh < cols) return MISGEMM_BAD_LD;
    if (act < MI_ACT_NONE || act > MI_ACT_GELU_TANH) return MISGEMM_BAD_ACT;
    if (ztype != type && !is_f8(ztype)) return MISGEMM_BAD_TYPE;
    const bool in8 = is_f8(ztype);
    if (some && g == nullptr) return MISGEMM_NULL_INPUT;
    if (ldg < cols) return MISGEMM_BAD_LD;
    if (in8 && some && gscale == nullptr) return MISGEMM_NULL_SCALE;
    if (in8 && ldsg < rows) return MISGEMM_BAD_LDS;
    if (some && u == nullptr) return MISGEMM_NULL_INPUT;
    if (ldu < cols) return MISGEMM_BAD_LD;
    if (in8 && some && uscale == nullptr) return MISGEMM_NULL_SCALE;
    if (in8 && ldsu < rows) return MISGEMM_BAD_LDS;
    if (some && dg == nullptr) return MISGEMM_NULL_OUTPUT;
    if (lddg < cols) return MISGEMM_BAD_LD;
    if (some && du == nullptr) return MISGEMM_NULL_OUTPUT;
    if (lddu < cols) return MISGEMM_BAD_LD;
    if (h != nullptr && ldh < cols) return MISGEMM_BAD_LD;
    if (cols > 0x7fffffff - kCols) return MISGEMM_TOO_LARGE;
    if (idle(rows, cols, beta, dbiasG != nullptr || dbiasU != nullptr)) return MISGEMM_SUCCESS;

    BackArgs a = {};
    a.dy = dh;
    a.lddy = lddh;
    a.z = g;
    a.ldz = ldg;
    a.zs = gscale;
    a.lds = ldsg;
    a.u = u;
    a.ldu = ldu;
    a.us = uscale;
    a.ldsu = ldsu;
    a.dz = dg;
    a.lddz = lddg;
    a.du = du;
    a.lddu = lddu;
    a.y = h;
    a.ldy = ldh;
    a.dbz = dbiasG;
    a.dbu = dbiasU;
    a.rows = rows;
    a.cols = cols;
    a.beta = beta;
    return launch_back<true>(type, ztype, act, a, stream);
}
