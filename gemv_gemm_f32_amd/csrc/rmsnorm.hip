// rmsnorm.hip -- root-mean-square norm of rows with the residual's addition,
// and its gradients.
//
//   S = X + R,  rstd = 1 / sqrt(mean_k S^2 + eps),  Y = S * rstd * gamma
//
//   g = gamma * dY,  xhat = S * rstd
//   dX = dR = rstd * (g - xhat * mean_k(g * xhat)) + dS
//   dgamma = sum over rows of dY * xhat
//
// Both directions are bound by memory.  A row is read once: its values stay
// in the registers of the T threads that share it (T = 64, one wave, up to
// 2,048 columns; 256 up to 8,192; 1,024 up to 32,768), the sum over the row
// is a wave reduction in registers (joined over waves through LDS), and the
// results are written from the same registers.  Longer rows are read twice.
// 1,024 threads leave 128 registers each, which the eight chunks of a row
// overflow where K is not a multiple of 4 (14 and 33 registers spill) and in the
// gradients (85 and 67).  Measured against reading rows twice: fp32 output of
// 1024 x 12288 41.6 against 43.5 us, 1024 x 32768 112 against 127, 1024 x 9001
// 45.5 against 33.1; 8 bits 43.3 against 37.6, 101 against 100, 63 against 35;
// gradients 140 against 72, 213 against 199, 135 against 60.
// All sums are fp32: per thread in column order, then a fixed tree.
//
// Output in 8 bits: 8 neighbouring lanes hold one block of 32 columns, whose
// largest magnitude is a maximum over those lanes in registers.
//
// dgamma: a workgroup takes rows blockIdx.x, blockIdx.x + grid, ... and adds
// each thread's columns in registers; its sums go to one row of the
// workspace, and the rows are added in order by a second kernel.  No atomics.
#include <hip/hip_runtime.h>

#include "kernels.hpp"
#include "mx8.hpp"
#include "wave.hpp"

namespace gg {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
// rows may start at any float (or byte): wide accesses without the promise of
// 16-byte alignment
typedef v4f v4f_any __attribute__((aligned(4)));
typedef unsigned u32_any __attribute__((aligned(1)));

constexpr int WG = 256;       // threads of a workgroup, where T <= 256

template <int T>
constexpr int group_threads() { return T > WG ? T : WG; }

// Sum over the T threads that share a row; every one of them receives it.
// `red` holds a float per wave of the workgroup and is used twice, so that
// one barrier per call is enough (`flip` alternates).
template <int T>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int flip) {
    v = wave64_sum(v);
    if constexpr (T == 64) return v;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[flip][wave] = v;
    __syncthreads();
    float s = 0.f;
    constexpr int W = T / 64;
    const int first = wave / W * W;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[flip][first + w];
    return s;
}

// 4 columns of a row in one 16-byte access; columns past K read as zeros and
// are not written.  ODD: K is not a multiple of 4 (where it is, a chunk exists
// whole or not at all, and the shorter test costs a sixth less time on small
// batches: 346 x 768 4.3 against 5.2 us).
template <bool ODD>
__device__ __forceinline__ v4f get(const float *row, int64_t col, int K) {
    v4f x = {0.f, 0.f, 0.f, 0.f};
    if (ODD ? col + 4 <= K : col < K) {
        x = *reinterpret_cast<const v4f_any *>(row + col);
    } else if (ODD && col < K) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (col + c < K) x[c] = row[col + c];
    }
    return x;
}

template <bool ODD>
__device__ __forceinline__ void put(float *row, int64_t col, int K, const v4f &x) {
    if (ODD ? col + 4 <= K : col < K) {
        *reinterpret_cast<v4f_any *>(row + col) = x;
    } else if (ODD && col < K) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (col + c < K) row[col + c] = x[c];
    }
}

// 8 bits: 8 neighbouring lanes hold a block of 32 columns and agree on its
// power of two; every lane of the wave takes part (columns past K are zeros).
template <bool ODD>
__device__ __forceinline__ void put_mx8(uint8_t *qrow, uint8_t *erow, int64_t col, int K,
                                        const v4f &y) {
    unsigned top = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) top = max(top, !ODD || col + c < K ? mag(y[c]) : 0u);
    const int e = mx8_exponent(oct_max(!ODD && col >= K ? 0u : top));
    const unsigned q = mx8_pack4(y[0], y[1], y[2], y[3], e);
    if (ODD ? col + 4 <= K : col < K) {
        *reinterpret_cast<u32_any *>(qrow + col) = q;
    } else if (ODD && col < K) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (col + c < K) qrow[col + c] = (uint8_t)(q >> (8 * c));
    }
    if (col < K && col % 32 == 0) erow[col / 32] = (uint8_t)e;
}

// T threads per row, NV chunks of 4 columns per thread.
template <int T, int NV, bool ODD, bool MX>
__global__ __launch_bounds__(group_threads<T>()) void rmsnorm_kernel(RmsNorm a) {
    __shared__ float red[2][16];
    constexpr int ROWS = group_threads<T>() / T;
    const int t = threadIdx.x % T;
    int flip = 0;
    // a workgroup's waves run the same number of rounds; a row past the end
    // is computed on the last one and not stored
    for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.M; base += (int64_t)gridDim.x * ROWS) {
        const int64_t want = base + threadIdx.x / T;
        const bool stored = want < a.M;
        const int64_t row = stored ? want : a.M - 1;
        const float *px = a.X + row * a.ldx;
        const float *pr = a.R ? a.R + row * a.ldr : nullptr;
        v4f x[NV];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] = get<ODD>(px, (t + T * j) * 4, a.K);
        if (pr) {
            v4f r[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) r[j] = get<ODD>(pr, (t + T * j) * 4, a.K);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) x[j][c] += r[j][c];
        }
        if (a.S && stored) {
#pragma unroll
            for (int j = 0; j < NV; ++j) put<ODD>(a.S + row * a.lds, (t + T * j) * 4, a.K, x[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) ss = __builtin_fmaf(x[j][c], x[j][c], ss);
        ss = row_sum<T>(ss, red, flip);
        flip ^= 1;
        const float rstd = 1.f / sqrtf(ss / (float)a.K + a.eps);
        if (a.rstd && stored && t == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = (int64_t)(t + T * j) * 4;
            v4f g;
            if (a.gamma) g = get<ODD>(a.gamma, col, a.K);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[j][c] *= rstd;
                if (a.gamma) x[j][c] *= g[c];
            }
            if constexpr (MX) {
                // a row that is not stored writes nowhere: K = 0 for it
                put_mx8<ODD>(a.Q + row * a.ldq, a.E + row * a.lde, col, stored ? a.K : 0, x[j]);
            } else if (stored) {
                put<ODD>(a.Y + row * a.ldy, col, a.K, x[j]);
            }
        }
    }
}

// Rows longer than the registers of 1,024 threads: S is made and summed in a
// first pass and read again (from S where it is kept, which is a thread's
// own earlier store and may lie in X's or R's place; else from X and R) in a
// second.
template <bool ODD, bool MX>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(RmsNorm a) {
    __shared__ float red[2][16];
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const float *px = a.X + row * a.ldx;
        const float *pr = a.R ? a.R + row * a.ldr : nullptr;
        float *ps = a.S ? a.S + row * a.lds : nullptr;
        auto sum_at = [&](int64_t col) {
            v4f x = get<ODD>(px, col, a.K);
            if (pr) {
                const v4f r = get<ODD>(pr, col, a.K);
#pragma unroll
                for (int c = 0; c < 4; ++c) x[c] += r[c];
            }
            return x;
        };
        float ss = 0.f;
        for (int64_t c0 = 0; c0 < a.K; c0 += 1024 * 4) {
            const int64_t col = c0 + threadIdx.x * 4;
            const v4f x = sum_at(col);
            if (ps) put<ODD>(ps, col, a.K, x);
#pragma unroll
            for (int c = 0; c < 4; ++c) ss = __builtin_fmaf(x[c], x[c], ss);
        }
        ss = row_sum<1024>(ss, red, flip);
        flip ^= 1;
        const float rstd = 1.f / sqrtf(ss / (float)a.K + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
        for (int64_t c0 = 0; c0 < a.K; c0 += 1024 * 4) {
            const int64_t col = c0 + threadIdx.x * 4;
            v4f y = ps ? get<ODD>(ps, col, a.K) : sum_at(col);
            v4f g;
            if (a.gamma) g = get<ODD>(a.gamma, col, a.K);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                y[c] *= rstd;
                if (a.gamma) y[c] *= g[c];
            }
            if constexpr (MX) put_mx8<ODD>(a.Q + row * a.ldq, a.E + row * a.lde, col, a.K, y);
            else put<ODD>(a.Y + row * a.ldy, col, a.K, y);
        }
    }
}

// One workgroup per partial row; its T-thread teams take rows in turn.
template <int T, int NV, bool ODD>
__global__ __launch_bounds__(group_threads<T>()) void rmsnorm_bwd_kernel(RmsNormBwd a) {
    constexpr int THREADS = group_threads<T>(), ROWS = THREADS / T;
    __shared__ float red[2][16];
    __shared__ float part[ROWS > 1 ? THREADS * 4 : 1];
    const int t = threadIdx.x % T;
    const int64_t stride = (int64_t)gridDim.x * ROWS;
    v4f gam[NV], dg[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (t + T * j) * 4;
        if (a.gamma) gam[j] = get<ODD>(a.gamma, col, a.K);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (!a.gamma) gam[j][c] = 1.f;
            dg[j][c] = 0.f;
        }
    }
    int flip = 0;
    for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.M; base += stride) {
        const int64_t want = base + threadIdx.x / T;
        const bool live = want < a.M;                 // uniform per wave
        const int64_t row = live ? want : a.M - 1;
        const float rstd = live ? a.rstd[row] : 0.f;
        v4f d[NV], x[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = live ? (t + T * j) * 4 : a.K;
            d[j] = get<ODD>(a.dY + row * a.lddy, col, a.K);
            x[j] = get<ODD>(a.S + row * a.lds, col, a.K);
        }
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[j][c] *= rstd;                                           // xhat
                dg[j][c] = __builtin_fmaf(d[j][c], x[j][c], dg[j][c]);
                d[j][c] *= gam[j][c];                                    // g
                dot = __builtin_fmaf(d[j][c], x[j][c], dot);
            }
        if (a.dX == nullptr) continue;                // uniform
        dot = row_sum<T>(dot, red, flip) / (float)a.K;
        flip ^= 1;
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (t + T * j) * 4;
            v4f o;
            if (a.dS) o = get<ODD>(a.dS + row * a.ldds, col, a.K);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float v = __builtin_fmaf(-x[j][c], dot, d[j][c]) * rstd;
                o[c] = a.dS ? v + o[c] : v;
            }
            put<ODD>(a.dX + row * a.lddx, col, a.K, o);
        }
    }
    if (a.dgamma == nullptr) return;
    // the teams' sums meet in LDS, chunk by chunk, added in team order
    float *out = a.ws + (int64_t)blockIdx.x * a.K;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (t + T * j) * 4;
        if constexpr (ROWS > 1) {
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 4; ++c) part[(threadIdx.x / T * T + t) * 4 + c] = dg[j][c];
            __syncthreads();
            if (threadIdx.x >= T) continue;
#pragma unroll
            for (int w = 1; w < ROWS; ++w)
#pragma unroll
                for (int c = 0; c < 4; ++c) dg[j][c] += part[(w * T + t) * 4 + c];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (col + c < a.K) out[col + c] = dg[j][c];
    }
}

// Longer rows: two passes over dY and S; the column sums live in the
// workgroup's row of the workspace, each column always touched by the same
// thread.
template <bool ODD>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_long_kernel(RmsNormBwd a) {
    __shared__ float red[2][16];
    float *out = a.dgamma ? a.ws + (int64_t)blockIdx.x * a.K : nullptr;
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const float rstd = a.rstd[row];
        const float *pd = a.dY + row * a.lddy, *ps = a.S + row * a.lds;
        float dot = 0.f;
        for (int64_t c0 = 0; c0 < a.K; c0 += 1024 * 4) {
            const int64_t col = c0 + threadIdx.x * 4;
            const v4f d = get<ODD>(pd, col, a.K), x = get<ODD>(ps, col, a.K);
            v4f g;
            if (a.gamma) g = get<ODD>(a.gamma, col, a.K);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float w = d[c] * (x[c] * rstd);
                dot = __builtin_fmaf(a.gamma ? g[c] : 1.f, w, dot);
                if (out && col + c < a.K)
                    out[col + c] = row == blockIdx.x ? w : out[col + c] + w;
            }
        }
        if (a.dX == nullptr) continue;                // uniform
        dot = row_sum<1024>(dot, red, flip) / (float)a.K;
        flip ^= 1;
        for (int64_t c0 = 0; c0 < a.K; c0 += 1024 * 4) {
            const int64_t col = c0 + threadIdx.x * 4;
            const v4f d = get<ODD>(pd, col, a.K), x = get<ODD>(ps, col, a.K);
            v4f g, o;
            if (a.gamma) g = get<ODD>(a.gamma, col, a.K);
            if (a.dS) o = get<ODD>(a.dS + row * a.ldds, col, a.K);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float gd = a.gamma ? d[c] * g[c] : d[c];
                const float v = __builtin_fmaf(-(x[c] * rstd), dot, gd) * rstd;
                o[c] = a.dS ? v + o[c] : v;
            }
            put<ODD>(a.dX + row * a.lddx, col, a.K, o);
        }
    }
}

constexpr int MAX_GROUPS = 1 << 20;

template <int T, int NV, bool ODD>
hipError_t norm(const RmsNorm &a, hipStream_t s) {
    constexpr int ROWS = group_threads<T>() / T;
    const int64_t groups = ((int64_t)a.M + ROWS - 1) / ROWS;
    const dim3 grid((unsigned)(groups < MAX_GROUPS ? groups : MAX_GROUPS));
    return a.Q ? launch(rmsnorm_kernel<T, NV, ODD, true>, grid, dim3(group_threads<T>()), s, a)
               : launch(rmsnorm_kernel<T, NV, ODD, false>, grid, dim3(group_threads<T>()), s, a);
}

template <int T, int NV, bool ODD>
hipError_t norm_bwd(const RmsNormBwd &a, int groups, hipStream_t s) {
    return launch(rmsnorm_bwd_kernel<T, NV, ODD>, dim3(groups), dim3(group_threads<T>()), s, a);
}

template <bool ODD>
hipError_t norm_of(const RmsNorm &a, hipStream_t s) {
    if (a.K <= 512) return norm<64, 2, ODD>(a, s);
    if (a.K <= 2048) return norm<64, 8, ODD>(a, s);
    if (a.K <= 8192) return norm<256, 8, ODD>(a, s);
    if (a.K <= 32768) return norm<1024, 8, ODD>(a, s);
    const dim3 grid((unsigned)(a.M < MAX_GROUPS ? a.M : MAX_GROUPS));
    return a.Q ? launch(rmsnorm_long_kernel<ODD, true>, grid, dim3(1024), s, a)
               : launch(rmsnorm_long_kernel<ODD, false>, grid, dim3(1024), s, a);
}

template <bool ODD>
hipError_t norm_bwd_of(const RmsNormBwd &a, int groups, hipStream_t s) {
    if (a.K <= 512) return norm_bwd<64, 2, ODD>(a, groups, s);
    if (a.K <= 2048) return norm_bwd<64, 8, ODD>(a, groups, s);
    if (a.K <= 8192) return norm_bwd<256, 8, ODD>(a, groups, s);
    if (a.K <= 32768) return norm_bwd<1024, 8, ODD>(a, groups, s);
    return launch(rmsnorm_bwd_long_kernel<ODD>, dim3(groups), dim3(1024), s, a);
}

}  // namespace

hipError_t launch_rmsnorm(const RmsNorm &a, hipStream_t s) {
    return a.K % 4 ? norm_of<true>(a, s) : norm_of<false>(a, s);
}

hipError_t launch_rmsnorm_bwd(const RmsNormBwd &a, hipStream_t s) {
    // a workgroup per row of the workspace; up to 2,048 columns it takes 4 rows
    // at a time
    const int64_t rows = a.K <= 2048 ? ((int64_t)a.M + 3) / 4 : a.M;
    const int groups = (int)(rows < RMSNORM_BWD_GROUPS ? rows : RMSNORM_BWD_GROUPS);
    if (a.M > 0) {
        const hipError_t e = a.K % 4 ? norm_bwd_of<true>(a, groups, s) : norm_bwd_of<false>(a, groups, s);
        if (e != hipSuccess) return e;
    }
    if (a.dgamma == nullptr) return hipSuccess;
    return launch_column_sum(groups, a.K, a.ws, a.accumulate, a.dgamma, s);
}

}  // namespace gg
