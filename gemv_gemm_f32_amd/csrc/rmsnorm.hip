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
// All sums are fp32: per thread in column order, then a fixed tree.
//
// Output in 8 bits: with 16-byte loads, 8 neighbouring lanes hold one block
// of 32 columns; with single loads, 32 lanes do.  The block's largest
// magnitude is a maximum over those lanes in registers.
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

// The V columns of chunk j of thread t: V = 4 in one 16-byte access, V = 1.
template <int V>
struct Vals {
    float v[V];
};

template <int V>
__device__ __forceinline__ Vals<V> get(const float *row, int64_t col, int K) {
    Vals<V> x;
    if constexpr (V == 4) {
        v4f q = {0.f, 0.f, 0.f, 0.f};
        if (col < K) q = *reinterpret_cast<const v4f *>(row + col);
#pragma unroll
        for (int c = 0; c < 4; ++c) x.v[c] = q[c];
    } else {
        x.v[0] = col < K ? row[col] : 0.f;
    }
    return x;
}

template <int V>
__device__ __forceinline__ void put(float *row, int64_t col, int K, const Vals<V> &x) {
    if (col >= K) return;
    if constexpr (V == 4) {
        *reinterpret_cast<v4f *>(row + col) = v4f{x.v[0], x.v[1], x.v[2], x.v[3]};
    } else {
        row[col] = x.v[0];
    }
}

// 8 bits: the lanes of a block agree on its power of two; every lane of the
// wave takes part (columns past K count as zeros).
template <int V>
__device__ __forceinline__ void put_mx8(uint8_t *qrow, uint8_t *erow, int64_t col, int K,
                                        const Vals<V> &y) {
    if constexpr (V == 4) {
        unsigned top = max(max(mag(y.v[0]), mag(y.v[1])), max(mag(y.v[2]), mag(y.v[3])));
        const int e = mx8_exponent(oct_max(top));
        if (col < K) {
            *reinterpret_cast<unsigned *>(qrow + col) = mx8_pack4(y.v[0], y.v[1], y.v[2], y.v[3], e);
            if (col % 32 == 0) erow[col / 32] = (uint8_t)e;
        }
    } else {
        const int e = mx8_exponent(half32_max(mag(y.v[0])));
        if (col < K) {
            qrow[col] = (uint8_t)mx8_pack2(y.v[0], 0.f, e);
            if (col % 32 == 0) erow[col / 32] = (uint8_t)e;
        }
    }
}

// T threads per row, NV chunks of V columns per thread.
template <int T, int V, int NV, bool MX>
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
        Vals<V> x[NV];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) x[j] = get<V>(px, (t + T * j) * V, a.K);
        if (pr) {
            Vals<V> r[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j) r[j] = get<V>(pr, (t + T * j) * V, a.K);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int c = 0; c < V; ++c) x[j].v[c] += r[j].v[c];
        }
        if (a.S && stored) {
#pragma unroll
            for (int j = 0; j < NV; ++j) put<V>(a.S + row * a.lds, (t + T * j) * V, a.K, x[j]);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int c = 0; c < V; ++c) ss = __builtin_fmaf(x[j].v[c], x[j].v[c], ss);
        ss = row_sum<T>(ss, red, flip);
        flip ^= 1;
        const float rstd = 1.f / sqrtf(ss / (float)a.K + a.eps);
        if (a.rstd && stored && t == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = (int64_t)(t + T * j) * V;
            Vals<V> g;
            if (a.gamma) g = get<V>(a.gamma, col, a.K);
#pragma unroll
            for (int c = 0; c < V; ++c) {
                x[j].v[c] *= rstd;
                if (a.gamma) x[j].v[c] *= g.v[c];
            }
            if constexpr (MX) {
                // a row that is not stored writes nowhere: K = 0 for it
                put_mx8<V>(a.Q + row * a.ldq, a.E + row * a.lde, col, stored ? a.K : 0, x[j]);
            } else if (stored) {
                put<V>(a.Y + row * a.ldy, col, a.K, x[j]);
            }
        }
    }
}

// Rows longer than the registers of 1,024 threads: S is made and summed in a
// first pass and read again (from S where it is kept, which is a thread's
// own earlier store and may lie in X's or R's place; else from X and R) in a
// second.
template <int V, bool MX>
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(RmsNorm a) {
    __shared__ float red[2][16];
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const float *px = a.X + row * a.ldx;
        const float *pr = a.R ? a.R + row * a.ldr : nullptr;
        float *ps = a.S ? a.S + row * a.lds : nullptr;
        auto sum_at = [&](int64_t col) {
            Vals<V> x = get<V>(px, col, a.K);
            if (pr) {
                const Vals<V> r = get<V>(pr, col, a.K);
#pragma unroll
                for (int c = 0; c < V; ++c) x.v[c] += r.v[c];
            }
            return x;
        };
        float ss = 0.f;
        for (int64_t c0 = 0; c0 < a.K; c0 += 1024 * V) {
            const int64_t col = c0 + threadIdx.x * V;
            const Vals<V> x = sum_at(col);
            if (ps) put<V>(ps, col, a.K, x);
#pragma unroll
            for (int c = 0; c < V; ++c) ss = __builtin_fmaf(x.v[c], x.v[c], ss);
        }
        ss = row_sum<1024>(ss, red, flip);
        flip ^= 1;
        const float rstd = 1.f / sqrtf(ss / (float)a.K + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
        for (int64_t c0 = 0; c0 < a.K; c0 += 1024 * V) {
            const int64_t col = c0 + threadIdx.x * V;
            Vals<V> y = ps ? get<V>(ps, col, a.K) : sum_at(col);
            Vals<V> g;
            if (a.gamma) g = get<V>(a.gamma, col, a.K);
#pragma unroll
            for (int c = 0; c < V; ++c) {
                y.v[c] *= rstd;
                if (a.gamma) y.v[c] *= g.v[c];
            }
            if constexpr (MX) put_mx8<V>(a.Q + row * a.ldq, a.E + row * a.lde, col, a.K, y);
            else put<V>(a.Y + row * a.ldy, col, a.K, y);
        }
    }
}

// One workgroup per partial row; its T-thread teams take rows in turn.
template <int T, int V, int NV>
__global__ __launch_bounds__(group_threads<T>()) void rmsnorm_bwd_kernel(RmsNormBwd a) {
    constexpr int THREADS = group_threads<T>(), ROWS = THREADS / T;
    __shared__ float red[2][16];
    __shared__ float part[ROWS > 1 ? THREADS * V : 1];
    const int t = threadIdx.x % T;
    const int64_t stride = (int64_t)gridDim.x * ROWS;
    Vals<V> gam[NV], dg[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (t + T * j) * V;
        if (a.gamma) gam[j] = get<V>(a.gamma, col, a.K);
#pragma unroll
        for (int c = 0; c < V; ++c) {
            if (!a.gamma) gam[j].v[c] = 1.f;
            dg[j].v[c] = 0.f;
        }
    }
    int flip = 0;
    for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.M; base += stride) {
        const int64_t want = base + threadIdx.x / T;
        const bool live = want < a.M;                 // uniform per wave
        const int64_t row = live ? want : a.M - 1;
        const float rstd = live ? a.rstd[row] : 0.f;
        Vals<V> d[NV], x[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = live ? (t + T * j) * V : a.K;
            d[j] = get<V>(a.dY + row * a.lddy, col, a.K);
            x[j] = get<V>(a.S + row * a.lds, col, a.K);
        }
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int c = 0; c < V; ++c) {
                x[j].v[c] *= rstd;                                           // xhat
                dg[j].v[c] = __builtin_fmaf(d[j].v[c], x[j].v[c], dg[j].v[c]);
                d[j].v[c] *= gam[j].v[c];                                    // g
                dot = __builtin_fmaf(d[j].v[c], x[j].v[c], dot);
            }
        if (a.dX == nullptr) continue;                // uniform
        dot = row_sum<T>(dot, red, flip) / (float)a.K;
        flip ^= 1;
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (t + T * j) * V;
            Vals<V> o;
            if (a.dS) o = get<V>(a.dS + row * a.ldds, col, a.K);
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const float v = __builtin_fmaf(-x[j].v[c], dot, d[j].v[c]) * rstd;
                o.v[c] = a.dS ? v + o.v[c] : v;
            }
            put<V>(a.dX + row * a.lddx, col, a.K, o);
        }
    }
    if (a.dgamma == nullptr) return;
    // the teams' sums meet in LDS, chunk by chunk, added in team order
    float *out = a.ws + (int64_t)blockIdx.x * a.K;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (t + T * j) * V;
        if constexpr (ROWS > 1) {
            __syncthreads();
#pragma unroll
            for (int c = 0; c < V; ++c) part[(threadIdx.x / T * T + t) * V + c] = dg[j].v[c];
            __syncthreads();
            if (threadIdx.x >= T) continue;
#pragma unroll
            for (int w = 1; w < ROWS; ++w)
#pragma unroll
                for (int c = 0; c < V; ++c) dg[j].v[c] += part[(w * T + t) * V + c];
        }
#pragma unroll
        for (int c = 0; c < V; ++c)
            if (col + c < a.K) out[col + c] = dg[j].v[c];
    }
}

// Longer rows: two passes over dY and S; the column sums live in the
// workgroup's row of the workspace, each column always touched by the same
// thread.
template <int V>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_long_kernel(RmsNormBwd a) {
    __shared__ float red[2][16];
    float *out = a.dgamma ? a.ws + (int64_t)blockIdx.x * a.K : nullptr;
    int flip = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const float rstd = a.rstd[row];
        const float *pd = a.dY + row * a.lddy, *ps = a.S + row * a.lds;
        float dot = 0.f;
        for (int64_t c0 = 0; c0 < a.K; c0 += 1024 * V) {
            const int64_t col = c0 + threadIdx.x * V;
            const Vals<V> d = get<V>(pd, col, a.K), x = get<V>(ps, col, a.K);
            Vals<V> g;
            if (a.gamma) g = get<V>(a.gamma, col, a.K);
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const float w = d.v[c] * (x.v[c] * rstd);
                dot = __builtin_fmaf(a.gamma ? g.v[c] : 1.f, w, dot);
                if (out && col + c < a.K)
                    out[col + c] = row == blockIdx.x ? w : out[col + c] + w;
            }
        }
        if (a.dX == nullptr) continue;                // uniform
        dot = row_sum<1024>(dot, red, flip) / (float)a.K;
        flip ^= 1;
        for (int64_t c0 = 0; c0 < a.K; c0 += 1024 * V) {
            const int64_t col = c0 + threadIdx.x * V;
            const Vals<V> d = get<V>(pd, col, a.K), x = get<V>(ps, col, a.K);
            Vals<V> g, o;
            if (a.gamma) g = get<V>(a.gamma, col, a.K);
            if (a.dS) o = get<V>(a.dS + row * a.ldds, col, a.K);
#pragma unroll
            for (int c = 0; c < V; ++c) {
                const float gd = a.gamma ? d.v[c] * g.v[c] : d.v[c];
                const float v = __builtin_fmaf(-(x.v[c] * rstd), dot, gd) * rstd;
                o.v[c] = a.dS ? v + o.v[c] : v;
            }
            put<V>(a.dX + row * a.lddx, col, a.K, o);
        }
    }
}

constexpr int MAX_GROUPS = 1 << 20;

inline bool aligned(const void *p, int64_t ld, int64_t bytes, int64_t elem) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * elem % bytes == 0;
}

template <int T, int V, int NV>
hipError_t norm(const RmsNorm &a, hipStream_t s) {
    constexpr int ROWS = group_threads<T>() / T;
    const int64_t groups = ((int64_t)a.M + ROWS - 1) / ROWS;
    const dim3 grid((unsigned)(groups < MAX_GROUPS ? groups : MAX_GROUPS));
    return a.Q ? launch(rmsnorm_kernel<T, V, NV, true>, grid, dim3(group_threads<T>()), s, a)
               : launch(rmsnorm_kernel<T, V, NV, false>, grid, dim3(group_threads<T>()), s, a);
}

template <int V>
hipError_t norm_of(const RmsNorm &a, hipStream_t s) {
    if (a.K <= 512) return norm<64, V, 8 / V>(a, s);
    if (a.K <= 2048) return norm<64, V, 32 / V>(a, s);
    if (a.K <= 8192) return norm<256, V, 32 / V>(a, s);
    if (a.K <= 32768) return norm<1024, V, 32 / V>(a, s);
    const dim3 grid((unsigned)(a.M < MAX_GROUPS ? a.M : MAX_GROUPS));
    return a.Q ? launch(rmsnorm_long_kernel<V, true>, grid, dim3(1024), s, a)
               : launch(rmsnorm_long_kernel<V, false>, grid, dim3(1024), s, a);
}

template <int T, int V, int NV>
hipError_t norm_bwd(const RmsNormBwd &a, hipStream_t s) {
    const int groups = a.M < RMSNORM_BWD_GROUPS ? a.M : RMSNORM_BWD_GROUPS;
    return launch(rmsnorm_bwd_kernel<T, V, NV>, dim3(groups), dim3(group_threads<T>()), s, a);
}

template <int V>
hipError_t norm_bwd_of(const RmsNormBwd &a, hipStream_t s) {
    if (a.K <= 512) return norm_bwd<64, V, 8 / V>(a, s);
    if (a.K <= 2048) return norm_bwd<64, V, 32 / V>(a, s);
    if (a.K <= 8192) return norm_bwd<256, V, 32 / V>(a, s);
    if (a.K <= 32768) return norm_bwd<1024, V, 32 / V>(a, s);
    const int groups = a.M < RMSNORM_BWD_GROUPS ? a.M : RMSNORM_BWD_GROUPS;
    return launch(rmsnorm_bwd_long_kernel<V>, dim3(groups), dim3(1024), s, a);
}

}  // namespace

hipError_t launch_rmsnorm(const RmsNorm &a, int num_cus, hipStream_t s) {
    (void)num_cus;
    const bool vec = a.K % 4 == 0 && aligned(a.X, a.ldx, 16, 4) && aligned(a.R, a.ldr, 16, 4) &&
                     aligned(a.gamma, 0, 16, 4) && aligned(a.S, a.lds, 16, 4) &&
                     aligned(a.Y, a.ldy, 16, 4) && aligned(a.Q, a.ldq, 4, 1);
    return vec ? norm_of<4>(a, s) : norm_of<1>(a, s);
}

hipError_t launch_rmsnorm_bwd(const RmsNormBwd &a, hipStream_t s) {
    if (a.M > 0) {
        const bool vec = a.K % 4 == 0 && aligned(a.dY, a.lddy, 16, 4) &&
                         aligned(a.S, a.lds, 16, 4) && aligned(a.gamma, 0, 16, 4) &&
                         aligned(a.dS, a.ldds, 16, 4) && aligned(a.dX, a.lddx, 16, 4);
        const hipError_t e = vec ? norm_bwd_of<4>(a, s) : norm_bwd_of<1>(a, s);
        if (e != hipSuccess) return e;
    }
    if (a.dgamma == nullptr) return hipSuccess;
    const int groups = a.M < RMSNORM_BWD_GROUPS ? a.M : RMSNORM_BWD_GROUPS;
    return launch_column_sum(groups, a.K, a.ws, a.accumulate, a.dgamma, s);
}

}  // namespace gg
