// block_norm.hip -- the norms behind a block and before the next one, with the
// block's gate and the residual's scale between them, and their gradients.
//
//   V = U rstd_u gamma_u,       rstd_u = 1 / sqrt(mean_k U^2 + eps)
//   S = alpha X + gate V
//   Y = S rstd_s gamma_s,       rstd_s = 1 / sqrt(mean_k S^2 + eps)
//
//   xs = S rstd_s,  g = gamma_s dY,  dS = rstd_s (g - xs mean_k(g xs)) + dS'
//   dX = alpha dS,  dV = gate dS,  dgate = dS V
//   xu = U rstd_u,  h = gamma_u dV,  dU = rstd_u (h - xu mean_k(h xu))
//   dgamma_s = sum over rows of dY xs,  dgamma_u = sum over rows of dV xu
//
// Both directions are bound by memory: forward reads U and X and writes S and
// Y, where norm, gate, addition and norm in launches of their own move 2.5
// times that.  A row stays in the registers of the T threads that share it
// (row.hpp) through both of its sums, which depend on each other; everything a
// row needs, vectors included, is asked for before the first sum, so that few
// rows pay one trip to memory.  Loads are unconditional, from columns clamped
// into the row: a load under a branch is waited for where the branch joins.
//
// Column sums: with one gate for all rows, dgamma_u = gate q and dgate =
// gamma_u q with one q = sum over rows of dS xu; with a gate per row, dgate is
// a row's own and dgamma_u = sum over rows of (gate dS) xu.  So there are two
// sums per column either way.  A workgroup adds its rows in registers, its
// sums become a row of the workspace, and a second kernel adds those rows in
// order and finishes both vectors.  No atomics; all sums are fp32.
#include <hip/hip_runtime.h>

#include "kernels.hpp"
#include "row.hpp"

namespace gg {
namespace {

// What K is: a multiple of 4, another number from 5 on, or less than 4.
enum Fit { WHOLE, CUT, TINY };

// 4 columns of a row; columns past K read as zeros.
template <Fit F>
__device__ __forceinline__ v4f take(const float *row, int64_t col, int K) {
    if constexpr (F == TINY) return get<true>(row, col, K);
    const int64_t from = min(col, (int64_t)K - 4);
    v4f x = *reinterpret_cast<const v4f_any *>(row + from);
    if constexpr (F == WHOLE) {
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = col < K ? x[c] : 0.f;
    } else {
        // the load ends where the row does: drop what comes before col
        const int64_t n = col - from;
        if (n & 1) x = v4f{x[1], x[2], x[3], 0.f};
        if (n & 2) x = v4f{x[2], x[3], 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = n < 4 ? x[c] : 0.f;
    }
    return x;
}

// The same of a vector, ones where there is none.
template <Fit F>
__device__ __forceinline__ v4f factor(const float *vec, int64_t col, int K) {
    if (vec == nullptr) return v4f{1.f, 1.f, 1.f, 1.f};
    return take<F>(vec, col, K);
}

// T threads per row, NV chunks of 4 columns per thread.
template <int T, int NV, Fit F, bool MX>
__global__ __launch_bounds__(group_threads<T>()) void block_norm_kernel(BlockNorm a) {
    __shared__ float red[2][16];
    constexpr int ROWS = group_threads<T>() / T;
    constexpr bool ODD = F != WHOLE;
    const int t = threadIdx.x % T;
    const float invk = 1.f / (float)a.K;
    // a workgroup's waves run the same number of rounds; a row past the end
    // is computed on the last one and not stored
    for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.M; base += (int64_t)gridDim.x * ROWS) {
        const int64_t want = base + threadIdx.x / T;
        const bool stored = want < a.M;
        const int64_t row = stored ? want : a.M - 1;
        v4f u[NV], x[NV], gu[NV], gt[NV], gs[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = (int64_t)(t + T * j) * 4;
            u[j] = take<F>(a.U + row * a.ldu, col, a.K);
            x[j] = take<F>(a.X + row * a.ldx, col, a.K);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = (int64_t)(t + T * j) * 4;
            gu[j] = factor<F>(a.gu, col, a.K);
            gt[j] = factor<F>(a.gate ? a.gate + row * a.ldg : nullptr, col, a.K);
            gs[j] = factor<F>(a.gs, col, a.K);
        }
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) ss = __builtin_fmaf(u[j][c], u[j][c], ss);
        ss = row_sum<T>(ss, red, 0);
        const float ru = 1.f / sqrtf(ss * invk + a.eps);
        ss = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[j][c] = __builtin_fmaf(a.alpha, x[j][c], u[j][c] * ru * gu[j][c] * gt[j][c]);
                ss = __builtin_fmaf(x[j][c], x[j][c], ss);
            }
            if (stored) put<ODD>(a.S + row * a.lds, (int64_t)(t + T * j) * 4, a.K, x[j]);
        }
        ss = row_sum<T>(ss, red, 1);
        const float rs = 1.f / sqrtf(ss * invk + a.eps);
        if (stored && t == 0) {
            if (a.ru) a.ru[row] = ru;
            if (a.rs) a.rs[row] = rs;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = (int64_t)(t + T * j) * 4;
#pragma unroll
            for (int c = 0; c < 4; ++c) x[j][c] = x[j][c] * rs * gs[j][c];
            if constexpr (MX) {
                // a row that is not stored writes nowhere: K = 0 for it
                put_mx8<ODD>(a.Q + row * a.ldq, a.E + row * a.lde, col, stored ? a.K : 0, x[j]);
            } else if (stored) {
                put<ODD>(a.Y + row * a.ldy, col, a.K, x[j]);
            }
        }
    }
}

// Rows longer than the registers hold: U is read twice, and S, a thread's own
// earlier store, again.
template <Fit F, bool MX>
__global__ __launch_bounds__(1024) void block_norm_long_kernel(BlockNorm a) {
    __shared__ float red[2][16];
    constexpr bool ODD = F != WHOLE;
    const float invk = 1.f / (float)a.K;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const float *pu = a.U + row * a.ldu, *px = a.X + row * a.ldx;
        const float *pg = a.gate ? a.gate + row * a.ldg : nullptr;
        float *ps = a.S + row * a.lds;
        float ss = 0.f;
        for (int64_t c0 = 0; c0 < a.K; c0 += 4096) {
            const v4f u = take<F>(pu, c0 + threadIdx.x * 4, a.K);
#pragma unroll
            for (int c = 0; c < 4; ++c) ss = __builtin_fmaf(u[c], u[c], ss);
        }
        ss = row_sum<1024>(ss, red, 0);
        const float ru = 1.f / sqrtf(ss * invk + a.eps);
        ss = 0.f;
        for (int64_t c0 = 0; c0 < a.K; c0 += 4096) {
            const int64_t col = c0 + threadIdx.x * 4;
            const v4f u = take<F>(pu, col, a.K), gu = factor<F>(a.gu, col, a.K);
            const v4f gt = factor<F>(pg, col, a.K);
            v4f x = take<F>(px, col, a.K);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[c] = __builtin_fmaf(a.alpha, x[c], u[c] * ru * gu[c] * gt[c]);
                ss = __builtin_fmaf(x[c], x[c], ss);
            }
            put<ODD>(ps, col, a.K, x);
        }
        ss = row_sum<1024>(ss, red, 1);
        const float rs = 1.f / sqrtf(ss * invk + a.eps);
        if (threadIdx.x == 0) {
            if (a.ru) a.ru[row] = ru;
            if (a.rs) a.rs[row] = rs;
        }
        for (int64_t c0 = 0; c0 < a.K; c0 += 4096) {
            const int64_t col = c0 + threadIdx.x * 4;
            v4f y = get<ODD>(ps, col, a.K);
            const v4f gs = factor<F>(a.gs, col, a.K);
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = y[c] * rs * gs[c];
            if constexpr (MX) put_mx8<ODD>(a.Q + row * a.ldq, a.E + row * a.lde, col, a.K, y);
            else put<ODD>(a.Y + row * a.ldy, col, a.K, y);
        }
    }
}

// One workgroup per row of the workspace (sums of dgamma_s, then q); its
// T-thread teams take rows in turn.  With more than two chunks per thread the
// column sums lie in LDS, each touched by its own thread alone, and vectors are
// read again for each row: registers hold the row and no more.
template <int T, int NV, Fit F>
__global__ __launch_bounds__(group_threads<T>()) void block_norm_bwd_kernel(BlockNormBwd a) {
    constexpr int THREADS = group_threads<T>(), ROWS = THREADS / T;
    constexpr bool ODD = F != WHOLE, FULL = NV > 2;
    static_assert(!FULL || ROWS == 1, "one team where the sums lie in LDS");
    __shared__ float red[2][16];
    __shared__ float part[ROWS > 1 ? THREADS * 4 : 1];
    __shared__ v4f sums[FULL ? 2 * NV * T : 1];
    const int t = threadIdx.x % T;
    const float invk = 1.f / (float)a.K;
    constexpr int HELD = FULL ? 1 : NV;
    v4f gu[HELD], gs[HELD], gt[NV], qs[HELD], qu[HELD];
    const auto zero = v4f{0.f, 0.f, 0.f, 0.f};
    const auto column = [&](int j) { return (int64_t)(t + T * j) * 4; };
    if constexpr (FULL) {
#pragma unroll
        for (int j = 0; j < 2 * NV; ++j) sums[j * T + t] = zero;
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            gu[j] = factor<F>(a.gu, column(j), a.K);
            gs[j] = factor<F>(a.gs, column(j), a.K);
            gt[j] = factor<F>(a.own ? nullptr : a.gate, column(j), a.K);
            qs[j] = qu[j] = zero;
        }
    }
    // chunk j of a vector, and of a column sum, to which w times x is added
    const auto vec = [&](const v4f (&held)[HELD], const float *from, int j) {
        if constexpr (FULL) return factor<F>(from, column(j), a.K);
        else return held[j];
    };
    const auto add = [&](v4f (&held)[HELD], int which, int j, const v4f &w, const v4f &x) {
        v4f q;
        if constexpr (FULL) q = sums[(which * NV + j) * T + t];
        else q = held[j];
#pragma unroll
        for (int c = 0; c < 4; ++c) q[c] = __builtin_fmaf(w[c], x[c], q[c]);
        if constexpr (FULL) sums[(which * NV + j) * T + t] = q;
        else held[j] = q;
    };
    for (int64_t base = (int64_t)blockIdx.x * ROWS; base < a.M; base += (int64_t)gridDim.x * ROWS) {
        const int64_t want = base + threadIdx.x / T;
        const bool live = want < a.M;                 // uniform per team
        const int64_t row = live ? want : a.M - 1;
        // a team without a row takes the last one again, and neither adds nor stores it
        const float rs = a.rs[row], ru = a.ru[row];
        v4f d[NV], s[NV], u[NV], in[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = column(j);
            d[j] = take<F>(a.dY + row * a.lddy, col, a.K);
            s[j] = take<F>(a.S + row * a.lds, col, a.K);
            u[j] = take<F>(a.U + row * a.ldu, col, a.K);
            in[j] = zero;
            if (a.dS) in[j] = take<F>(a.dS + row * a.ldds, col, a.K);
            if (a.own && !FULL) gt[j] = take<F>(a.gate + row * a.ldg, col, a.K);
        }
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const v4f g = vec(gs, a.gs, j);
#pragma unroll
            for (int c = 0; c < 4; ++c) s[j][c] *= rs;
            if (ROWS == 1 || live) add(qs, 0, j, d[j], s[j]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                d[j][c] *= g[c];
                dot = __builtin_fmaf(d[j][c], s[j][c], dot);
            }
        }
        dot = row_sum<T>(dot, red, 0) * invk;
        float dot_u = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const v4f g = vec(gu, a.gu, j);
            if constexpr (FULL) gt[j] = factor<F>(a.gate ? a.gate + row * a.ldg : nullptr, column(j), a.K);
            v4f dv;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                d[j][c] = __builtin_fmaf(__builtin_fmaf(-s[j][c], dot, d[j][c]), rs, in[j][c]);   // dS
                u[j][c] *= ru;
                dv[c] = d[j][c] * gt[j][c];
                s[j][c] = dv[c] * g[c];                                                           // h
                dot_u = __builtin_fmaf(s[j][c], u[j][c], dot_u);
            }
            if (ROWS == 1 || live) add(qu, 1, j, a.own ? dv : d[j], u[j]);
        }
        if (a.dU) dot_u = row_sum<T>(dot_u, red, 1) * invk;    // uniform
        else if (T > 64) __syncthreads();                      // red[0] is used again
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int64_t col = column(j);
            v4f o;
            if (a.dgate && a.own) {
                const v4f g = vec(gu, a.gu, j);
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = d[j][c] * u[j][c] * g[c];
                put<ODD>(a.dgate + row * a.lddg, col, a.K, o);
            }
            if (a.dX) {
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = d[j][c] * a.alpha;
                put<ODD>(a.dX + row * a.lddx, col, a.K, o);
            }
            if (a.dU) {
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = __builtin_fmaf(-u[j][c], dot_u, s[j][c]) * ru;
                put<ODD>(a.dU + row * a.lddu, col, a.K, o);
            }
        }
    }
    if (a.ws == nullptr) return;
    // the teams' sums meet in LDS, chunk by chunk, added in team order
    float *out = a.ws + (int64_t)blockIdx.x * 2 * a.K;
#pragma unroll
    for (int j = 0; j < 2 * NV; ++j) {
        v4f q;
        if constexpr (FULL) q = sums[j * T + t];
        else q = j < NV ? qs[j % NV] : qu[j % NV];
        if constexpr (ROWS > 1) {
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 4; ++c) part[threadIdx.x * 4 + c] = q[c];
            __syncthreads();
            if (threadIdx.x >= T) continue;
#pragma unroll
            for (int w = 1; w < ROWS; ++w)
#pragma unroll
                for (int c = 0; c < 4; ++c) q[c] += part[(w * T + t) * 4 + c];
        }
        put<ODD>(out + (j < NV ? 0 : a.K), column(j % NV), a.K, q);
    }
}

// Longer rows: three passes; the column sums live in the workgroup's row of
// the workspace, each column always touched by the same thread.
template <Fit F>
__global__ __launch_bounds__(1024) void block_norm_bwd_long_kernel(BlockNormBwd a) {
    __shared__ float red[2][16];
    constexpr bool ODD = F != WHOLE;
    float *qs = a.ws ? a.ws + (int64_t)blockIdx.x * 2 * a.K : nullptr, *qu = qs ? qs + a.K : nullptr;
    const float invk = 1.f / (float)a.K;
    const auto add = [&](float *to, int64_t col, const v4f &v, bool first) {
        v4f q = {0.f, 0.f, 0.f, 0.f};
        if (!first) q = get<ODD>(to, col, a.K);
#pragma unroll
        for (int c = 0; c < 4; ++c) q[c] += v[c];
        put<ODD>(to, col, a.K, q);
    };
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const float rs = a.rs[row], ru = a.ru[row];
        const float *pd = a.dY + row * a.lddy, *ps = a.S + row * a.lds, *pu = a.U + row * a.ldu;
        const float *pg = a.gate ? a.gate + row * a.ldg : nullptr;
        const float *pi = a.dS ? a.dS + row * a.ldds : nullptr;
        const bool first = row == blockIdx.x;
        float dot = 0.f;
        for (int64_t c0 = 0; c0 < a.K; c0 += 4096) {
            const int64_t col = c0 + threadIdx.x * 4;
            const v4f d = take<F>(pd, col, a.K), s = take<F>(ps, col, a.K), g = factor<F>(a.gs, col, a.K);
            v4f w;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                w[c] = d[c] * (s[c] * rs);
                dot = __builtin_fmaf(g[c], w[c], dot);
            }
            if (qs) add(qs, col, w, first);
        }
        dot = row_sum<1024>(dot, red, 0) * invk;
        // dS of 4 columns
        const auto ds_at = [&](int64_t col) {
            v4f d = take<F>(pd, col, a.K);
            const v4f s = take<F>(ps, col, a.K), g = factor<F>(a.gs, col, a.K);
            v4f in = {0.f, 0.f, 0.f, 0.f};
            if (pi) in = take<F>(pi, col, a.K);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                d[c] = __builtin_fmaf(__builtin_fmaf(-(s[c] * rs), dot, d[c] * g[c]), rs, in[c]);
            return d;
        };
        float dot_u = 0.f;
        for (int64_t c0 = 0; c0 < a.K; c0 += 4096) {
            const int64_t col = c0 + threadIdx.x * 4;
            const v4f d = ds_at(col), u = take<F>(pu, col, a.K), gu = factor<F>(a.gu, col, a.K);
            const v4f gt = factor<F>(pg, col, a.K);
            v4f w;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float dv = d[c] * gt[c], xu = u[c] * ru;
                w[c] = (a.own ? dv : d[c]) * xu;
                dot_u = __builtin_fmaf(dv * gu[c], xu, dot_u);
            }
            if (qu) add(qu, col, w, first);
        }
        dot_u = row_sum<1024>(dot_u, red, 1) * invk;
        for (int64_t c0 = 0; c0 < a.K; c0 += 4096) {
            const int64_t col = c0 + threadIdx.x * 4;
            const v4f d = ds_at(col), u = take<F>(pu, col, a.K), gu = factor<F>(a.gu, col, a.K);
            const v4f gt = factor<F>(pg, col, a.K);
            v4f o;
            if (a.dgate && a.own) {
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = d[c] * (u[c] * ru) * gu[c];
                put<ODD>(a.dgate + row * a.lddg, col, a.K, o);
            }
            if (a.dX) {
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] = d[c] * a.alpha;
                put<ODD>(a.dX + row * a.lddx, col, a.K, o);
            }
            if (a.dU) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    o[c] = __builtin_fmaf(-(u[c] * ru), dot_u, d[c] * gt[c] * gu[c]) * ru;
                put<ODD>(a.dU + row * a.lddu, col, a.K, o);
            }
        }
    }
}

// The workspace's rows added in order, per column: 32 interleaved runs of rows
// with 8 loads in flight, then the runs.  blockIdx.y picks the sum: that of
// dgamma_s, or q of dgamma_u and dgate.
constexpr int RUNS = 32, INFLIGHT = 8;

__global__ __launch_bounds__(32 * RUNS) void block_norm_sums_kernel(int n, BlockNormBwd a) {
    __shared__ float red[RUNS][33];
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    const bool q = blockIdx.y == 1;
    if (q ? !a.dgu && !(a.dgate && !a.own) : !a.dgs) return;      // uniform
    for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < a.K; c0 += (int64_t)gridDim.x * 32) {
        const int64_t col = c0 + tx;
        const float *p = a.ws + (q ? a.K : 0) + min(col, (int64_t)a.K - 1);
        float sum = 0.f;
        for (int i = ty; i < n; i += RUNS * INFLIGHT) {
            float v[INFLIGHT];
#pragma unroll
            for (int k = 0; k < INFLIGHT; ++k) v[k] = p[(int64_t)min(i + RUNS * k, n - 1) * 2 * a.K];
#pragma unroll
            for (int k = 0; k < INFLIGHT; ++k) sum += i + RUNS * k < n ? v[k] : 0.f;
        }
        red[ty][tx] = sum;
        __syncthreads();
        if (ty == 0 && col < a.K) {
#pragma unroll
            for (int y = 1; y < RUNS; ++y) sum += red[y][tx];
            const auto store = [&](float *to, float v) { to[col] = a.accumulate ? to[col] + v : v; };
            if (!q) {
                store(a.dgs, sum);
            } else {
                if (a.dgu) store(a.dgu, a.gate && !a.own ? a.gate[col] * sum : sum);
                if (a.dgate && !a.own) store(a.dgate, a.gu ? a.gu[col] * sum : sum);
            }
        }
        __syncthreads();
    }
}

constexpr int MAX_GROUPS = 1 << 20;

template <int T, int NV, Fit F>
hipError_t norm(const BlockNorm &a, hipStream_t s) {
    constexpr int ROWS = group_threads<T>() / T;
    const int64_t groups = ((int64_t)a.M + ROWS - 1) / ROWS;
    const dim3 grid((unsigned)(groups < MAX_GROUPS ? groups : MAX_GROUPS));
    return a.Q ? launch(block_norm_kernel<T, NV, F, true>, grid, dim3(group_threads<T>()), s, a)
               : launch(block_norm_kernel<T, NV, F, false>, grid, dim3(group_threads<T>()), s, a);
}

// Threads and chunks per row (16 bytes per chunk) by the row's length: as few idle
// threads as there can be, and no more than two chunks, whose loads are all in
// flight at once (us, fp32 / 8 bits: 100000 x 64 21 / 20 on 16 threads, 37 / 40 on a
// wave; 30000 x 100 11.4 / 10.0 on 32, 14.8 / 14.9; 65536 x 256 46 / 41, on two
// chunks 51 / 50; 32768 x 768 81 / 75 on 256 threads, 85 / 82 on a wave with four
// chunks, 104 / 112 on 256 threads with two; 8192 x 4096 115 / 93 on 512, 136 / 146 on
// 1,024 threads; 1024 x 16384 66 / 53 read twice, 57 / 65 on four chunks of 1,024
// threads).
template <Fit F>
hipError_t norm_of(const BlockNorm &a, hipStream_t s) {
    if (a.K <= 64) return norm<16, 1, F>(a, s);
    if (a.K <= 128) return norm<32, 1, F>(a, s);
    if (a.K <= 256) return norm<64, 1, F>(a, s);
    if (a.K <= 512) return norm<64, 2, F>(a, s);
    if (a.K <= 1024) return norm<256, 1, F>(a, s);
    if (a.K <= 2048) return norm<256, 2, F>(a, s);
    if (a.K <= 4096) return norm<512, 2, F>(a, s);
    if (a.K <= 8192) return norm<1024, 2, F>(a, s);
    const dim3 grid((unsigned)(a.M < MAX_GROUPS ? a.M : MAX_GROUPS));
    return a.Q ? launch(block_norm_long_kernel<F, true>, grid, dim3(1024), s, a)
               : launch(block_norm_long_kernel<F, false>, grid, dim3(1024), s, a);
}

// The same for the gradients (100000 x 64 31 us, on a wave 72), and how many workgroups (rows of the workspace)
// they take: two per CU, one of 1,024 threads (16384 x 2048: 153 us on 512, 159 on
// 768, 162 on 1,024; 4096 x 8192: 161 on 256, 170 on 512, 182 on 1,024).  Up to
// 16,384 columns rows are read once (2048 x 12288: 145 us, in three passes 245).
template <int T, int NV, Fit F>
hipError_t norm_bwd(const BlockNormBwd &a, int &groups, hipStream_t s) {
    constexpr int ROWS = group_threads<T>() / T;
    const int64_t rows = ((int64_t)a.M + ROWS - 1) / ROWS;
    const int most = T == 1024 ? BLOCK_NORM_BWD_GROUPS / 2 : BLOCK_NORM_BWD_GROUPS;
    groups = (int)(rows < most ? rows : most);
    return launch(block_norm_bwd_kernel<T, NV, F>, dim3(groups), dim3(group_threads<T>()), s, a);
}

template <Fit F>
hipError_t norm_bwd_of(const BlockNormBwd &a, int &groups, hipStream_t s) {
    if (a.K <= 64) return norm_bwd<16, 1, F>(a, groups, s);
    if (a.K <= 128) return norm_bwd<32, 1, F>(a, groups, s);
    if (a.K <= 256) return norm_bwd<64, 1, F>(a, groups, s);
    if (a.K <= 512) return norm_bwd<64, 2, F>(a, groups, s);
    if (a.K <= 1024) return norm_bwd<256, 1, F>(a, groups, s);
    if (a.K <= 2048) return norm_bwd<256, 2, F>(a, groups, s);
    if (a.K <= 4096) return norm_bwd<512, 2, F>(a, groups, s);
    if (a.K <= 8192) return norm_bwd<1024, 2, F>(a, groups, s);
    if (a.K <= 12288) return norm_bwd<1024, 3, F>(a, groups, s);
    if (a.K <= 16384) return norm_bwd<1024, 4, F>(a, groups, s);
    groups = a.M < BLOCK_NORM_BWD_GROUPS ? a.M : BLOCK_NORM_BWD_GROUPS;
    return launch(block_norm_bwd_long_kernel<F>, dim3(groups), dim3(1024), s, a);
}

}  // namespace

hipError_t launch_block_norm(const BlockNorm &a, hipStream_t s) {
    if (a.K < 4) return norm<16, 1, TINY>(a, s);
    return a.K % 4 ? norm_of<CUT>(a, s) : norm_of<WHOLE>(a, s);
}

hipError_t launch_block_norm_bwd(const BlockNormBwd &a, hipStream_t s) {
    int groups = 0;
    if (a.M > 0) {
        const hipError_t e = a.K < 4    ? norm_bwd<16, 1, TINY>(a, groups, s)
                             : a.K % 4 ? norm_bwd_of<CUT>(a, groups, s) : norm_bwd_of<WHOLE>(a, groups, s);
        if (e != hipSuccess) return e;
    }
    if (a.ws == nullptr && a.M > 0) return hipSuccess;
    const int64_t blocks = ((int64_t)a.K + 31) / 32;
    return launch(block_norm_sums_kernel, dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20), 2),
                  dim3(32 * RUNS), s, groups, a);
}

}  // namespace gg
