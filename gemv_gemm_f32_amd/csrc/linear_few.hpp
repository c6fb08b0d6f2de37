// linear_few.hpp -- the fp32 dense layer on few rows of X, for workgroups that
// own ROWS rows (few_nk) or 32 columns (few_kn) of W from n0 on.  x(m) is the
// address of row m of X.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "linear_layer.hpp"
#include "wave.hpp"

namespace gg {
namespace {

// W stored N x K: KW waves share a row of W, a lane takes 4 columns in 256
// (per U chunks in flight) and the same of up to MB rows of X; row sums are
// taken in the wave (wave.hpp) and joined over the waves in order.  ROWS rows
// of W per workgroup.
template <int MB, int KW, int ROWS, class XRow>
__device__ __forceinline__ void few_nk(int M, int N, int K, XRow x, const float *__restrict__ W,
                                       int64_t ldw, float *__restrict__ Y, int64_t ldy,
                                       const Layer &e, int64_t n0) {
    constexpr int U = MB > 4 ? 2 : 4;
    __shared__ float red[ROWS][KW][MB];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = wave / KW, kw = wave % KW;
    const int n = (int)min(n0 + sub, (int64_t)N - 1);
    const float *w = W + (int64_t)n * ldw;
    float acc[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[m] = 0.f;
    // this wave's share of the whole 256-column chunks, then the rest of the
    // row column by column
    const int chunks = K / 256, first = (int)((int64_t)chunks * kw / KW),
              end = (int)((int64_t)chunks * (kw + 1) / KW);
    auto chunk = [&](auto count, int c) {
        constexpr int C = decltype(count)::value;
        v4f wv[C], xv[C][MB];
#pragma unroll
        for (int u = 0; u < C; ++u) {
            const int64_t k = (int64_t)(c + u) * 256 + 4 * lane;
            wv[u] = *reinterpret_cast<const v4f_any *>(w + k);
#pragma unroll
            for (int m = 0; m < MB; ++m)
                xv[u][m] = *reinterpret_cast<const v4f_any *>(x(min(m, M - 1)) + k);
        }
#pragma unroll
        for (int u = 0; u < C; ++u)
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m] = __builtin_fmaf(wv[u][i], xv[u][m][i], acc[m]);
    };
    int c = first;
    for (; c + U <= end; c += U) chunk(std::integral_constant<int, U>{}, c);
    for (; c < end; ++c) chunk(std::integral_constant<int, 1>{}, c);
    if (kw == KW - 1)
        for (int64_t k = (int64_t)chunks * 256 + lane; k < K; k += 64) {
            const float wk = w[k];
#pragma unroll
            for (int m = 0; m < MB; ++m) acc[m] = __builtin_fmaf(wk, x(min(m, M - 1))[k], acc[m]);
        }
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[m] = wave64_sum(acc[m]);
    if (KW > 1) {
        if (lane == 0)
#pragma unroll
            for (int m = 0; m < MB; ++m) red[sub][kw][m] = acc[m];
        __syncthreads();
    }
    if (kw > 0 || n0 + sub >= N || lane >= MB || lane >= M) return;
    float sum = 0.f;                                  // lane m finishes row m
    if (KW > 1) {
#pragma unroll
        for (int i = 0; i < KW; ++i) sum += red[sub][i][lane];
    } else {
#pragma unroll
        for (int m = 0; m < MB; ++m) sum = lane == m ? acc[m] : sum;
    }
    finish(e, sum, lane, n, Y, ldy);
}

// W stored K x N: a workgroup owns 32 columns (128 bytes of a row of W), a
// wave reads 8 rows at a time, 16 bytes per lane, and the KW waves take rows
// in turn.  The 8 rows' sums are joined in the wave, the waves' through LDS in
// order.
template <int MB, int KW, class XRow>
__device__ __forceinline__ void few_kn(int M, int N, int K, XRow x, const float *__restrict__ W,
                                       int64_t ldw, float *__restrict__ Y, int64_t ldy,
                                       const Layer &e, int64_t n0) {
    constexpr int U = MB > 4 ? 4 : 6;                 // loads of W in flight
    __shared__ float red[KW][MB][32];
    const int lane = threadIdx.x & 63, sub = lane >> 3;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t col = n0 + 4 * (lane & 7);
    const int live = (int)min(max((int64_t)N - col, (int64_t)0), (int64_t)4);
    const bool whole = n0 + 32 <= N;                  // uniform
    v4f acc[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[m] = v4f{0.f, 0.f, 0.f, 0.f};
    auto rows = [&](auto count, int64_t k0) {
        constexpr int C = decltype(count)::value;
        v4f wv[C];
        float xv[C][MB];
#pragma unroll
        for (int u = 0; u < C; ++u) {
            const int64_t k = k0 + 8 * KW * u + sub;
            const int64_t kk = min(k, (int64_t)K - 1);
            const float *p = W + kk * ldw + col;
            wv[u] = v4f{0.f, 0.f, 0.f, 0.f};
            if (whole) {
                wv[u] = *reinterpret_cast<const v4f_any *>(p);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < live) wv[u][i] = p[i];
            }
#pragma unroll
            for (int m = 0; m < MB; ++m) xv[u][m] = x(min(m, M - 1))[kk];
        }
#pragma unroll
        for (int u = 0; u < C; ++u)
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                // a row past K adds nothing, whatever the clamped loads hold
                const bool there = k0 + 8 * KW * u + sub < K;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[m][i] = there ? __builtin_fmaf(wv[u][i], xv[u][m], acc[m][i]) : acc[m][i];
            }
    };
    int64_t k0 = 8 * wave;
    for (; k0 + 8 * KW * (U - 1) < K; k0 += 8 * KW * U) rows(std::integral_constant<int, U>{}, k0);
    for (; k0 < K; k0 += 8 * KW) rows(std::integral_constant<int, 1>{}, k0);
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = acc[m][i];
            v += __shfl_xor(v, 8);
            v += __shfl_xor(v, 16);
            v += __shfl_xor(v, 32);
            if (lane < 8) red[wave][m][4 * lane + i] = v;
        }
    __syncthreads();
    for (int t = threadIdx.x; t < 32 * min(M, MB); t += 64 * KW) {
        const int m = t / 32, c = t % 32;
        if (n0 + c >= N) continue;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) sum += red[w][m][c];
        finish(e, sum, m, (int)(n0 + c), Y, ldy);
    }
}

}  // namespace
}  // namespace gg
