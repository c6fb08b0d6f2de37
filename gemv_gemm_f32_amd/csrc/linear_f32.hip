// linear_f32.hip -- fp32 Y = act(X.op(W) + b) + R: the product kernels of
// gemm_f32_tile.hpp with the dense layer's epilogue.
//
// Bias, activation and residual are applied to the sums while they are still
// in the accumulators, so Z = X.op(W) + b and act(Z) never travel to memory
// and back between launches: against a product followed by element-wise
// passes, each of which reads and writes M x N floats, the layer reads R and
// writes Y (and Z, when the backward pass will want it) once.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "activation.hpp"
#include "gemm_f32_tile.hpp"
#include "kernels.hpp"
#include "wave.hpp"

namespace gg {
namespace {

struct Layer {
    const float *bias;   // NULL: none
    const float *R;      // NULL: none; may be C itself (each element is read
    int64_t ldr;         //   by the lane that then writes it)
    float *Z;            // NULL: not kept
    int64_t ldz;
    int act;

    // the epilogue of the rectangle at (m, n)
    Layer from(int64_t m, int64_t n) const {
        return {bias ? bias + n : nullptr, R ? R + m * ldr + n : nullptr, ldr,
                Z ? Z + m * ldz + n : nullptr, ldz, act};
    }

    // Bias and residuals of one column's NS sums, fetched before the K walk.
    template <int NS>
    struct Fetched {
        float bias, res[NS];
    };
    template <int NS, class Row, class Mine>
    __device__ __forceinline__ void fetch(Fetched<NS> &f, int col, int M, int N, Row row,
                                          Mine mine) const {
        f.bias = bias && col < N ? bias[col] : 0.f;
#pragma unroll
        for (int r = 0; r < NS; ++r) {
            f.res[r] = 0.f;
            if (R && col < N && mine(r) && row(r) < M) f.res[r] = R[(int64_t)row(r) * ldr + col];
        }
    }

    // The NS sums of one column that a lane holds: acc[r] belongs to row
    // row(r), if mine(r).
    template <int NS, class Acc, class Row, class Mine>
    __device__ __forceinline__ void block(const Acc &acc, const Fetched<NS> &f, int col, int M,
                                          float *C, int64_t ldc, Row row, Mine mine) const {
        with_act(act, [&](auto a) {
#pragma unroll
            for (int r = 0; r < NS; ++r) {
                if (!mine(r) || row(r) >= M) continue;
                const float z = acc[r] + f.bias;
                if (Z) Z[(int64_t)row(r) * ldz + col] = z;
                const float y = act_value<decltype(a)::value>(z);
                C[(int64_t)row(r) * ldc + col] = R ? y + f.res[r] : y;
            }
        });
    }
};

// ---------------------------------------------------------------------------
// Few rows of X: bound by W's way from memory, so W is read once, by as many
// waves as it has rows (or slabs of columns), and no tile is padded (one row
// over 4096 x 4096: 11.6 us, 5.8 TB/s; in tiles 21.0).

typedef v4f v4f_any __attribute__((aligned(4)));   // rows may start at any float

// One finished sum.
__device__ __forceinline__ void finish(const Layer &e, float sum, int m, int n, float *Y,
                                       int64_t ldy) {
    const float z = e.bias ? sum + e.bias[n] : sum;
    const float res = e.R ? e.R[(int64_t)m * e.ldr + n] : 0.f;
    if (e.Z) e.Z[(int64_t)m * e.ldz + n] = z;
    float y = 0.f;
    with_act(e.act, [&](auto a) { y = act_value<decltype(a)::value>(z); });
    Y[(int64_t)m * ldy + n] = e.R ? y + res : y;
}

// W stored N x K: KW waves share a row of W, a lane takes 4 columns in 256
// (per U chunks in flight) and the same of up to MB rows of X; row sums are
// taken in the wave (wave.hpp) and joined over the waves in order.  ROWS rows
// of W per workgroup.
template <int MB, int KW, int ROWS>
__global__ __launch_bounds__(64 * KW * ROWS) void linear_few_nk(
    int M, int N, int K, const float *__restrict__ X, int64_t ldx, const float *__restrict__ W,
    int64_t ldw, float *__restrict__ Y, int64_t ldy, Layer e) {
    constexpr int U = MB > 4 ? 2 : 4;
    __shared__ float red[ROWS][KW][MB];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = wave / KW, kw = wave % KW;
    const int n = (int)min((int64_t)blockIdx.x * ROWS + sub, (int64_t)N - 1);
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
                xv[u][m] = *reinterpret_cast<const v4f_any *>(X + min(m, M - 1) * ldx + k);
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
            for (int m = 0; m < MB; ++m) acc[m] = __builtin_fmaf(wk, X[min(m, M - 1) * ldx + k], acc[m]);
        }
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[m] = wave64_sum(acc[m]);
    if (KW > 1) {
        if (lane == 0)
#pragma unroll
            for (int m = 0; m < MB; ++m) red[sub][kw][m] = acc[m];
        __syncthreads();
    }
    if (kw > 0 || (int64_t)blockIdx.x * ROWS + sub >= N || lane >= MB || lane >= M) return;
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
template <int MB, int KW>
__global__ __launch_bounds__(64 * KW) void linear_few_kn(
    int M, int N, int K, const float *__restrict__ X, int64_t ldx, const float *__restrict__ W,
    int64_t ldw, float *__restrict__ Y, int64_t ldy, Layer e) {
    constexpr int U = MB > 4 ? 4 : 6;                 // loads of W in flight
    __shared__ float red[KW][MB][32];
    const int lane = threadIdx.x & 63, sub = lane >> 3;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 32;
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
            for (int m = 0; m < MB; ++m) xv[u][m] = X[min(m, M - 1) * ldx + kk];
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

template <int MB>
hipError_t launch_few(bool trans_w, int M, int N, int K, const float *X, int64_t ldx,
                      const float *W, int64_t ldw, float *Y, int64_t ldy, const Layer &e,
                      int num_cus, hipStream_t s) {
    // A launch has fewer than 2^32 threads: wider outputs take several.
    constexpr int64_t MOST = 1 << 25;
    for (int64_t n = 0; n < N; n += MOST) {
        const int cols = (int)(N - n < MOST ? N - n : MOST);
#define GG_FEW M, cols, K, X, ldx, W + (trans_w ? n * ldw : n), ldw, Y + n, ldy, e.from(0, n)
        const hipError_t st =
            !trans_w ? launch(linear_few_kn<MB, 16>, dim3((cols + 31) / 32), dim3(1024), s, GG_FEW)
            : N >= 8 * num_cus
                ? launch(linear_few_nk<MB, 1, 4>, dim3((cols + 3) / 4), dim3(256), s, GG_FEW)
                : launch(linear_few_nk<MB, 4, 1>, dim3(cols), dim3(256), s, GG_FEW);
        if (st != hipSuccess) return st;
#undef GG_FEW
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_linear(bool trans_w, int act, int M, int N, int K, const float *X, int64_t ldx,
                         const float *W, int64_t ldw, const float *bias, const float *R,
                         int64_t ldr, float *Z, int64_t ldz, float *Y, int64_t ldy, int num_cus,
                         hipStream_t s) {
    const Layer e{bias, R, ldr, Z, ldz, act};
    // Up to 8 rows over W stored N x K, up to 4 over K x N, where every lane
    // reads X at a stride: with 768 columns of X and 2304 of Y, one row takes
    // 3.0 (N x K) and 4.0 us (K x N) against 7.4 and 7.7 in tiles, 4 rows over
    // K x N 6.6 against 7.7, 8 rows 5.6 against 7.4 over N x K but 10.8 against
    // 7.8 over K x N; 16 rows stay in tiles.
    if (M <= (trans_w ? 8 : 4)) {
        if (M == 1) return launch_few<1>(trans_w, M, N, K, X, ldx, W, ldw, Y, ldy, e, num_cus, s);
        if (M == 2) return launch_few<2>(trans_w, M, N, K, X, ldx, W, ldw, Y, ldy, e, num_cus, s);
        if (M <= 4) return launch_few<4>(trans_w, M, N, K, X, ldx, W, ldw, Y, ldy, e, num_cus, s);
        return launch_few<8>(true, M, N, K, X, ldx, W, ldw, Y, ldy, e, num_cus, s);
    }
    const Tiles t = pick_tiles(true, trans_w, M, N, K, X, ldx, W, ldw, num_cus);
    return trans_w ? launch_product<true, true>(t, M, N, K, X, ldx, W, ldw, Y, ldy, e, s)
                   : launch_product<true, false>(t, M, N, K, X, ldx, W, ldw, Y, ldy, e, s);
}

}  // namespace gg
