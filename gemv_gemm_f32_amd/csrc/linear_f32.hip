// linear_f32.hip -- fp32 Y = act(X.op(W) + b) + R: the product kernels of
// gemm_f32_tile.hpp with the dense layer's epilogue.
//
// Bias, activation and residual are applied to the sums while they are still
// in the accumulators, so Z = X.op(W) + b and act(Z) never travel to memory
// and back between launches: against a product followed by element-wise
// passes, each of which reads and writes M x N floats, the layer reads R and
// writes Y (and Z, when the backward pass will want it) once.
#include <hip/hip_runtime.h>

#include "gemm_f32_tile.hpp"
#include "kernels.hpp"
#include "linear_few.hpp"

namespace gg {
namespace {

// ---------------------------------------------------------------------------
// Few rows of X: bound by W's way from memory, so W is read once, by as many
// waves as it has rows (or slabs of columns), and no tile is padded (one row
// over 4096 x 4096: 11.6 us, 5.8 TB/s; in tiles 21.0).

template <int MB, int KW, int ROWS>
__global__ __launch_bounds__(64 * KW * ROWS) void linear_few_nk(
    int M, int N, int K, const float *__restrict__ X, int64_t ldx, const float *__restrict__ W,
    int64_t ldw, float *__restrict__ Y, int64_t ldy, Layer e) {
    few_nk<MB, KW, ROWS>(M, N, K, [=](int m) { return X + m * ldx; }, W, ldw, Y, ldy, e,
                         (int64_t)blockIdx.x * ROWS);
}

template <int MB, int KW>
__global__ __launch_bounds__(64 * KW) void linear_few_kn(
    int M, int N, int K, const float *__restrict__ X, int64_t ldx, const float *__restrict__ W,
    int64_t ldw, float *__restrict__ Y, int64_t ldy, Layer e) {
    few_kn<MB, KW>(M, N, K, [=](int m) { return X + m * ldx; }, W, ldw, Y, ldy, e,
                   (int64_t)blockIdx.x * 32);
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
