// gemm_f32.hip -- fp32 C = alpha * op(A).op(B) + beta * C: the kernels of
// gemm_f32_tile.hpp with the scaling, accumulating epilogue.
#include <hip/hip_runtime.h>

#include "gemm_f32_tile.hpp"
#include "kernels.hpp"

namespace gg {
namespace {

// C = alpha * acc, plus beta * C when beta != 0 (C is not read otherwise).
// With alpha = 1 and beta = 0 the stored value is the accumulator itself.
struct ScaleAdd {
    float alpha, beta;

    // the epilogue of the rectangle at (m, n)
    ScaleAdd from(int64_t, int64_t) const { return *this; }

    template <int N>
    struct Fetched {};
    template <int N, class Row, class Mine>
    __device__ __forceinline__ void fetch(Fetched<N> &, int, int, int, Row, Mine) const {}

    // The NS sums of one column that a lane holds: acc[r] belongs to row
    // row(r), if mine(r).
    template <int NS, class Acc, class Row, class Mine>
    __device__ __forceinline__ void block(const Acc &acc, const Fetched<NS> &, int col, int M,
                                          float *C, int64_t ldc, Row row, Mine mine) const {
#pragma unroll
        for (int r = 0; r < NS; ++r) {
            if (!mine(r) || row(r) >= M) continue;
            float *c = C + (int64_t)row(r) * ldc + col;
            float v = alpha * acc[r];
            if (beta != 0.f) v = __builtin_fmaf(beta, *c, v);
            *c = v;
        }
    }
};

}  // namespace

hipError_t launch_gemm(bool ax, bool bx, int M, int N, int K, float alpha, const float *A,
                       int64_t lda, const float *B, int64_t ldb, float beta, float *C,
                       int64_t ldc, int num_cus, hipStream_t s) {
    const Tiles t = pick_tiles(ax, bx, M, N, K, A, lda, B, ldb, num_cus);
    const ScaleAdd e{alpha, beta};
    if (ax && !bx) return launch_product<true, false>(t, M, N, K, A, lda, B, ldb, C, ldc, e, s);   // A.B
    if (!ax && !bx) return launch_product<false, false>(t, M, N, K, A, lda, B, ldb, C, ldc, e, s); // A^T.B
    if (ax && bx) return launch_product<true, true>(t, M, N, K, A, lda, B, ldb, C, ldc, e, s);     // A.B^T
    return launch_product<false, true>(t, M, N, K, A, lda, B, ldb, C, ldc, e, s);                  // A^T.B^T
}

}  // namespace gg
