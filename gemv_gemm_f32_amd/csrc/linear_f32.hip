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

namespace gg {
namespace {

struct Layer {
    const float *bias;   // NULL: none
    const float *R;      // NULL: none; may be C itself (each element is read
    int64_t ldr;         //   by the lane that then writes it)
    float *Z;            // NULL: not kept
    int64_t ldz;
    int act;

    // The N sums of one column that a lane holds: acc[r] belongs to row
    // row(r), if mine(r).  The residuals are fetched before any of them is
    // used, so their latencies overlap.
    template <int N, class Acc, class Row, class Mine>
    __device__ __forceinline__ void block(const Acc &acc, int col, int M, float *C, int64_t ldc,
                                          Row row, Mine mine) const {
        const float b = bias ? bias[col] : 0.f;
        float res[N];
#pragma unroll
        for (int r = 0; r < N; ++r) {
            res[r] = 0.f;
            if (R && mine(r) && row(r) < M) res[r] = R[(int64_t)row(r) * ldr + col];
        }
        with_act(act, [&](auto a) {
#pragma unroll
            for (int r = 0; r < N; ++r) {
                if (!mine(r) || row(r) >= M) continue;
                const float z = acc[r] + b;
                if (Z) Z[(int64_t)row(r) * ldz + col] = z;
                const float y = act_value<decltype(a)::value>(z);
                C[(int64_t)row(r) * ldc + col] = R ? y + res[r] : y;
            }
        });
    }
};

}  // namespace

hipError_t launch_linear(bool trans_w, int act, int M, int N, int K, const float *X, int64_t ldx,
                         const float *W, int64_t ldw, const float *bias, const float *R,
                         int64_t ldr, float *Z, int64_t ldz, float *Y, int64_t ldy, int num_cus,
                         hipStream_t s) {
    const Layer e{bias, R, ldr, Z, ldz, act};
    const Tiles t = pick_tiles(true, trans_w, M, N, K, X, ldx, W, ldw, num_cus);
    return trans_w ? launch_product<true, true>(t, M, N, K, X, ldx, W, ldw, Y, ldy, e, s)
                   : launch_product<true, false>(t, M, N, K, X, ldx, W, ldw, Y, ldy, e, s);
}

}  // namespace gg
