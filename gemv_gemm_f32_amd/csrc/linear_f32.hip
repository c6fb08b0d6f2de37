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
