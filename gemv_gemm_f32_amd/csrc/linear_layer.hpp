// linear_layer.hpp -- the epilogue of the fp32 dense layer, act(Z) + R with Z
// the finished sum plus the bias: on the tiles of gemm_f32_tile.hpp, and for
// sums that are finished one by one.
#pragma once
#include <hip/hip_runtime.h>

#include "activation.hpp"
#include "gemm_f32_tile.hpp"

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

}  // namespace
}  // namespace gg
