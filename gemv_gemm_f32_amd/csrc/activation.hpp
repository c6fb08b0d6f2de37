// activation.hpp -- the activations of the dense layers and their
// derivatives, fp32 in and out.
//
// All but ReLU are z times a rising weight p(z) in [0, 1]:
//   GELU (tanh form)  p = (1 + tanh u) / 2 = 1 / (1 + exp(-2u)),
//                     u = sqrt(2/pi) * (z + 0.044715 z^3)
//   GELU (erf form)   p = (1 + erf(z / sqrt 2)) / 2
//   SiLU              p = 1 / (1 + exp(-z))
// The logistic form of the first has no cancellation for negative z, where
// (1 + tanh u) loses digits.  NaN in gives NaN out; +inf gives +inf; -inf
// meets p = 0 and gives NaN in the three of them (0 in ReLU).
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/gemvgemm.h"

namespace gg {

constexpr float GELU_2C = 1.5957691216057308f;        // 2 sqrt(2/pi)
constexpr float GELU_2CA = 0.07135481627260025f;      // 2 sqrt(2/pi) * 0.044715
constexpr float SQRT_HALF = 0.7071067811865476f;
constexpr float INV_SQRT_2PI = 0.3989422804014327f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == GG_ACT_RELU) return z < 0.f ? 0.f : z;
    if constexpr (ACT == GG_ACT_GELU_TANH)
        return z / (1.f + expf(-z * __builtin_fmaf(GELU_2CA, z * z, GELU_2C)));
    if constexpr (ACT == GG_ACT_GELU_ERF) {
        // erfc keeps the digits of 1 + erf for negative z
        const float p = 0.5f * erfcf(-z * SQRT_HALF);
        return z * p;
    }
    if constexpr (ACT == GG_ACT_SILU) return z / (1.f + expf(-z));
    return z;
}

// d act / dz.  z is first brought into [-100, 100], outside of which every
// derivative has reached its limit, 0 or 1 (to 1e-41 in fp32), so no factor
// overflows and infinities give the limits; NaN stays NaN.  ReLU's
// derivative at 0 is 0.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == GG_ACT_NONE) return 1.f;
    if constexpr (ACT == GG_ACT_RELU) return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
    z = z > 100.f ? 100.f : (z < -100.f ? -100.f : z);
    if constexpr (ACT == GG_ACT_GELU_TANH) {
        const float zz = z * z;
        const float p = 1.f / (1.f + expf(-z * __builtin_fmaf(GELU_2CA, zz, GELU_2C)));
        return __builtin_fmaf(p * (1.f - p), z * __builtin_fmaf(3.f * GELU_2CA, zz, GELU_2C), p);
    }
    if constexpr (ACT == GG_ACT_GELU_ERF) {
        const float p = 0.5f * erfcf(-z * SQRT_HALF);
        return __builtin_fmaf(z * INV_SQRT_2PI, expf(-0.5f * z * z), p);
    }
    const float p = 1.f / (1.f + expf(-z));
    return __builtin_fmaf(p * (1.f - p), z, p);
}

// f(std::integral_constant<int, ACT>) for the activation `act`; one uniform
// branch outside the element loops.
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
    case GG_ACT_RELU: f(std::integral_constant<int, GG_ACT_RELU>{}); break;
    case GG_ACT_GELU_TANH: f(std::integral_constant<int, GG_ACT_GELU_TANH>{}); break;
    case GG_ACT_GELU_ERF: f(std::integral_constant<int, GG_ACT_GELU_ERF>{}); break;
    case GG_ACT_SILU: f(std::integral_constant<int, GG_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, GG_ACT_NONE>{}); break;
    }
}

}  // namespace gg
