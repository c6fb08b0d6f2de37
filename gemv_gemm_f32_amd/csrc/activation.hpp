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
//
// Element passes and epilogues are bound by memory only while an element costs
// a few tens of instructions, so the exponential is the hardware's 2^x (its
// argument's rounding makes a relative error of |t| 2^-23 in exp(t), at most
// 2^-24 in p, where exp(t) counts for p (1 - p)), the quotient a product with
// the hardware's reciprocal (1 step), and erf the rational form of Hastings
// (Abramowitz and Stegun 7.1.26, absolute error 1.5e-7, half of that in p):
// p is within 2^-22 of its value in all three.  With the library's erfc and
// exp the slope of the erf form over 1024 x 4096 took 12.2 us against
// 10.5, and the layer 1024 x 2304 x 768 41.2 against 39.1.
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/gemvgemm.h"

namespace gg {

constexpr float GELU_2C = 1.5957691216057308f;        // 2 sqrt(2/pi)
constexpr float GELU_2CA = 0.07135481627260025f;      // 2 sqrt(2/pi) * 0.044715
constexpr float SQRT_HALF = 0.7071067811865476f;
constexpr float INV_SQRT_2PI = 0.3989422804014327f;

constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float exp_fast(float t) { return __builtin_amdgcn_exp2f(t * LOG2E); }

// 1 / (1 + exp(-t))
__device__ __forceinline__ float logistic(float t) {
    return __builtin_amdgcn_rcpf(1.f + exp_fast(-t));
}

// (1 + erf(z / sqrt 2)) / 2, and exp(-z^2 / 2) on the way
__device__ __forceinline__ float normal_weight(float z, float &gauss) {
    const float a = __builtin_fabsf(z) * SQRT_HALF;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, a, 1.f));
    float q = __builtin_fmaf(1.061405429f, t, -1.453152027f);
    q = __builtin_fmaf(q, t, 1.421413741f);
    q = __builtin_fmaf(q, t, -0.284496736f);
    q = __builtin_fmaf(q, t, 0.254829592f);
    gauss = exp_fast(-a * a);
    const float tail = 0.5f * (q * t) * gauss;         // (1 - erf(a)) / 2
    return z < 0.f ? tail : 1.f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == GG_ACT_RELU) return z < 0.f ? 0.f : z;
    if constexpr (ACT == GG_ACT_GELU_TANH)
        return z * logistic(z * __builtin_fmaf(GELU_2CA, z * z, GELU_2C));
    if constexpr (ACT == GG_ACT_GELU_ERF) {
        float gauss;
        return z * normal_weight(z, gauss);
    }
    if constexpr (ACT == GG_ACT_SILU) return z * logistic(z);
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
        const float p = logistic(z * __builtin_fmaf(GELU_2CA, zz, GELU_2C));
        return __builtin_fmaf(p * (1.f - p), z * __builtin_fmaf(3.f * GELU_2CA, zz, GELU_2C), p);
    }
    if constexpr (ACT == GG_ACT_GELU_ERF) {
        float gauss;
        const float p = normal_weight(z, gauss);
        return __builtin_fmaf(z * INV_SQRT_2PI, gauss, p);
    }
    const float p = logistic(z);
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
