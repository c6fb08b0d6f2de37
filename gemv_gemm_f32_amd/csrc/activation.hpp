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
// 2^-24 in p, where exp(t) counts for p (1 - p)) and the quotient a product with
// the hardware's reciprocal (1 step): p is within 2^-22 of its value.
//
// The erf form is made of two least-maximum fits of its own (weighted by z and
// by the tail's inverse, found by linear programming in 64 bits):
//   |z| < 1.25:  p = 1/2 + z P(z^2), P of degree 5, within 2^-28.8
//   beyond:      (1 - erf(|z| / sqrt 2)) / 2 = exp(-z^2 / 2) t Q(t) with
//                t = 1 / (1 + 0.4 |z|), Q of degree 6, within 2^-24.3 relative
// so p is within 2^-23 of its value and in the left tail, where p is small,
// within (12 + 2 z^2) 2^-24 relative (to z = -13; 0 where exp(-z^2 / 2) falls
// below 2^-126).
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/gemvgemm.h"

namespace gg {

constexpr float GELU_2C = 1.5957691216057308f;        // 2 sqrt(2/pi)
constexpr float GELU_2CA = 0.07135481627260025f;      // 2 sqrt(2/pi) * 0.044715
constexpr float INV_SQRT_2PI = 0.3989422804014327f;

constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float exp_fast(float t) { return __builtin_amdgcn_exp2f(t * LOG2E); }

// 1 / (1 + exp(-t))
__device__ __forceinline__ float logistic(float t) {
    return __builtin_amdgcn_rcpf(1.f + exp_fast(-t));
}

// (1 + erf(z / sqrt 2)) / 2, and exp(-z^2 / 2) on the way
__device__ __forceinline__ float normal_weight(float z, float &gauss) {
    const float a = __builtin_fabsf(z), zz = z * z;
    gauss = __builtin_amdgcn_exp2f(-0.5f * LOG2E * zz);
    float p = __builtin_fmaf(-6.6448406e-06f, zz, 1.10327375e-04f);
    p = __builtin_fmaf(p, zz, -1.18270947e-03f);
    p = __builtin_fmaf(p, zz, 9.97150037e-03f);
    p = __builtin_fmaf(p, zz, -6.64899871e-02f);
    p = __builtin_fmaf(p, zz, 0.398942262f);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.4f, a, 1.f));
    float q = __builtin_fmaf(6.93908185e-02f, t, -0.189606979f);
    q = __builtin_fmaf(q, t, 0.108559087f);
    q = __builtin_fmaf(q, t, 5.38959317e-02f);
    q = __builtin_fmaf(q, t, 0.139457434f);
    q = __builtin_fmaf(q, t, 0.159035996f);
    q = __builtin_fmaf(q, t, 0.159599349f);
    const float tail = q * t * gauss;
    return a < 1.25f ? __builtin_fmaf(z, p, 0.5f) : z < 0.f ? tail : 1.f - tail;
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
