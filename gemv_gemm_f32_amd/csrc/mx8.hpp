// mx8.hpp -- rows in 8 bits: e4m3 values with one power of two (e8m0) per
// block of 32 columns, the form that gfx950's block-scaled matrix
// instructions take.
//
//   value(i, k) = e4m3(Q[i, k]) * 2^(E[i, k/32] - 127)
//
// E is the smallest power that keeps the block's largest magnitude within
// e4m3's 448 (= 1.75 * 2^8), so no value saturates, and dividing by it is
// exact: each value is rounded once, to e4m3's 4 significant bits (nearest,
// ties to even; below 2^-6 of the scale to steps of 2^-9).  E is at least 1,
// which keeps 2^(127 - E) a normal number.  A block that holds a NaN or an
// infinity gets E = 255 (NaN) and bytes 0x7f (NaN).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wave.hpp"

namespace gg {

// The bits of |v|; ordered like the magnitudes, infinity and NaN above all.
__device__ __forceinline__ unsigned mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }

template <int CTRL>
__device__ __forceinline__ unsigned dpp_max(unsigned v) {
    const unsigned o = (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return v > o ? v : o;
}

// Maximum over aligned groups of 8 lanes; every lane receives it.
__device__ __forceinline__ unsigned oct_max(unsigned v) {
    v = dpp_max<DPP_QUAD_XOR1>(v);
    v = dpp_max<DPP_QUAD_XOR2>(v);
    return dpp_max<DPP_ROW_HALF_MIRROR>(v);
}

// Maximum over each 32-lane half of the wave.
__device__ __forceinline__ unsigned half32_max(unsigned v) {
    v = dpp_max<DPP_ROW_MIRROR>(oct_max(v));
    const unsigned o = (unsigned)__builtin_amdgcn_ds_swizzle((int)v, 0x401F);   // lane ^ 16
    return v > o ? v : o;
}

// e8m0 of a block whose largest magnitude has the bits `top`.
__device__ __forceinline__ int mx8_exponent(unsigned top) {
    if (top >= 0x7f800000u) return 255;
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
    return e > 1 ? e : 1;
}

// 2^(127 - E), for E < 255 (E is at most 247 there).
__device__ __forceinline__ float mx8_inverse(int e) {
    return __uint_as_float((unsigned)(254 - e) << 23);
}

// Two and four values of a block as bytes, in the low bits.
__device__ __forceinline__ unsigned mx8_pack2(float a, float b, int e) {
    if (e == 255) return 0x7f7fu;
#if defined(__HIP_DEVICE_COMPILE__)
    const float f = mx8_inverse(e);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(a * f, b * f, 0, false) & 0xffffu;
#else
    return 0;
#endif
}

__device__ __forceinline__ unsigned mx8_pack4(float a, float b, float c, float d, int e) {
    return mx8_pack2(a, b, e) | mx8_pack2(c, d, e) << 16;
}

}  // namespace gg
