// linear_mx8.hip -- Y = act(X8.W^T + b) + R with X8 in 8 bits (mx8.hpp) and W
// as 2-bit or 4-bit codes with one binary16 scale per 64 columns, on gfx950's
// block-scaled matrix instruction.
//
//   w(n, k) = (code - 7.5) s(n, k/64) = (2 code - 15) s/2     (4 bits)
//   w(n, k) = (code - 1.5) s(n, k/64) = (2 code - 3) s/2      (2 bits)
//
// The odd integers up to 15 have 4 significant bits, so 2 code - 15 is an
// e4m3 number exactly: codes become matrix operands without any rounding.
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 rows of x by 32 rows of W
// over 64 columns, the width of one weight scale, and applies x's two powers
// of two itself: registers 0-3 of both half-waves are the columns of the first
// block of 32, whose power lanes 0-31 give, registers 4-7 those of the second,
// whose power lanes 32-63 give.  What is left per weight group is one fp32
// multiply-add per sum with s/2.
// Products are exact in fp32 (4 x 4 significant bits), sums are fp32.
//
// Rows of x are the instruction's A operand (they spread over a lane's 16
// sums), rows of W its B operand: a lane belongs to one output column n, so
// its weight scale is one register and stores of Y run along rows.
//
// Codes reach the lanes as they lie in memory and are expanded there by
// shifts and a byte permutation that looks their e4m3 bytes up; shifting
// yields them in the order 0, 2, 4, 6, 1, 3, 5, 7 (4 bits) or 0, 4, 8, 12, 1,
// 5, ... (2 bits), and x's bytes are permuted the same way, since a sum over
// k may be taken in any order as long as both operands agree.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "activation.hpp"
#include "kernels.hpp"
#include "mx8.hpp"

namespace gg {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));

__device__ __forceinline__ unsigned perm(unsigned hi, unsigned lo, unsigned sel) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_perm(hi, lo, sel);
#else
    return 0;
#endif
}

// Four 4-bit codes, one per byte, as the e4m3 bytes of 15 - 2 code: the
// magnitudes 1, 3, ..., 15 are looked up at code mod 8 (upper codes) or its
// complement, bit 3 becomes the sign.  The caller's scale is negative.
__device__ __forceinline__ unsigned e4m3_of_4bit(unsigned c) {
    const unsigned up = c & 0x08080808u;
    const unsigned seven = up - (up >> 3);              // 7 in bytes of codes >= 8
    const unsigned idx = (c ^ ~seven) & 0x07070707u;
    return perm(0x57555351u, 0x4E4A4438u, idx) | up << 4;
}

// Four 2-bit codes, one per byte, as the e4m3 bytes of 2 code - 3.
__device__ __forceinline__ unsigned e4m3_of_2bit(unsigned c) {
    return perm(0, 0x4438B8C4u, c);
}

template <int BITS>
constexpr float code_scale() { return BITS == 4 ? -0.5f : 0.5f; }

// Half-wave h has loaded the 32 codes of block h (BITS dwords); afterwards it
// has the h-th 16 of block 0 in the lower dwords and of block 1 in the upper.
template <int BITS>
__device__ __forceinline__ void deal(unsigned (&w)[BITS]) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) {
        const auto p = __builtin_amdgcn_permlane32_swap(w[i], w[i + BITS / 2], false, false);
        w[i] = p[0];
        w[i + BITS / 2] = p[1];
    }
#endif
}

// The 32 codes of one lane (BITS dwords) as a matrix operand.
template <int BITS>
__device__ __forceinline__ v8i expand(const unsigned (&w)[BITS]) {
    v8i o;
    if constexpr (BITS == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[2 * j] = (int)e4m3_of_4bit(w[j] & 0x0F0F0F0Fu);
            o[2 * j + 1] = (int)e4m3_of_4bit(w[j] >> 4 & 0x0F0F0F0Fu);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[4 * j + i] = (int)e4m3_of_2bit(w[j] >> (2 * i) & 0x03030303u);
    }
    return o;
}

// 32 bytes of x in the order of expand's codes.
template <int BITS>
__device__ __forceinline__ v8i shuffle(const unsigned (&x)[8]) {
    v8i o;
    if constexpr (BITS == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[2 * j] = (int)perm(x[2 * j + 1], x[2 * j], 0x06040200u);
            o[2 * j + 1] = (int)perm(x[2 * j + 1], x[2 * j], 0x07050301u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const unsigned *d = x + 4 * j;
            const unsigned a0 = perm(d[1], d[0], 0x05010400u), b0 = perm(d[3], d[2], 0x05010400u);
            const unsigned a1 = perm(d[1], d[0], 0x07030602u), b1 = perm(d[3], d[2], 0x07030602u);
            o[4 * j] = (int)perm(b0, a0, 0x05040100u);
            o[4 * j + 1] = (int)perm(b0, a0, 0x07060302u);
            o[4 * j + 2] = (int)perm(b1, a1, 0x05040100u);
            o[4 * j + 3] = (int)perm(b1, a1, 0x07060302u);
        }
    }
    return o;
}

__device__ __forceinline__ v16f mfma(const v8i &a, const v8i &b, int scale_a) {
    const v16f zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, zero, 0, 0, 0, scale_a, 0, 127);
#else
    return zero;
#endif
}

// N bytes from p, of which `have` exist; the rest reads as zeros.
template <int N>
__device__ __forceinline__ void load_bytes(unsigned (&d)[N / 4], const uint8_t *p, int have) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        unsigned v = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
            if (4 * i + b < have) v |= (unsigned)p[4 * i + b] << (8 * b);
        d[i] = v;
    }
}

// What a finished sum becomes.  All 64 lanes call it together: the half-wave
// shares a token, its lanes are 32 neighbouring columns n.
__device__ __forceinline__ float finish(const PackedLinear &a, float sum, int64_t tok, int n,
                                        float bias, bool live) {
    float y = 0.f;
    with_act(a.act, [&](auto t) { y = act_value<decltype(t)::value>(sum + bias); });
    if (a.R && live) y += a.R[tok * a.ldr + n];
    if (a.Y && live) a.Y[tok * a.ldy + n] = y;
    if (a.Y8) {
        const int e = mx8_exponent(half32_max(live ? mag(y) : 0u));
        if (live) {
            a.Y8[tok * a.ldy8 + n] = (uint8_t)mx8_pack2(y, 0.f, e);
            if (n % 32 == 0) a.YE[tok * a.ldye + n / 32] = (uint8_t)e;
        }
    }
    return y;
}

// Few rows: a workgroup owns 32 columns n and 32 rows of x, its KS waves
// share the weight groups in runs of RUN, and their sums meet in LDS, added
// in wave order.  WIDE: x and codes are loaded 16 (2-bit codes: 8) bytes at
// a time; else, and in a last group that K cuts short, byte by byte.
constexpr int KS = 8, RUN = 4;

template <int BITS, bool WIDE>
__global__ __launch_bounds__(64 * KS) void packed_rows_kernel(PackedLinear a) {
    __shared__ float red[KS][16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, l32 = lane & 31;
    const int64_t m0 = (int64_t)blockIdx.y * 32;
    const int n0 = blockIdx.x * 32;
    const int64_t tok = min(m0 + l32, (int64_t)a.M - 1);
    const int64_t nrow = min(n0 + l32, a.N - 1);
    const uint8_t *px = a.X + tok * a.ldx, *pe = a.XE + tok * a.ldxe;
    const uint8_t *pq = a.Q + nrow * a.ldq;
    const uint16_t *ps = a.S + nrow * a.lds;
    const int groups = (int)(((int64_t)a.K + 63) / 64);
    constexpr int CB = 4 * BITS;                      // bytes of 32 codes

    v16f acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.f;
    for (int g0 = wave * RUN; g0 < groups; g0 += KS * RUN) {
        unsigned w[RUN][BITS], x[RUN][8];
        int e[RUN];
        float s[RUN];
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            const int g = min(g0 + i, groups - 1);
            const int k = 64 * g + 32 * h;            // the codes this lane loads
            const int have = min(max(a.K - k, 0), 32);
            const int kx = 64 * g + 16 * h;           // and its bytes of x: 16 here,
            const int left = a.K - kx;                // 16 from kx + 32
            s[i] = g0 + i < groups ? (float)__builtin_bit_cast(_Float16, ps[g]) * code_scale<BITS>() : 0.f;
            e[i] = have > 0 ? pe[2 * g + h] : 127;
            if (WIDE && have == 32) {
                if constexpr (BITS == 4) {
                    const v4u q = *reinterpret_cast<const v4u *>(pq + (k >> 1));
#pragma unroll
                    for (int d = 0; d < 4; ++d) w[i][d] = q[d];
                } else {
                    const v2u q = *reinterpret_cast<const v2u *>(pq + (k >> 2));
                    w[i][0] = q[0];
                    w[i][1] = q[1];
                }
            } else {
                load_bytes<CB>(w[i], pq + (int64_t)k * BITS / 8, (have * BITS + 7) / 8);
            }
            if (WIDE && left >= 48) {
                const v4u x0 = *reinterpret_cast<const v4u *>(px + kx);
                const v4u x1 = *reinterpret_cast<const v4u *>(px + kx + 32);
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    x[i][d] = x0[d];
                    x[i][4 + d] = x1[d];
                }
            } else {
                unsigned t[4];
                load_bytes<16>(t, px + kx, left);
#pragma unroll
                for (int d = 0; d < 4; ++d) x[i][d] = t[d];
                load_bytes<16>(t, px + kx + 32, left - 32);
#pragma unroll
                for (int d = 0; d < 4; ++d) x[i][4 + d] = t[d];
            }
        }
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            deal<BITS>(w[i]);
            const v16f p = mfma(shuffle<BITS>(x[i]), expand<BITS>(w[i]), e[i]);
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (g0 + i < groups) acc[r] = __builtin_fmaf(p[r], s[i], acc[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) red[wave][r][lane] = acc[r];
    __syncthreads();
    const int n = n0 + l32;
    const float bias = a.bias && n < a.N ? a.bias[n] : 0.f;
#pragma unroll
    for (int i = 0; i < 16 / KS; ++i) {
        const int r = wave * (16 / KS) + i;
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < KS; ++w) sum += red[w][r][lane];
        const int64_t t = m0 + 8 * (r >> 2) + 4 * h + (r & 3);
        finish(a, sum, t, n, bias, t < a.M && n < a.N);
    }
}

template <int BITS>
hipError_t launch_rows(const PackedLinear &a, hipStream_t s) {
    const auto al = [](const void *p, int64_t ld, int64_t b) {
        return reinterpret_cast<uintptr_t>(p) % b == 0 && ld % b == 0;
    };
    const bool wide = al(a.X, a.ldx, 16) && al(a.Q, a.ldq, 4 * BITS);
    const int64_t nb = ((int64_t)a.N + 31) / 32, mb = ((int64_t)a.M + 31) / 32;
    if (mb > 65535 || nb * mb * 64 * KS > UINT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)nb, (unsigned)mb);
    return launch(wide ? packed_rows_kernel<BITS, true> : packed_rows_kernel<BITS, false>, grid,
                  dim3(64 * KS), s, a);
}

}  // namespace

hipError_t launch_packed_linear(int bits, const PackedLinear &a, int num_cus, hipStream_t s) {
    (void)num_cus;
    return bits == 2 ? launch_rows<2>(a, s) : launch_rows<4>(a, s);
}

}  // namespace gg
