// row.hpp -- rows of fp32 as the norm kernels hold them: T threads share a row,
// a thread has chunks of 4 columns in registers, sums over the row are wave
// reductions joined through LDS, and a row leaves as fp32 or in 8 bits.
#pragma once
#include <hip/hip_runtime.h>

#include "mx8.hpp"
#include "wave.hpp"

namespace gg {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
// rows may start at any float (or byte): wide accesses without the promise of
// 16-byte alignment
typedef v4f v4f_any __attribute__((aligned(4)));
typedef unsigned u32_any __attribute__((aligned(1)));

constexpr int WG = 256;       // threads of a workgroup, where T <= 256

template <int T>
constexpr int group_threads() { return T > WG ? T : WG; }

// Sum over the T threads that share a row; every one of them receives it.
// `red` holds a float per wave of the workgroup and is used twice, so that
// one barrier per call is enough (`flip` alternates).
template <int T>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int flip) {
    if constexpr (T == 16) return row16_sum(v);
    if constexpr (T == 32) return half32_sum(v);
    v = wave64_sum(v);
    if constexpr (T == 64) return v;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[flip][wave] = v;
    __syncthreads();
    float s = 0.f;
    constexpr int W = T / 64;
    const int first = wave / W * W;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[flip][first + w];
    return s;
}

// 4 columns of a row in one 16-byte access; columns past K read as zeros and
// are not written.  ODD: K is not a multiple of 4 (where it is, a chunk exists
// whole or not at all, and the shorter test costs a sixth less time on small
// batches: 346 x 768 4.3 against 5.2 us).
template <bool ODD>
__device__ __forceinline__ v4f get(const float *row, int64_t col, int K) {
    v4f x = {0.f, 0.f, 0.f, 0.f};
    if (ODD ? col + 4 <= K : col < K) {
        x = *reinterpret_cast<const v4f_any *>(row + col);
    } else if (ODD && col < K) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (col + c < K) x[c] = row[col + c];
    }
    return x;
}

template <bool ODD>
__device__ __forceinline__ void put(float *row, int64_t col, int K, const v4f &x) {
    if (ODD ? col + 4 <= K : col < K) {
        *reinterpret_cast<v4f_any *>(row + col) = x;
    } else if (ODD && col < K) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (col + c < K) row[col + c] = x[c];
    }
}

// 8 bits: 8 neighbouring lanes hold a block of 32 columns and agree on its
// power of two; every lane of the wave takes part (columns past K are zeros).
template <bool ODD>
__device__ __forceinline__ void put_mx8(uint8_t *qrow, uint8_t *erow, int64_t col, int K,
                                        const v4f &y) {
    unsigned top = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) top = max(top, !ODD || col + c < K ? mag(y[c]) : 0u);
    const int e = mx8_exponent(oct_max(!ODD && col >= K ? 0u : top));
    const unsigned q = mx8_pack4(y[0], y[1], y[2], y[3], e);
    if (ODD ? col + 4 <= K : col < K) {
        *reinterpret_cast<u32_any *>(qrow + col) = q;
    } else if (ODD && col < K) {
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (col + c < K) qrow[col + c] = (uint8_t)(q >> (8 * c));
    }
    if (col < K && col % 32 == 0) erow[col / 32] = (uint8_t)e;
}

}  // namespace
}  // namespace gg
