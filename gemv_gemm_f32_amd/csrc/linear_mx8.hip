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
typedef float v4f __attribute__((ext_vector_type(4)));
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

// 16 bytes of x in the order of expand's codes.
template <int BITS>
__device__ __forceinline__ v4u shuffle16(const v4u &d) {
    if constexpr (BITS == 4)
        return v4u{perm(d[1], d[0], 0x06040200u), perm(d[1], d[0], 0x07050301u),
                   perm(d[3], d[2], 0x06040200u), perm(d[3], d[2], 0x07050301u)};
    const unsigned a0 = perm(d[1], d[0], 0x05010400u), b0 = perm(d[3], d[2], 0x05010400u);
    const unsigned a1 = perm(d[1], d[0], 0x07030602u), b1 = perm(d[3], d[2], 0x07030602u);
    return v4u{perm(b0, a0, 0x05040100u), perm(b0, a0, 0x07060302u),
               perm(b1, a1, 0x05040100u), perm(b1, a1, 0x07060302u)};
}

template <int BITS>
__device__ __forceinline__ v8i shuffle(const unsigned (&x)[8]) {
    const v4u lo = shuffle16<BITS>(v4u{x[0], x[1], x[2], x[3]});
    const v4u hi = shuffle16<BITS>(v4u{x[4], x[5], x[6], x[7]});
    return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// A: x (its powers of two in byte SEL of scale_a), B: W (unscaled); C = 0.
template <int SEL>
__device__ __forceinline__ v16f mfma(const v8i &a, const v8i &b, int scale_a) {
    const v16f zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, zero, 0, 0, SEL, scale_a, 0, 127);
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

// The same for a BM x BN tile of sums at (m0, n0) that the 256 threads read
// back 4 columns at a time: at(row, col) gives 4 sums.
template <int BM, int BN, class At>
__device__ __forceinline__ void finish_tile(const PackedLinear &a, int64_t m0, int64_t n0, int tid,
                                            At at) {
    constexpr int PER_ROW = BN / 4;                    // threads along a row
    const int col = tid % PER_ROW * 4;
    const int64_t n = n0 + col;
    const int live = (int)min(max((int64_t)a.N - n, (int64_t)0), (int64_t)4);
    const auto wide = [](const void *p, int64_t ld, int bytes) {
        return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * 4 % bytes == 0;
    };
    // uniform: whole 16-byte accesses
    const bool vr = n0 + BN <= a.N && wide(a.R, a.ldr, 16), vy = n0 + BN <= a.N && wide(a.Y, a.ldy, 16);
    const bool v8 = n0 + BN <= a.N && reinterpret_cast<uintptr_t>(a.Y8) % 4 == 0 && a.ldy8 % 4 == 0;
    v4f bias = {0.f, 0.f, 0.f, 0.f};
    if (a.bias)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < live) bias[c] = a.bias[n + c];
    with_act(a.act, [&](auto act) {
        constexpr int ROWS = 256 / PER_ROW;            // rows at a time
#pragma unroll 4
        for (int i = 0; i < BM / ROWS; ++i) {
            const int row = tid / PER_ROW + ROWS * i;
            const int64_t m = m0 + row;
            v4f y = at(row, col);
            const int w = m < a.M ? live : 0;          // columns to store
            v4f res = {0.f, 0.f, 0.f, 0.f};
            if (a.R) {
                const float *p = a.R + m * a.ldr + n;
                if (vr && w == 4) {
                    res = *reinterpret_cast<const v4f *>(p);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c < w) res[c] = p[c];
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                y[c] = act_value<decltype(act)::value>(y[c] + bias[c]);
                if (a.R) y[c] += res[c];
            }
            if (a.Y) {
                float *p = a.Y + m * a.ldy + n;
                if (vy && w == 4) {
                    *reinterpret_cast<v4f *>(p) = y;
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c < w) p[c] = y[c];
                }
            }
            if (a.Y8) {
                unsigned top = 0;                      // 8 lanes hold a block of 32
#pragma unroll
                for (int c = 0; c < 4; ++c) top = max(top, c < w ? mag(y[c]) : 0u);
                const int e = mx8_exponent(oct_max(top));
                const unsigned q = mx8_pack4(y[0], y[1], y[2], y[3], e);
                uint8_t *p = a.Y8 + m * a.ldy8 + n;
                if (v8 && w == 4) {
                    *reinterpret_cast<unsigned *>(p) = q;
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c < w) p[c] = (uint8_t)(q >> (8 * c));
                }
                if (w > 0 && n % 32 == 0) a.YE[m * a.ldye + n / 32] = (uint8_t)e;
            }
        }
    });
}

// Up to 32 rows: a workgroup owns 32 columns n, its KS waves
// share the weight groups in runs of RUN, and their sums meet in LDS, added
// in wave order.  WIDE: x and codes are loaded 16 (2-bit codes: 8) bytes at
// a time; else, and in a last group that K cuts short, byte by byte.
constexpr int KS = 8, RUN = 4;

template <int BITS, bool WIDE>
__global__ __launch_bounds__(64 * KS) void packed_rows_kernel(PackedLinear a) {
    __shared__ float red[KS][16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, l32 = lane & 31;
    constexpr int64_t m0 = 0;
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
            const v16f p = mfma<0>(shuffle<BITS>(x[i]), expand<BITS>(w[i]), e[i]);
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

// ---------------------------------------------------------------------------
// Many rows: a workgroup of 4 waves owns BM rows of x by 128 columns n and
// walks k in steps of 128 (two weight groups), double-buffered in LDS.
//
//  * Codes are expanded once per workgroup, on their way into LDS, and then
//    feed the BM / 32 row blocks; x's bytes are permuted on the same way.
//  * LDS rows hold 128 bytes, 8 chunks of 16; chunk c of row r lies at slot
//    c ^ (r mod 8), so that the 16-byte fragment reads of 8 neighbouring
//    rows, and the writes, meet no bank twice.
//  * The next step's loads are in flight while this step's fragments are
//    multiplied; one barrier per step.
//  * The finished sums pass through LDS, so that bias, residual and the
//    stores of Y run along rows, 16 bytes per lane.
constexpr int BN = 128, STEP = 128;

// Chunk `c` (16 bytes) of a row of `n` bytes at p, zeros past its end.
template <bool WIDE>
__device__ __forceinline__ v4u load_chunk(const uint8_t *p, int64_t at, int64_t n) {
    if (WIDE && at + 16 <= n) return *reinterpret_cast<const v4u *>(p + at);
    unsigned d[4];
    load_bytes<16>(d, p + at, (int)min(max(n - at, (int64_t)0), (int64_t)16));
    return v4u{d[0], d[1], d[2], d[3]};
}

template <int BM, int BITS, bool WIDE>
__global__ __launch_bounds__(256, 2) void packed_tile_kernel(PackedLinear a, int tiles_m) {
    constexpr int IB = BM / 64, JB = 2;               // 32 x 32 blocks per wave
    constexpr int XC = BM * 8 / 256;                  // chunks of x per thread
    constexpr int CODES = 64 / BITS * 2;              // codes per 16-byte chunk: 32, 64
    constexpr int WPR = STEP / CODES;                 // code chunks per row and step: 4, 2
    constexpr int WC = BN * WPR / 256;                // code chunks per thread: 2, 1
    constexpr int XBYTES = BM * STEP, WBYTES = BN * STEP, STAGE = XBYTES + WBYTES;
    constexpr int TILE = BM * BN * 4;                 // the finished sums
    constexpr int SMEM = 2 * STAGE > TILE ? 2 * STAGE : TILE;
    __shared__ __attribute__((aligned(16))) char smem[SMEM];
    __shared__ unsigned scales[2][BM + BN];           // x: 4 e8m0 bytes, W: 2 halves per step

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h = lane >> 5, l32 = lane & 31;
    int t = blockIdx.x;
    if ((gridDim.x & 7) == 0) t = (t & 7) * (gridDim.x >> 3) + (t >> 3);   // runs per XCD
    const int64_t m0 = (int64_t)(t % tiles_m) * BM;
    const int64_t n0 = (int64_t)(t / tiles_m) * BN;
    const int wm = (wave >> 1) * (BM / 2), wn = (wave & 1) * 64;

    const uint8_t *px[XC], *pw[WC];
#pragma unroll
    for (int i = 0; i < XC; ++i) px[i] = a.X + min(m0 + tid / 8 + 32 * i, (int64_t)a.M - 1) * a.ldx;
#pragma unroll
    for (int i = 0; i < WC; ++i)
        pw[i] = a.Q + min(n0 + tid / WPR + 256 / WPR * i, (int64_t)a.N - 1) * a.ldq;
    // threads below BM fetch a row's powers of two, the next BN a row's scales
    const bool fetch_e = tid < BM, fetch_s = tid >= 256 - BN;
    const uint8_t *pe = a.XE + min(m0 + (fetch_e ? tid : 0), (int64_t)a.M - 1) * a.ldxe;
    const uint16_t *ps = a.S + min(n0 + (fetch_s ? tid - (256 - BN) : 0), (int64_t)a.N - 1) * a.lds;
    const int64_t kb = ((int64_t)a.K * BITS + 7) / 8;
    const int64_t eb = ((int64_t)a.K + 31) / 32, sb = ((int64_t)a.K + 63) / 64;

    v4u xr[XC], wr[WC];
    unsigned er = 0, sr = 0;
    auto load = [&](int64_t k0) {
#pragma unroll
        for (int i = 0; i < XC; ++i) xr[i] = load_chunk<WIDE>(px[i], k0 + 16 * (tid % 8), a.K);
#pragma unroll
        for (int i = 0; i < WC; ++i)
            wr[i] = load_chunk<WIDE>(pw[i], k0 * BITS / 8 + 16 * (tid % WPR), kb);
        if (fetch_e) {
            const int64_t b = k0 / 32;
            if (WIDE && b + 4 <= eb) {
                er = *reinterpret_cast<const unsigned *>(pe + b);
            } else {
                er = 0;
                for (int i = 0; i < 4; ++i) er |= (b + i < eb ? (unsigned)pe[b + i] : 127u) << (8 * i);
            }
        }
        if (fetch_s) {
            const int64_t g = k0 / 64;
            if (WIDE && g + 2 <= sb) sr = *reinterpret_cast<const unsigned *>(ps + g);
            else sr = (unsigned)ps[g] | (g + 1 < sb ? (unsigned)ps[g + 1] << 16 : 0u);
        }
    };
    auto slot = [](int row, int c) { return row * STEP + ((c ^ (row & 7)) * 16); };
    auto store = [&](int buf) {
        char *xs = smem + buf * STAGE, *ws = xs + XBYTES;
#pragma unroll
        for (int i = 0; i < XC; ++i)
            *reinterpret_cast<v4u *>(xs + slot(tid / 8 + 32 * i, tid % 8)) = shuffle16<BITS>(xr[i]);
#pragma unroll
        for (int i = 0; i < WC; ++i) {
            const int row = tid / WPR + 256 / WPR * i;
#pragma unroll
            for (int c = 0; c < CODES / 32; ++c) {
                unsigned w[BITS];
#pragma unroll
                for (int d = 0; d < BITS; ++d) w[d] = wr[i][c * BITS + d];
                const v8i o = expand<BITS>(w);
                const int c0 = (tid % WPR) * (CODES / 16) + 2 * c;
                *reinterpret_cast<v4u *>(ws + slot(row, c0)) =
                    v4u{(unsigned)o[0], (unsigned)o[1], (unsigned)o[2], (unsigned)o[3]};
                *reinterpret_cast<v4u *>(ws + slot(row, c0 + 1)) =
                    v4u{(unsigned)o[4], (unsigned)o[5], (unsigned)o[6], (unsigned)o[7]};
            }
        }
        if (fetch_e) scales[buf][tid] = er;
        if (fetch_s) scales[buf][BM + tid - (256 - BN)] = sr;
    };
    // an operand of group g: chunks 4g + h and 4g + 2 + h of the lane's row
    auto frag = [&](const char *base, int row, int g) {
        const v4u lo = *reinterpret_cast<const v4u *>(base + slot(row, 4 * g + h));
        const v4u hi = *reinterpret_cast<const v4u *>(base + slot(row, 4 * g + 2 + h));
        return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                   (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    };

    v16f acc[IB][JB];
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    if (a.K > 0) {
        load(0);
        store(0);
        __syncthreads();
    }
    int buf = 0;
    for (int64_t k0 = 0; k0 < a.K; k0 += STEP, buf ^= 1) {
        const bool more = k0 + STEP < a.K;
        if (more) load(k0 + STEP);
        const char *xs = smem + buf * STAGE, *ws = xs + XBYTES;
        unsigned e[IB], s2[JB];
#pragma unroll
        for (int i = 0; i < IB; ++i) e[i] = scales[buf][wm + 32 * i + l32] >> (8 * h);
#pragma unroll
        for (int j = 0; j < JB; ++j) s2[j] = scales[buf][BM + wn + 32 * j + l32];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            v8i fx[IB], fw[JB];
#pragma unroll
            for (int i = 0; i < IB; ++i) fx[i] = frag(xs, wm + 32 * i + l32, g);
#pragma unroll
            for (int j = 0; j < JB; ++j) fw[j] = frag(ws, wn + 32 * j + l32, g);
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                const float s = (float)__builtin_bit_cast(_Float16, (uint16_t)(s2[j] >> (16 * g)));
#pragma unroll
                for (int i = 0; i < IB; ++i) {
                    const v16f p = g == 0 ? mfma<0>(fx[i], fw[j], (int)e[i]) : mfma<2>(fx[i], fw[j], (int)e[i]);
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_fmaf(p[r], s, acc[i][j][r]);
                }
            }
        }
        if (more) store(buf ^ 1);
        __syncthreads();
    }

    // sums to LDS: row-major, 16-byte chunks of a row rotated by the row so
    // that the lanes of a store spread over the banks
    float *tile = reinterpret_cast<float *>(smem);
    auto cell = [](int row, int col) { return row * BN + (col ^ ((row & 7) << 2)); };
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = wm + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
                tile[cell(row, wn + 32 * j + l32)] = acc[i][j][r] * code_scale<BITS>();
            }
    __syncthreads();
    finish_tile<BM, BN>(a, m0, n0, tid, [&](int row, int col) {
        return *reinterpret_cast<const v4f *>(tile + cell(row, col));
    });
}

template <int BM, int BITS>
hipError_t launch_tiles(const PackedLinear &a, bool wide, hipStream_t s) {
    const int64_t tm = ((int64_t)a.M + BM - 1) / BM, tn = ((int64_t)a.N + BN - 1) / BN;
    if (tm * tn * 256 > UINT32_MAX) return hipErrorInvalidValue;
    return launch(wide ? packed_tile_kernel<BM, BITS, true> : packed_tile_kernel<BM, BITS, false>,
                  dim3((unsigned)(tm * tn)), dim3(256), s, a, (int)tm);
}

template <int BITS>
hipError_t launch_bits(const PackedLinear &a, hipStream_t s) {
    const auto al = [](const void *p, int64_t ld, int64_t b) {
        return reinterpret_cast<uintptr_t>(p) % b == 0 && ld % b == 0;
    };
    const bool wide = al(a.X, a.ldx, 16) && al(a.Q, a.ldq, 16) && al(a.XE, a.ldxe, 4) &&
                      al(a.S, a.lds * 2, 4);
    if (a.M > 64) return launch_tiles<128, BITS>(a, wide, s);
    if (a.M > 32) return launch_tiles<64, BITS>(a, wide, s);
    const bool wide_rows = al(a.X, a.ldx, 16) && al(a.Q, a.ldq, 4 * BITS);
    const dim3 grid((unsigned)(((int64_t)a.N + 31) / 32));
    if ((int64_t)grid.x * 64 * KS > UINT32_MAX) return hipErrorInvalidValue;
    return launch(wide_rows ? packed_rows_kernel<BITS, true> : packed_rows_kernel<BITS, false>, grid,
                  dim3(64 * KS), s, a);
}

}  // namespace

hipError_t launch_packed_linear(int bits, const PackedLinear &a, int num_cus, hipStream_t s) {
    (void)num_cus;
    return bits == 2 ? launch_bits<2>(a, s) : launch_bits<4>(a, s);
}

}  // namespace gg
