// linear_mx8_tile.hpp -- tiles of Y = act(X8.W^T + b) + R with X8 in 8 bits (mx8.hpp) and W
// as 2-bit or 4-bit codes with one binary16 scale per 64 columns, on gfx950's
// bf16 matrix instructions.
//
//   w(n, k) = (code - 7.5) s(n, k/64) = (2 code - 15) s/2     (4 bits)
//   w(n, k) = (code - 1.5) s(n, k/64) = (2 code - 3) s/2      (2 bits)
//
// Every factor has at most 4 significant bits (the odd integers up to 15, and
// e4m3 numbers times a power of two), so both operands are bf16 numbers
// exactly and products are exact in fp32: v_mfma_f32_32x32x16_bf16 sums them in
// fp32, group by group, and one fp32 multiply-add per sum and group applies
// s/2.  Nothing is rounded but the sums, and values of x below bf16's smallest
// step, 2^-133 (in blocks whose power of two is 2^-125 or less), to that step.
//
// The 8-bit matrix instructions (f8f6f4 and fp8) would take both operands as
// they are, twice as fast, but add products within parts of their k in an
// adder that keeps 13 bits below the largest product (measured: 448 + 2^-7 =
// 448): sums of 64 random products were off by 3e-6 relative to their size,
// 0 with bf16.
//
// Rows of x are the instruction's A operand (they spread over a lane's 16
// sums), rows of W its B operand: a lane belongs to one output column n, so
// its weight scale is one register and stores of Y run along rows.
//
// Codes are expanded by shifts and a byte permutation that looks their e4m3
// bytes up, and e4m3 bytes of both operands are widened two at a time by
// v_cvt_scalef32_pk_bf16_fp8, which applies x's power of two.  Shifting yields
// the codes in the order 0, 2, 4, 6, 1, 3, 5, 7 (4 bits) or 0, 4, 8, 12, 1, 5,
// ... (2 bits), and x's bytes are permuted the same way, since a sum over k
// may be taken in any order as long as both operands agree.
//
// A tile is told the place (m0, n0) of its cells and, by x_of(m), which row of
// X feeds row m of Y: the same row for the dense layers (linear_mx8.hip), the
// one that the grouping picks for layers grouped by expert
// (linear_mx8_grouped.hip).
#pragma once
#include <hip/hip_runtime.h>

#include <type_traits>

#include "activation.hpp"
#include "kernels.hpp"
#include "mx8.hpp"

namespace gg {
namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v2u __attribute__((ext_vector_type(2)));
// rows may start at any byte: the same loads, without the promise of alignment
typedef v4u v4u_any __attribute__((aligned(1)));
typedef v2u v2u_any __attribute__((aligned(1)));
typedef unsigned u32_any __attribute__((aligned(1)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef v4f v4f_any __attribute__((aligned(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

__device__ __forceinline__ unsigned perm(unsigned hi, unsigned lo, unsigned sel) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_perm(hi, lo, sel);
#else
    return 0;
#endif
}

// Eight 4-bit codes as the e4m3 bytes of 15 - 2 code, even nibbles in lo, odd
// ones in hi.  The magnitudes 1, 3, ..., 15 are looked up at code mod 8 (upper
// codes) or its complement, bit 3 becomes the sign; both are found for all
// eight nibbles at once.  The caller's scale is negative.
__device__ __forceinline__ void e4m3_of_4bit(unsigned w, unsigned &lo, unsigned &hi) {
    const unsigned up = w & 0x88888888u;
    const unsigned seven = up - (up >> 3);              // 7 in nibbles of codes >= 8
    const unsigned idx = (w ^ ~seven) & 0x77777777u;
    lo = perm(0x57555351u, 0x4E4A4438u, idx & 0x07070707u) | (up << 4 & 0x80808080u);
    hi = perm(0x57555351u, 0x4E4A4438u, idx >> 4 & 0x07070707u) | (up & 0x80808080u);
}

// Four 2-bit codes, one per byte, as the e4m3 bytes of 2 code - 3.
__device__ __forceinline__ unsigned e4m3_of_2bit(unsigned c) {
    return perm(0, 0x4438B8C4u, c);
}

template <int BITS>
constexpr float code_scale() { return BITS == 4 ? -0.5f : 0.5f; }

// 16 codes (BITS / 2 dwords) as e4m3 bytes.
template <int BITS>
__device__ __forceinline__ v4u expand16(const unsigned *w) {
    v4u o;
    if constexpr (BITS == 4) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            unsigned lo, hi;
            e4m3_of_4bit(w[j], lo, hi);
            o[2 * j] = lo;
            o[2 * j + 1] = hi;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = e4m3_of_2bit(w[0] >> (2 * i) & 0x03030303u);
    }
    return o;
}

// 16 bytes of x in the order of expand16's codes.
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

// 8 e4m3 bytes times 2^(e - 127) as bf16 (e = 255: NaN).
__device__ __forceinline__ v4u widen(unsigned lo, unsigned hi, unsigned e) {
#if defined(__HIP_DEVICE_COMPILE__)
    const float f = __uint_as_float(e << 23);         // only its exponent counts
    const auto pk = [f](unsigned w, auto half) {
        return __builtin_bit_cast(
            unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, f, decltype(half)::value));
    };
    return v4u{pk(lo, std::false_type{}), pk(lo, std::true_type{}), pk(hi, std::false_type{}),
               pk(hi, std::true_type{})};
#else
    return v4u{0, 0, 0, 0};
#endif
}

__device__ __forceinline__ v8b operand(const v4u &x) { return __builtin_bit_cast(v8b, x); }

__device__ __forceinline__ v16f mfma(const v4u &a, const v4u &b, const v16f &c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(operand(a), operand(b), c, 0, 0, 0);
#else
    return c;
#endif
}

// The same for 16 rows of x by 16 rows of W over 32 columns.
__device__ __forceinline__ v4f mfma16(const v4u &a, const v4u &b, const v4f &c) {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(operand(a), operand(b), c, 0, 0, 0);
#else
    return c;
#endif
}

// A weight scale as fp32, in a register of its own: left to itself the compiler
// folds the conversion into every multiply-add, and the mixed-precision form
// takes 4.4 cycles a wave where the plain one takes 2.8.
__device__ __forceinline__ float scale_of(unsigned half) {
    float s = (float)__builtin_bit_cast(_Float16, (uint16_t)half);
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(s));
#endif
    return s;
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

// 16 bytes less the first n, zeros behind them.
__device__ __forceinline__ v4u drop_bytes(v4u v, unsigned n) {
    const v4u none = {0, 0, 0, 0};
    if (n & 8) v = v4u{v[2], v[3], 0, 0};
    if (n & 4) v = v4u{v[1], v[2], v[3], 0};
#if defined(__HIP_DEVICE_COMPILE__)
    v = v4u{__builtin_amdgcn_alignbyte(v[1], v[0], n), __builtin_amdgcn_alignbyte(v[2], v[1], n),
            __builtin_amdgcn_alignbyte(v[3], v[2], n), __builtin_amdgcn_alignbyte(0, v[3], n)};
#endif
    return n < 16 ? v : none;
}

// N bytes (8 or 16) from p, of which `have` exist (none if negative), as one
// load that ends where the row does and drops what comes before p; byte by byte
// if the row is too short for that.
template <int N>
__device__ __forceinline__ void load_cut(unsigned (&d)[N / 4], const uint8_t *p, int have, bool row_long) {
    if (!row_long) {
        load_bytes<N>(d, p, have);
        return;
    }
    const int n = max(N - have, 0);
    if constexpr (N == 16) {
        const v4u v = drop_bytes(*reinterpret_cast<const v4u_any *>(p - n), (unsigned)n);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = v[i];
    } else {
        const v2u v = *reinterpret_cast<const v2u_any *>(p - n);
        const uint64_t b = n < 8 ? ((uint64_t)v[1] << 32 | v[0]) >> (8 * n) : 0;
        d[0] = (unsigned)b;
        d[1] = (unsigned)(b >> 32);
    }
}

// D dwords in one load, from any byte.
template <int D>
__device__ __forceinline__ void load_codes(unsigned (&w)[D], const uint8_t *p) {
    if constexpr (D == 4) {
        const v4u q = *reinterpret_cast<const v4u_any *>(p);
#pragma unroll
        for (int d = 0; d < 4; ++d) w[d] = q[d];
    } else if constexpr (D == 2) {
        const v2u q = *reinterpret_cast<const v2u_any *>(p);
        w[0] = q[0];
        w[1] = q[1];
    } else {
        w[0] = *reinterpret_cast<const u32_any *>(p);
    }
}

// What the finished sum of (tok, n) becomes.  For an output in 8 bits the 32
// lanes of a half-wave call together, on 32 neighbouring columns of a token
// (`live`: whether the cell exists).
__device__ __forceinline__ void finish(const PackedLinear &a, float sum, int64_t tok, int64_t n,
                                       bool live) {
    float y = 0.f, res = 0.f;
    if (live) {
        if (a.bias) sum += a.bias[n];
        if (a.R) res = a.R[tok * a.ldr + n];
    }
    with_act(a.act, [&](auto t) { y = act_value<decltype(t)::value>(sum); });
    if (a.R) y += res;
    if (a.Y && live) a.Y[tok * a.ldy + n] = y;
    if (a.Y8) {
        const int e = mx8_exponent(half32_max(live ? mag(y) : 0u));
        if (live) {
            a.Y8[tok * a.ldy8 + n] = (uint8_t)mx8_pack2(y, 0.f, e);
            if (n % 32 == 0) a.YE[tok * a.ldye + n / 32] = (uint8_t)e;
        }
    }
}

// The same for a BM x BN tile of sums at (m0, n0) that THREADS threads read
// back 4 columns at a time: at(row, col) gives 4 sums.
template <int BM, int BN, int THREADS, class At>
__device__ __forceinline__ void finish_tile(const PackedLinear &a, int64_t m0, int64_t n0, int tid,
                                            At at) {
    constexpr int PER_ROW = BN / 4;                    // threads along a row
    constexpr int USED = THREADS < BM * PER_ROW ? THREADS : BM * PER_ROW;
    if (tid >= USED) return;                           // whole waves
    constexpr int ROWS = USED / PER_ROW;               // rows at a time
    const int col = tid % PER_ROW * 4, rows = (int)min((int64_t)a.M - m0, (int64_t)BM);
    const int64_t n = n0 + col, m = m0 + tid / PER_ROW;
    const bool whole = n0 + BN <= a.N;                 // uniform
    const int live = whole ? 4 : (int)min(max((int64_t)a.N - n, (int64_t)0), (int64_t)4);
    v4f bias = {0.f, 0.f, 0.f, 0.f};
    if (a.bias) {
        if (whole) {
            bias = *reinterpret_cast<const v4f_any *>(a.bias + n);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c < live) bias[c] = a.bias[n + c];
        }
    }
    // a thread's first row, and ROWS rows on from there with each step
    const float *pr = a.R + m * a.ldr + n;
    float *py = a.Y + m * a.ldy + n;
    uint8_t *p8 = a.Y8 + m * a.ldy8 + n, *pe = a.YE + m * a.ldye + n / 32;
    with_act(a.act, [&](auto act) {
#pragma unroll 4
        for (int i = 0; i < BM / ROWS; ++i) {
            const int row = tid / PER_ROW + ROWS * i;
            v4f y = at(row, col);
            const bool there = row < rows;
            const int w = there ? live : 0;            // columns to store
            v4f res = {0.f, 0.f, 0.f, 0.f};
            if (a.R) {
                if (w == 4) {
                    res = *reinterpret_cast<const v4f_any *>(pr);
                } else if (!whole) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c < w) res[c] = pr[c];
                }
                pr += ROWS * a.ldr;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                y[c] = act_value<decltype(act)::value>(y[c] + bias[c]);
                if (a.R) y[c] += res[c];
            }
            if (a.Y) {
                if (w == 4) {
                    *reinterpret_cast<v4f_any *>(py) = y;
                } else if (!whole) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c < w) py[c] = y[c];
                }
                py += ROWS * a.ldy;
            }
            if (a.Y8) {
                unsigned top = 0;                      // 8 lanes hold a block of 32
#pragma unroll
                for (int c = 0; c < 4; ++c) top = max(top, c < w ? mag(y[c]) : 0u);
                const int e = mx8_exponent(oct_max(top));
                const unsigned q = mx8_pack4(y[0], y[1], y[2], y[3], e);
                if (w == 4) {
                    *reinterpret_cast<u32_any *>(p8) = q;
                } else if (!whole) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c < w) p8[c] = (uint8_t)(q >> (8 * c));
                }
                if (w > 0 && n % 32 == 0) *pe = (uint8_t)e;
                p8 += ROWS * a.ldy8;
                pe += ROWS * a.ldye;
            }
        }
    });
}

// Up to 16 rows: bound by the codes' way from memory, with one row of x by
// its latency.  No LDS on the way in: a lane loads 32 neighbouring codes of
// its row of W, half of each of two weight groups after an exchange between
// lanes, and expands them in registers for the 16 x 16 x 32 instruction, which
// gives twice the workgroups of 32 x 32 tiles.
//
// A workgroup owns 16 NH columns n (NH = 2 for an output in 8 bits, whose
// blocks are 32 wide); its waves split into NH column sets by KW runs of
// groups, and the runs' sums meet in LDS, added in order.  Loads are 16 bytes
// of x, 32 codes, and x's powers of two (lower lanes) with both scales (upper).
//
// Lanes 16q .. 16q + 15 have loaded codes 32q .. 32q + 31 of a pair of
// groups; afterwards they have codes 16q .. 16q + 15 of the first group in the
// lower dwords and of the second in the upper.
template <int BITS>
__device__ __forceinline__ void deal(unsigned (&w)[BITS]) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) {
        const auto p = __builtin_amdgcn_permlane16_swap(w[i], w[i + BITS / 2], false, false);
        const auto o = __builtin_amdgcn_permlane32_swap(p[0], p[1], false, false);
        w[i] = o[0];
        w[i + BITS / 2] = o[1];
    }
#endif
}

// One pair of groups, as loaded, and its products added to the sums.
template <int BITS>
struct Pair {
    unsigned w[BITS], es;            // codes; x's four powers of two in the lower
    v4u x[2];                        // lanes, both scales in the upper

    __device__ __forceinline__ void multiply(int q, v4f &acc) {
        deal<BITS>(w);
        unsigned e = es, s = es;
#if defined(__HIP_DEVICE_COMPILE__)
        const auto both = __builtin_amdgcn_permlane32_swap(es, es, false, false);
        e = both[0];
        s = both[1];
#endif
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            // 16 columns of block 2 g + q / 2
            const unsigned eg = e >> (16 * g + 8 * (q >> 1)) & 255u;
            const v4u b = expand16<BITS>(w + g * (BITS / 2)), a = shuffle16<BITS>(x[g]);
            v4f r = {0.f, 0.f, 0.f, 0.f};
            r = mfma16(widen(a[0], a[1], eg), widen(b[0], b[1], 127), r);
            r = mfma16(widen(a[2], a[3], eg), widen(b[2], b[3], 127), r);
            const float sg = scale_of(s >> (16 * g));
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(r[i], sg, acc[i]);
        }
    }
};

// A lane's pointers to its rows, at one pair of groups.
template <int BITS>
struct Rows {
    const uint8_t *w, *x, *es;

    __device__ __forceinline__ void advance(int64_t pairs) {
        w += pairs * (16 * BITS);
        x += pairs * 128;
        es += pairs * 4;
    }
    // N whole pairs, all loads in flight together
    template <int N>
    __device__ __forceinline__ void run(int q, v4f &acc) {
        Pair<BITS> p[N];
#pragma unroll
        for (int i = 0; i < N; ++i) load_codes<BITS>(p[i].w, w + i * (16 * BITS));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            p[i].x[0] = *reinterpret_cast<const v4u_any *>(x + i * 128);
            p[i].x[1] = *reinterpret_cast<const v4u_any *>(x + i * 128 + 64);
            p[i].es = *reinterpret_cast<const u32_any *>(es + 4 * i);
        }
        advance(N);
#pragma unroll
        for (int i = 0; i < N; ++i) p[i].multiply(q, acc);
    }
    // the pair at hand, of which columns 0 .. left - 1 exist, of a row of K
    __device__ __forceinline__ void part(int left, int K, int q, v4f &acc) {
        const bool row_long = K >= 128;
        Pair<BITS> p;
        load_cut<4 * BITS>(p.w, w, ((left * BITS + 7) >> 3) - 4 * BITS * q, row_long);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            unsigned d[4];
            load_cut<16>(d, x + 64 * g, left - 64 * g - 16 * q, row_long);
            p.x[g] = v4u{d[0], d[1], d[2], d[3]};
        }
        unsigned d[1];
        load_bytes<4>(d, es, q < 2 ? (left + 31) / 32 : left > 64 ? 4 : 2);
        p.es = d[0];
        advance(1);
        p.multiply(q, acc);
    }
};

template <int BITS, int NH, int KW, class XOf>
__device__ __forceinline__ void packed_rows(const PackedLinear &a, int64_t n0, XOf x_of) {
    constexpr int NC = 16 * NH;                       // columns
    __shared__ float red[KW][16][NC];
    const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nh = wave % NH, kw = wave / NH;
    const int64_t tok = x_of(min(l16, a.M - 1));
    const int64_t nrow = min(n0 + 16 * nh + l16, (int64_t)a.N - 1);
    const int64_t pairs = ((int64_t)a.K + 127) / 128;
    // run kw of KW: as even a share as whole pairs allow
    const int64_t first = pairs * kw / KW, end = pairs * (kw + 1) / KW;
    // the pairs of it that exist in full
    int n = (int)max(min(end, (int64_t)a.K / 128) - first, (int64_t)0);
    Rows<BITS> rows = {a.Q + nrow * a.ldq + 4 * BITS * q, a.X + tok * a.ldx + 16 * q,
                       q < 2 ? a.XE + tok * a.ldxe
                             : reinterpret_cast<const uint8_t *>(a.S + nrow * a.lds)};
    rows.advance(first);
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    int64_t p = first + n;
    for (; n >= 4; n -= 4) rows.template run<4>(q, acc);
    if (n == 3) rows.template run<3>(q, acc);
    else if (n == 2) rows.template run<2>(q, acc);
    else if (n == 1) rows.template run<1>(q, acc);
#pragma unroll 1
    for (; p < end; ++p) rows.part((int)(a.K - p * 128), a.K, q, acc);

#pragma unroll
    for (int r = 0; r < 4; ++r) red[kw][4 * q + r][16 * nh + l16] = acc[r];
    __syncthreads();
    const int t = threadIdx.x / NC, col = threadIdx.x % NC;
#pragma unroll 1
    for (int m = t; m < a.M; m += 64 * NH * KW / NC) {    // uniform per half-wave where NH = 2
        float sum = red[0][m][col];
#pragma unroll
        for (int w = 1; w < KW; ++w) sum += red[w][m][col];
        finish(a, sum * code_scale<BITS>(), m, n0 + col, n0 + col < a.N);
    }
}

// ---------------------------------------------------------------------------
// More than 16 rows where tiles are few: bound by the vector unit (about 100
// instructions of expansion and multiply-adds per 4 products) and by latency.
// A workgroup owns 32 x 32 cells, and its KW waves split k: each walks its own
// run of pairs of groups without a barrier, and the runs' sums meet in LDS,
// added in order.
//
//  * Loads are 16 bytes per lane with a row's neighbouring units in
//    neighbouring lanes; lanes whose loads lie in 32 rows each would take four
//    times as long (64 x 1536 x 12288, 2 bits: 27.7 us against 17.2).  A
//    stage of LDS of the wave's own deals the bytes out to the lanes that
//    multiply them; 16-byte units of a row are permuted by the row so that reads
//    and writes meet no bank twice.
//  * x's powers of two and W's scales come in one load, powers in the lower
//    half of the lanes, scales in the upper.
template <int KW, int BITS, class XOf>
__device__ __forceinline__ void packed_block(const PackedLinear &a, int64_t m0, int64_t n0, XOf x_of) {
    constexpr int THREADS = 64 * KW;
    // of a wave: 32 rows of 128 columns of x as they are, and of W's codes
    constexpr int WROW = 16 * BITS, XBYTES = 32 * 128, STAGE = XBYTES + 32 * WROW;
    constexpr int UNITS = WROW / 16, WL = UNITS / 2;           // 16-byte units of a row, loads
    constexpr int SMEM = KW * (STAGE > 4096 ? STAGE : 4096);
    __shared__ __attribute__((aligned(16))) char smem[SMEM];
    const int lane = threadIdx.x & 63, h = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char *const xs = smem + wave * STAGE, *const ws = xs + XBYTES;
    const int64_t pairs = ((int64_t)a.K + 127) / 128;
    const int64_t first = pairs * wave / KW, end = pairs * (wave + 1) / KW;
    const auto xrow = [&](int r) { return x_of(min(m0 + r, (int64_t)a.M - 1)); };
    const auto wrow = [&](int r) { return min(n0 + r, (int64_t)a.N - 1); };

    const uint8_t *px[4], *pw[WL], *pes;
#pragma unroll
    for (int j = 0; j < 4; ++j) px[j] = a.X + xrow(lane / 8 + 8 * j) * a.ldx;
#pragma unroll
    for (int j = 0; j < WL; ++j) pw[j] = a.Q + wrow(lane / UNITS + 64 / UNITS * j) * a.ldq;
    // 4 bytes of either: x's powers of two in the lower lanes, scales in the upper
    pes = h == 0 ? a.XE + xrow(l32) * a.ldxe
                 : reinterpret_cast<const uint8_t *>(a.S + wrow(l32) * a.lds);
    const auto xslot = [](int row, int c) { return row * 128 + ((c ^ (row & 7)) * 16); };
    const auto wslot = [](int row, int c) {
        return row * WROW + ((c ^ (BITS == 4 ? row >> 2 & 3 : row >> 3 & 1)) * 16);
    };

    struct Regs {
        v4u x[4], w[WL];
        unsigned es;
    };
    // bytes of a row of x, of codes, and of powers or scales
    const unsigned rx = a.K, rw = ((int64_t)a.K * BITS + 7) / 8;
    const unsigned re = h == 0 ? ((unsigned)a.K + 31) / 32 : ((unsigned)a.K + 63) / 64 * 2;
    // Where K cuts a pair short, loads end where the rows do, and `cut` drops
    // what they hold of columns before their own.  (K >= 128.)
    auto load = [&](int64_t pair, Regs &d) {
        const unsigned p = (unsigned)pair;
        const unsigned cw = min(p * WROW + 16 * (lane % UNITS), rw - 16);
        const unsigned cx = min(p * 128 + 16 * (lane % 8), rx - 16);
#pragma unroll
        for (int j = 0; j < WL; ++j) d.w[j] = *reinterpret_cast<const v4u_any *>(pw[j] + cw);
#pragma unroll
        for (int j = 0; j < 4; ++j) d.x[j] = *reinterpret_cast<const v4u_any *>(px[j] + cx);
        d.es = *reinterpret_cast<const u32_any *>(pes + min(p * 4, re - 4));
    };
    auto cut = [&](int64_t pair, Regs &d) {
        const unsigned p = (unsigned)pair;
        const unsigned ow = p * WROW + 16 * (lane % UNITS), ox = p * 128 + 16 * (lane % 8);
        const unsigned dw = ow - min(ow, rw - 16), dx = ox - min(ox, rx - 16);
#pragma unroll
        for (int j = 0; j < WL; ++j) d.w[j] = drop_bytes(d.w[j], dw);
#pragma unroll
        for (int j = 0; j < 4; ++j) d.x[j] = drop_bytes(d.x[j], dx);
        const unsigned de = p * 4 - min(p * 4, re - 4);
        d.es = de < 4 ? d.es >> (8 * de) : 0u;
    };
    // the same for K < 128, byte by byte
    auto load_short = [&](Regs &d) {
        const auto bytes = [](const uint8_t *from, int have) {
            unsigned b[4];
            load_bytes<16>(b, from, have);
            return v4u{b[0], b[1], b[2], b[3]};
        };
        const int cw = 16 * (lane % UNITS), cx = 16 * (lane % 8);
#pragma unroll
        for (int j = 0; j < WL; ++j) d.w[j] = bytes(pw[j] + cw, (int)rw - cw);
#pragma unroll
        for (int j = 0; j < 4; ++j) d.x[j] = bytes(px[j] + cx, (int)rx - cx);
        unsigned b[1];
        load_bytes<4>(b, pes, (int)re);
        d.es = b[0];
    };

    float acc[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.f;
    // Registers to this wave's stage: LDS takes a wave's accesses in order, so
    // that neither these stores nor the reads below need a barrier.
    auto in_order = [] {
#if defined(__HIP_DEVICE_COMPILE__)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#endif
    };
    auto store = [&](const Regs &d) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<v4u *>(xs + xslot(lane / 8 + 8 * j, lane % 8)) = d.x[j];
#pragma unroll
        for (int j = 0; j < WL; ++j)
            *reinterpret_cast<v4u *>(ws + wslot(lane / UNITS + 64 / UNITS * j, lane % UNITS)) = d.w[j];
        in_order();
    };
    auto multiply = [&](unsigned es) {
        unsigned e = es, s = es;
#if defined(__HIP_DEVICE_COMPILE__)
        const auto o = __builtin_amdgcn_permlane32_swap(es, es, false, false);
        e = o[0];
        s = o[1];
#endif
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            unsigned w[BITS];
            if constexpr (BITS == 4) {
                const v4u q = *reinterpret_cast<const v4u *>(ws + wslot(l32, 2 * g + h));
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = q[i];
            } else {
                const v2u q = *reinterpret_cast<const v2u *>(ws + wslot(l32, g) + 8 * h);
                w[0] = q[0];
                w[1] = q[1];
            }
            const unsigned eg = e >> (16 * g + 8 * h) & 255u;
            v16f q;
#pragma unroll
            for (int r = 0; r < 16; ++r) q[r] = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const v4u x = shuffle16<BITS>(*reinterpret_cast<const v4u *>(xs + xslot(l32, 4 * g + 2 * h + u)));
                const v4u b = expand16<BITS>(w + u * (BITS / 2));
                q = mfma(widen(x[0], x[1], eg), widen(b[0], b[1], 127), q);
                q = mfma(widen(x[2], x[3], eg), widen(b[2], b[3], 127), q);
            }
            const float sg = scale_of(s >> (16 * g));
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[r] = __builtin_fmaf(q[r], sg, acc[r]);
        }
        in_order();
    };
    // Loads run two pairs ahead; past the end they take the last pair again,
    // since a load under a branch is waited for where it joins.
    if (first < end) {
        Regs d[2];
        if (a.K < 128) {
            load_short(d[0]);
        } else {
            load(first, d[0]);
            load(min(first + 1, end - 1), d[1]);
        }
        auto step = [&](int64_t p, Regs &r) {
            const unsigned es = r.es;
            store(r);
            load(min(p + 2, end - 1), r);
            multiply(es);
        };
        int64_t p = first;
        // the last pair or two apart: they load nothing and may be cut short
        for (; p + 2 < end; p += 2) {
            step(p, d[0]);
            step(p + 1, d[1]);
        }
        const int64_t whole = a.K / 128;
        if (a.K >= 128 && p >= whole) cut(p, d[0]);
        store(d[0]);
        multiply(d[0].es);
        if (p + 1 < end) {
            if (p + 1 >= whole) cut(p + 1, d[1]);
            store(d[1]);
            multiply(d[1].es);
        }
    }

    __syncthreads();
    float *tile = reinterpret_cast<float *>(smem);
    auto cell = [](int row, int col) { return row * 32 + (col ^ ((row & 7) << 2)); };
#pragma unroll
    for (int r = 0; r < 16; ++r)
        tile[wave * 1024 + cell(8 * (r >> 2) + 4 * h + (r & 3), l32)] = acc[r] * code_scale<BITS>();
    __syncthreads();
    finish_tile<32, 32, THREADS>(a, m0, n0, threadIdx.x, [&](int row, int col) {
        v4f y = *reinterpret_cast<const v4f *>(tile + cell(row, col));
#pragma unroll
        for (int w = 1; w < KW; ++w) y += *reinterpret_cast<const v4f *>(tile + w * 1024 + cell(row, col));
        return y;
    });
}

// ---------------------------------------------------------------------------
// Many rows: NW waves, each with 32 columns n of its own and all BM rows of x.
// A wave expands its own codes in registers, so W needs no LDS and each code
// feeds BM / 32 blocks; only x passes through LDS, 128 columns at a time.
// Lanes 0-31 hold codes 0-31 of a group, lanes 32-63 codes 32-63: part t of a
// group multiplies columns 8 t .. 8 t + 7 of either half.  At BM = 128 the
// matrix unit (4 x 4 x 32 cycles per wave and group), the vector unit (64
// instructions of expansion, 64 multiply-adds) and LDS (16 KiB per wave) have
// about equally much to do, so products and vector work are interleaved turn
// by turn: 2048 x 4096 x 4096 takes 73-77 us at 2 bits and 78-82 at 4 (890-940
// and 840-880 TFLOP/s; at 4 bits vector issue is busy for 65% of the time and
// the matrix unit for 44%), 89 and 93 with a block's products before its vector
// work.  Four waves of 64 rows (three workgroups per CU) leave 168 registers; 500
// x 1536 x 12288 with a residual takes 31.7 and 34.1 us (vector issue 63 and 65%,
// matrix unit 29 and 25%; 32.6 and 35.6 with a 64-bit product per stored row).  MW: waves
// per SIMD that the registers leave room for; a SIMD issues vector
// instructions of one wave every 7 cycles, of two or more every 3 to 4.
//
// A stage's rows are padded by 16 bytes: 8 neighbouring rows' reads meet no
// bank twice, and every place within a stage is one address and a constant.
constexpr int SPAN = 128, SPANB = 2 * SPAN + 16;      // columns of x in a stage, bytes of a row

//
// smem: wide_bytes<BM, NW>() of LDS, 16-byte aligned, the caller's, so that one
// kernel may run tiles of several shapes.
template <int BM, int NW>
constexpr int wide_bytes() {
    return 3 * BM * SPANB > BM * 32 * NW * 4 ? 3 * BM * SPANB : BM * 32 * NW * 4;
}

template <int BM, int NW, int BITS, class XOf>
__device__ __forceinline__ void packed_wide(const PackedLinear &a, int64_t m0, int64_t n0, XOf x_of,
                                            char *smem) {
    constexpr int THREADS = 64 * NW, BN = 32 * NW, IB = BM / 32;
    constexpr int XC = BM * (SPAN / 16) / THREADS;    // units of 16 columns of x per thread
    static_assert(XC * THREADS == BM * (SPAN / 16), "loads must split evenly");
    constexpr int STAGE = BM * SPANB;

    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    const int unit = tid % 8;                         // THREADS is a multiple of 8
    const uint8_t *px[XC], *pe[XC];
#pragma unroll
    for (int i = 0; i < XC; ++i) {
        const int64_t row = x_of(min(m0 + (tid + THREADS * i) / 8, (int64_t)a.M - 1));
        px[i] = a.X + row * a.ldx + 16 * unit;
        pe[i] = a.XE + row * a.ldxe + unit / 2;
    }
    const int64_t nrow = min(n0 + 32 * wave + l32, (int64_t)a.N - 1);
    const uint8_t *pq = a.Q + nrow * a.ldq + 4 * BITS * h;
    const uint16_t *ps = a.S + nrow * a.lds;

    v4u xr[XC];
    unsigned er[XC];
    // a span whose 128 columns all exist, and the last one, cut short by K
    auto load_x = [&](int64_t span) {
        const int64_t k0 = span * SPAN;
#pragma unroll
        for (int i = 0; i < XC; ++i) {
            xr[i] = *reinterpret_cast<const v4u_any *>(px[i] + k0);
            er[i] = pe[i][k0 / 32];
        }
    };
    auto load_x_part = [&](int64_t span) {
        const int64_t k0 = span * SPAN;
        const int left = (int)(a.K - k0) - 16 * unit;
#pragma unroll
        for (int i = 0; i < XC; ++i) {
            unsigned d[4];
            load_cut<16>(d, px[i] + k0, left, a.K >= 128);
            xr[i] = v4u{d[0], d[1], d[2], d[3]};
            er[i] = left > 0 ? pe[i][k0 / 32] : 127u;
        }
    };
    auto slot = [](int row, int c) { return row * SPANB + c * 16; };
    auto store_x = [&](int buf) {
        char *xs = smem + buf * STAGE;
#pragma unroll
        for (int i = 0; i < XC; ++i) {
            const int row = (tid + THREADS * i) / 8;
            const v4u b = shuffle16<BITS>(xr[i]);
            *reinterpret_cast<v4u *>(xs + slot(row, 2 * unit)) = widen(b[0], b[1], er[i]);
            *reinterpret_cast<v4u *>(xs + slot(row, 2 * unit + 1)) = widen(b[2], b[3], er[i]);
        }
    };
    // codes and scales of the two groups of a span
    struct Codes {
        unsigned w[2][BITS];
        unsigned s[2];
    };
    auto load_w = [&](int64_t span, Codes &c) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            load_codes<BITS>(c.w[g], pq + (span * SPAN + 64 * g) * BITS / 8);
            c.s[g] = ps[2 * span + g];
        }
    };
    auto load_w_part = [&](int64_t span, Codes &c) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int64_t k0 = span * SPAN + 64 * g;
            const int left = (int)(a.K - k0);
            load_cut<4 * BITS>(c.w[g], pq + k0 * BITS / 8,
                               ((left * BITS + 7) >> 3) - 4 * BITS * h, a.K >= 128);
            c.s[g] = left > 0 ? ps[2 * span + g] : 0u;
        }
    };

    float acc[IB][16];
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;

    // 8 of the 32 codes that a lane holds of a group, as bf16
    auto expand = [&](const unsigned (&w)[BITS], int f) {
        if constexpr (BITS == 4) {
            unsigned lo, hi;
            e4m3_of_4bit(w[f], lo, hi);
            return widen(lo, hi, 127);
        } else {
            const unsigned c = w[f / 2] >> (4 * (f & 1));
            return widen(e4m3_of_2bit(c & 0x03030303u), e4m3_of_2bit(c >> 2 & 0x03030303u), 127);
        }
    };
    // half of a unit of x to its place: 8 columns as bf16
    auto put_x = [&](int buf, int i, int half) {
        const int row = (tid + THREADS * i) / 8;
        const v4u d = shuffle16<BITS>(xr[i]);
        *reinterpret_cast<v4u *>(smem + buf * STAGE + slot(row, 2 * unit + half)) =
            widen(d[2 * half], d[2 * half + 1], er[i]);
    };

    // A span in 8 IB turns, each a product and the vector work that the matrix
    // unit covers: multiply-adds of the block before (the last one's of the
    // span before), an eighth of the next group's codes, half a unit of x.  A
    // block's operand of x is read as the block before it lets go of the
    // registers.  x is stored two spans ahead, into the third stage, which the
    // span before this one read, after a barrier in the middle of the span.
    v4u fx[4], fw[2][4];
    v16f p[2];
    float s[2] = {0.f, 0.f};
    auto read = [&](int st, int b, int t) {
        fx[t] = *reinterpret_cast<const v4u *>(
            smem + st * STAGE + slot(32 * (b % IB) + l32, 8 * (b / IB) + 4 * h + t));
    };
    auto fma_block = [&](int d, int from, int to, float sg) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
            if (r >= from && r < to) {
                acc[d % IB][r] = __builtin_fmaf(p[d & 1][r], sg, acc[d % IB][r]);
                asm volatile("" : "+v"(acc[d % IB][r]));       // here, not later
            }
    };
    // stage `st`, whose first operands are in fx; `more`: x in registers goes
    // to stage `st2`, and fx gets the first operands of stage `st1`
    auto multiply = [&](int st, int st1, int st2, const Codes &c, const Codes &next, auto more,
                        auto load) {
        constexpr int NB = 2 * IB;
        const float before = s[1];
        s[0] = scale_of(c.s[0]);
        s[1] = scale_of(c.s[1]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int g = b / IB;
            v16f q;
#pragma unroll
            for (int r = 0; r < 16; ++r) q[r] = 0.f;
            if (decltype(more)::value && b == IB) __syncthreads();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                __builtin_amdgcn_sched_barrier(0);
                q = mfma(fx[t], fw[g][t], q);
                if (b + 1 < NB) read(st, b + 1, t);
                else if (decltype(more)::value) read(st1, 0, t);
                const int turn = 4 * (b % IB) + t;              // of 4 IB in the group
                if (turn % IB == 0 && (g == 0 || decltype(more)::value)) {
                    v4u &f = fw[1 - g][turn / IB];
                    f = expand(g == 0 ? c.w[1] : next.w[0], turn / IB);
                    asm volatile("" : "+v"(f));
                }
                if (decltype(more)::value && g == 1 && turn % 2 == 1 && turn / 2 < 2 * XC)
                    put_x(st2, turn / 4, turn / 2 % 2);
                constexpr int from[5] = {0, 0, 4, 10, 16};
                fma_block(b == 0 ? NB - 1 : b - 1, from[t], from[t + 1],
                          b == 0 ? before : s[(b - 1) / IB]);
            }
            p[b & 1] = q;
        }
        load();
        __builtin_amdgcn_sched_barrier(0);
    };
    auto expand0 = [&](const Codes &c) {
#pragma unroll
        for (int f = 0; f < 4; ++f) fw[0][f] = expand(c.w[0], f);
    };
    auto read0 = [&](int st) {
#pragma unroll
        for (int t = 0; t < 4; ++t) read(st, 0, t);
    };

#pragma unroll
    for (int r = 0; r < 16; ++r) p[1][r] = 0.f;
    // Loads are unconditional, as in the kernel above: past the end they take
    // the last whole span again.
    const int64_t whole = a.K / SPAN;
    int st = 0, st1 = 1, st2 = 2;
    Codes cur;
    if (whole > 0) {
        load_x(0);
        load_w(0, cur);
        store_x(0);
        load_x(min((int64_t)1, whole - 1));
        store_x(1);
        load_x(min((int64_t)2, whole - 1));
        expand0(cur);
        __syncthreads();
        read0(0);
        for (int64_t span = 0; span < whole; ++span) {
            Codes next;
            load_w(min(span + 1, whole - 1), next);
            multiply(st, st1, st2, cur, next, std::true_type{},
                     [&] { load_x(min(span + 3, whole - 1)); });
            cur = next;
            const int done = st;
            st = st1;
            st1 = st2;
            st2 = done;
        }
        __syncthreads();
    }
    if (a.K % SPAN) {                                 // one more, cut short
        load_x_part(whole);
        load_w_part(whole, cur);
        store_x(st1);
        expand0(cur);
        __syncthreads();
        read0(st1);
        multiply(st1, 0, 0, cur, cur, std::false_type{}, [] {});
        __syncthreads();
    }
    fma_block(2 * IB - 1, 0, 16, s[1]);

    // sums to LDS, as in the kernel above
    float *tile = reinterpret_cast<float *>(smem);
    auto cell = [](int row, int col) { return row * BN + (col ^ ((row & 7) << 2)); };
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            tile[cell(32 * i + 8 * (r >> 2) + 4 * h + (r & 3), 32 * wave + l32)] =
                acc[i][r] * code_scale<BITS>();
    __syncthreads();
    finish_tile<BM, BN, THREADS>(a, m0, n0, tid, [&](int row, int col) {
        return *reinterpret_cast<const v4f *>(tile + cell(row, col));
    });
}

}  // namespace
}  // namespace gg
