// linear_mx8.hip -- Y = act(X8.W^T + b) + R with X8 in 8 bits (mx8.hpp) and W
// as 2-bit or 4-bit codes with one binary16 scale per 64 columns, on gfx950's
// block-scaled matrix instruction.
//
//   w(n, k) = (code - 7.5) s(n, k/64) = (2 code - 15) s/2     (4 bits)
//   w(n, k) = (code - 1.5) s(n, k/64) = (2 code - 3) s/2      (2 bits)
//
// Every factor has at most 4 significant bits (the odd integers up to 15, and
// e4m3 numbers times a power of two), so both operands are bf16 numbers
// exactly and products are exact in fp32: v_mfma_f32_32x32x16_bf16 sums them in
// fp32, group by group, and one fp32 multiply-add per sum and group applies
// s/2.  Nothing is rounded but the sums.
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
    const int col = tid % PER_ROW * 4;
    const int64_t n = n0 + col;
    const int live = (int)min(max((int64_t)a.N - n, (int64_t)0), (int64_t)4);
    v4f bias = {0.f, 0.f, 0.f, 0.f};
    if (a.bias)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < live) bias[c] = a.bias[n + c];
    with_act(a.act, [&](auto act) {
        constexpr int ROWS = THREADS / PER_ROW;            // rows at a time
#pragma unroll 4
        for (int i = 0; i < BM / ROWS; ++i) {
            const int row = tid / PER_ROW + ROWS * i;
            const int64_t m = m0 + row;
            v4f y = at(row, col);
            const int w = m < a.M ? live : 0;          // columns to store
            v4f res = {0.f, 0.f, 0.f, 0.f};
            if (a.R) {
                const float *p = a.R + m * a.ldr + n;
                if (w == 4) {
                    res = *reinterpret_cast<const v4f_any *>(p);
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
                if (w == 4) {
                    *reinterpret_cast<v4f_any *>(p) = y;
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
                if (w == 4) {
                    *reinterpret_cast<u32_any *>(p) = q;
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

// Up to 16 rows: bound by the codes' way from memory, with one row of x by
// its latency.  No LDS on the way in: a lane loads 32 neighbouring codes of
// its row of W, half of each of two weight groups after an exchange between
// lanes, and expands them in registers for the 16 x 16 x 32 instruction, which
// gives twice the workgroups of 32 x 32 tiles.
//
// A workgroup owns 16 NH columns n (NH = 2 for an output in 8 bits, whose
// blocks are 32 wide); its waves split into NH column sets by KW runs of
// groups, and the runs' sums meet in LDS, added in order.  Loads are 16 bytes
// of x, 32 codes and both scales each; a pair that K cuts short is loaded byte
// by byte.
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
    unsigned w[BITS], e, s;          // codes, x's four powers of two, both scales
    v4u x[2];

    __device__ __forceinline__ void multiply(int q, v4f &acc) {
        deal<BITS>(w);
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
    const uint8_t *w, *x, *e;
    const uint16_t *s;

    __device__ __forceinline__ void advance(int64_t pairs) {
        w += pairs * (16 * BITS);
        x += pairs * 128;
        e += pairs * 4;
        s += pairs * 2;
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
            p[i].e = *reinterpret_cast<const u32_any *>(e + 4 * i);
            p[i].s = *reinterpret_cast<const u32_any *>(s + 2 * i);
        }
        advance(N);
#pragma unroll
        for (int i = 0; i < N; ++i) p[i].multiply(q, acc);
    }
    // the pair at hand, of which columns 0 .. left - 1 exist, byte by byte
    __device__ __forceinline__ void part(int64_t left, int q, v4f &acc) {
        const auto have = [&](int at, int most) {
            return (int)min(max(left - at, (int64_t)0), (int64_t)most);
        };
        Pair<BITS> p;
        load_bytes<4 * BITS>(p.w, w, (have(32 * q, 32) * BITS + 7) / 8);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            unsigned d[4];
            load_bytes<16>(d, x + 64 * g, have(64 * g + 16 * q, 16));
            p.x[g] = v4u{d[0], d[1], d[2], d[3]};
        }
        p.e = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) p.e |= (left > 32 * b ? (unsigned)e[b] : 127u) << (8 * b);
        p.s = (unsigned)s[0] | (left > 64 ? (unsigned)s[1] << 16 : 0u);
        advance(1);
        p.multiply(q, acc);
    }
};

template <int BITS, int NH, int KW>
__global__ __launch_bounds__(64 * NH * KW) void packed_rows_kernel(PackedLinear a) {
    constexpr int NC = 16 * NH;                       // columns
    __shared__ float red[KW][16][NC];
    const int lane = threadIdx.x & 63, q = lane >> 4, l16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nh = wave % NH, kw = wave / NH;
    const int64_t n0 = (int64_t)blockIdx.x * NC;
    const int64_t tok = min(l16, a.M - 1);
    const int64_t nrow = min(n0 + 16 * nh + l16, (int64_t)a.N - 1);
    const int64_t pairs = ((int64_t)a.K + 127) / 128;
    // run kw of KW: as even a share as whole pairs allow
    const int64_t first = pairs * kw / KW, end = pairs * (kw + 1) / KW;
    // the pairs of it that exist in full
    int n = (int)max(min(end, (int64_t)a.K / 128) - first, (int64_t)0);
    Rows<BITS> rows = {a.Q + nrow * a.ldq + 4 * BITS * q, a.X + tok * a.ldx + 16 * q,
                       a.XE + tok * a.ldxe, a.S + nrow * a.lds};
    rows.advance(first);
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    int64_t p = first + n;
    for (; n >= 4; n -= 4) rows.template run<4>(q, acc);
    if (n == 3) rows.template run<3>(q, acc);
    else if (n == 2) rows.template run<2>(q, acc);
    else if (n == 1) rows.template run<1>(q, acc);
#pragma unroll 1
    for (; p < end; ++p) rows.part(a.K - p * 128, q, acc);

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

template <int BITS, int NH, int KW>
hipError_t launch_rows(const PackedLinear &a, hipStream_t s) {
    const int64_t nb = ((int64_t)a.N + 16 * NH - 1) / (16 * NH);
    if (nb * 64 * NH * KW > UINT32_MAX) return hipErrorInvalidValue;
    return launch(packed_rows_kernel<BITS, NH, KW>, dim3((unsigned)nb), dim3(64 * NH * KW), s, a);
}

// ---------------------------------------------------------------------------
// More than 16 rows: a workgroup owns BM rows of x by BN columns n and walks k
// in steps of one weight group, 64, double-buffered in LDS as bf16.  Bound by
// the latency of a step (LDS, expansion, products and barrier in turn) where
// tiles are few, which is where these are used.
//
//  * Codes are expanded, and both operands widened, once per workgroup, on
//    their way into LDS.
//  * LDS rows hold 64 values, 8 chunks of 16 bytes; chunk c of row r lies at slot
//    c ^ (r mod 8), so that the 16-byte fragment reads of 8 neighbouring
//    rows, and the writes, meet no bank twice.
//  * Loads run two steps ahead: registers hold the next step while LDS holds
//    this one; one barrier per step.
//  * Where tiles are few, KS groups of waves share a tile's steps, each with
//    its own stages, and their sums are added in group order.
//  * The finished sums pass through LDS, so that bias, residual and the
//    stores of Y run along rows, 16 bytes per lane.
constexpr int STEP = 64, ROWB = 2 * STEP;   // columns of a step, bytes of an LDS row

// KS groups of WR x WC waves, each wave with IB x JB blocks of 32 x 32.
template <int BM, int BN, int WR, int WC, int KS, int BITS>
__global__ __launch_bounds__(64 * WR * WC * KS, WR * WC * KS >= 8 ? WR * WC * KS / 4 : 2)
void packed_tile_kernel(PackedLinear a, int tiles_m) {
    constexpr int THREADS = 64 * WR * WC;             // of a group
    constexpr int IB = BM / WR / 32, JB = BN / WC / 32;
    static_assert(IB * WR * 32 == BM && JB * WC * 32 == BN, "waves must cover the tile");
    // a row's step is 4 units of 16 columns: 16 bytes of x, CB bytes of codes
    constexpr int CB = 2 * BITS;
    constexpr int XC = BM * 4 / THREADS, WL = BN * 4 / THREADS;   // units per thread
    static_assert(XC * THREADS == BM * 4 && WL * THREADS == BN * 4, "loads must split evenly");
    static_assert(BM <= THREADS && BN <= THREADS, "one scale per thread");
    constexpr int XBYTES = BM * ROWB, WBYTES = BN * ROWB, STAGE = XBYTES + WBYTES;
    constexpr int TILE = BM * BN * 4;                 // a group's finished sums
    constexpr int SMEM = KS * (2 * STAGE > TILE ? 2 * STAGE : TILE);
    __shared__ __attribute__((aligned(16))) char smem[SMEM];
    __shared__ unsigned all_scales[KS][2][BN];        // W: a half per row and step

    const int grp = KS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / THREADS);
    const int tid = threadIdx.x % THREADS, lane = tid & 63, wave = tid >> 6, h = lane >> 5,
              l32 = lane & 31;
    char *const gsmem = smem + grp * 2 * STAGE;
    unsigned(*const scales)[BN] = all_scales[grp];
    int t = blockIdx.x;
    if ((gridDim.x & 7) == 0) t = (t & 7) * (gridDim.x >> 3) + (t >> 3);   // runs per XCD
    const int64_t m0 = (int64_t)(t % tiles_m) * BM;
    const int64_t n0 = (int64_t)(t / tiles_m) * BN;
    const int wm = wave / WC * (32 * IB), wn = wave % WC * (32 * JB);

    const int unit = tid % 4;
    const uint8_t *px[XC], *pe[XC], *pw[WL];
#pragma unroll
    for (int i = 0; i < XC; ++i) {
        const int64_t row = min(m0 + tid / 4 + THREADS / 4 * i, (int64_t)a.M - 1);
        px[i] = a.X + row * a.ldx + 16 * unit;
        pe[i] = a.XE + row * a.ldxe + unit / 2;
    }
#pragma unroll
    for (int i = 0; i < WL; ++i)
        pw[i] = a.Q + min(n0 + tid / 4 + THREADS / 4 * i, (int64_t)a.N - 1) * a.ldq + CB * unit;
    // the first BN threads fetch a row's scale
    const bool fetch_s = tid < BN;
    const uint16_t *ps = a.S + min(n0 + (fetch_s ? tid : 0), (int64_t)a.N - 1) * a.lds;

    v4u xr[XC];
    unsigned wr[WL][BITS / 2], er[XC], sr = 0;
    // a step whose 64 columns all exist, and the last one, cut short by K
    auto load = [&](int64_t step) {
        const int64_t k0 = step * STEP, kq = k0 * BITS / 8;
#pragma unroll
        for (int i = 0; i < WL; ++i) load_codes<BITS / 2>(wr[i], pw[i] + kq);
#pragma unroll
        for (int i = 0; i < XC; ++i) {
            xr[i] = *reinterpret_cast<const v4u_any *>(px[i] + k0);
            er[i] = pe[i][k0 / 32];
        }
        sr = ps[step];
    };
    auto load_part = [&](int64_t step) {
        const int64_t k0 = step * STEP;
        const int left = (int)(a.K - k0) - 16 * unit;              // columns of this unit on
#pragma unroll
        for (int i = 0; i < WL; ++i)
            load_bytes<CB>(wr[i], pw[i] + k0 * BITS / 8, (min(max(left, 0), 16) * BITS + 7) / 8);
#pragma unroll
        for (int i = 0; i < XC; ++i) {
            unsigned d[4];
            load_bytes<16>(d, px[i] + k0, left);
            xr[i] = v4u{d[0], d[1], d[2], d[3]};
            er[i] = left > 0 ? pe[i][k0 / 32] : 127u;
        }
        sr = ps[step];
    };
    auto slot = [](int row, int c) { return row * ROWB + ((c ^ (row & 7)) * 16); };
    auto put = [&](char *base, int row, const v4u &bytes, unsigned e) {
        *reinterpret_cast<v4u *>(base + slot(row, 2 * unit)) = widen(bytes[0], bytes[1], e);
        *reinterpret_cast<v4u *>(base + slot(row, 2 * unit + 1)) = widen(bytes[2], bytes[3], e);
    };
    auto store = [&](int buf) {
        char *xs = gsmem + buf * STAGE, *ws = xs + XBYTES;
#pragma unroll
        for (int i = 0; i < XC; ++i)
            put(xs, tid / 4 + THREADS / 4 * i, shuffle16<BITS>(xr[i]), er[i]);
#pragma unroll
        for (int i = 0; i < WL; ++i)
            put(ws, tid / 4 + THREADS / 4 * i, expand16<BITS>(wr[i]), 127);
        if (fetch_s) scales[buf][tid] = sr;
    };
    // the operand of 16 columns: part t of the lane's row
    auto frag = [&](const char *base, int row, int t) {
        return *reinterpret_cast<const v4u *>(base + slot(row, 2 * t + h));
    };

    v16f acc[IB][JB];
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    auto multiply = [&](int buf) {
        const char *xs = gsmem + buf * STAGE, *ws = xs + XBYTES;
        float s[JB];
#pragma unroll
        for (int j = 0; j < JB; ++j)
            s[j] = scale_of(scales[buf][wn + 32 * j + l32]);
        v4u fx[IB][4], fw[JB][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int i = 0; i < IB; ++i) fx[i][t] = frag(xs, wm + 32 * i + l32, t);
#pragma unroll
            for (int j = 0; j < JB; ++j) fw[j][t] = frag(ws, wn + 32 * j + l32, t);
        }
        // A block's products and the multiply-adds of the block before it
        // alternate, two result tuples in turn, so neither unit waits for the
        // other.
        v16f p[2];
        constexpr int BLOCKS = IB * JB;
#pragma unroll
        for (int b = 0; b <= BLOCKS; ++b) {
            if (b < BLOCKS) {
                v16f q;
#pragma unroll
                for (int r = 0; r < 16; ++r) q[r] = 0.f;
#pragma unroll
                for (int t = 0; t < 4; ++t) q = mfma(fx[b % IB][t], fw[b / IB][t], q);
                p[b & 1] = q;
            }
            __builtin_amdgcn_sched_barrier(0);
            if (b > 0) {
                const int c = b - 1, i = c % IB, j = c / IB;
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    acc[i][j][r] = __builtin_fmaf(p[c & 1][r], s[j], acc[i][j][r]);
                // a use here, or all of this moves past the stores and the
                // barrier below
                asm volatile("" : "+v"(acc[i][j]));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    // Group g takes the steps g, g + KS, ...; every group goes through the same
    // number of rounds.  The next step's data, in registers since the last
    // round, go to the stage that the last round read, and the loads of the one
    // after it have this whole round to arrive: they are unconditional (past
    // the end, the last whole step again), because a load under a branch is
    // waited for where the branch joins.
    const int64_t whole = a.K / STEP;
    int buf = 0;
    if (whole > 0) {
        load(min((int64_t)grp, whole - 1));
        store(0);
        load(min((int64_t)grp + KS, whole - 1));
        __syncthreads();
        for (int64_t s0 = 0; s0 < whole; s0 += KS, buf ^= 1) {
            store(buf ^ 1);
            load(min(s0 + grp + 2 * KS, whole - 1));
            if (KS == 1 || s0 + grp < whole) multiply(buf);        // uniform
            __syncthreads();
        }
    }
    if (a.K % STEP) {                                 // one more, cut short
        const bool mine = KS == 1 || whole % KS == grp;
        if (mine) {
            load_part(whole);
            store(buf);
        }
        __syncthreads();
        if (mine) multiply(buf);
        __syncthreads();
    }

    // Sums to LDS, a tile per group: row-major, 16-byte chunks of a row rotated
    // by the row so that the lanes of a store spread over the banks.  (Every
    // stage has been read: the last round ended with a barrier.)
    float *tile = reinterpret_cast<float *>(smem);
    auto cell = [](int row, int col) { return row * BN + (col ^ ((row & 7) << 2)); };
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = wm + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3);
                tile[grp * BM * BN + cell(row, wn + 32 * j + l32)] = acc[i][j][r] * code_scale<BITS>();
            }
    __syncthreads();
    finish_tile<BM, BN, THREADS * KS>(a, m0, n0, threadIdx.x, [&](int row, int col) {
        v4f y = *reinterpret_cast<const v4f *>(tile + cell(row, col));
#pragma unroll
        for (int g = 1; g < KS; ++g)                  // in group order
            y += *reinterpret_cast<const v4f *>(tile + g * BM * BN + cell(row, col));
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
// about equally much to do; 2048 x 4096 x 4096 runs at 770 TFLOP/s, the
// matrix unit busy for a third of the time.  MW: waves per SIMD that the
// registers leave room for; a SIMD issues vector instructions of one wave
// every 7 cycles, of two or more every 3 to 4.
constexpr int SPAN = 128, SPANB = 2 * SPAN + 16;      // columns of x in a stage, bytes of a row

template <int BM, int NW, int BITS, int MW = 2>
__global__ __launch_bounds__(64 * NW, MW) void packed_wide_kernel(PackedLinear a, int tiles_m) {
    constexpr int THREADS = 64 * NW, BN = 32 * NW, IB = BM / 32;
    constexpr int XC = BM * (SPAN / 16) / THREADS;    // units of 16 columns of x per thread
    static_assert(XC * THREADS == BM * (SPAN / 16), "loads must split evenly");
    constexpr int STAGE = BM * SPANB, TILE = BM * BN * 4;
    constexpr int SMEM = 3 * STAGE > TILE ? 3 * STAGE : TILE;
    __shared__ __attribute__((aligned(16))) char smem[SMEM];

    const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, l32 = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int tb = blockIdx.x;
    if ((gridDim.x & 7) == 0) tb = (tb & 7) * (gridDim.x >> 3) + (tb >> 3);   // runs per XCD
    const int64_t m0 = (int64_t)(tb % tiles_m) * BM, n0 = (int64_t)(tb / tiles_m) * BN;

    const int unit = tid % 8;                         // THREADS is a multiple of 8
    const uint8_t *px[XC], *pe[XC];
#pragma unroll
    for (int i = 0; i < XC; ++i) {
        const int64_t row = min(m0 + (tid + THREADS * i) / 8, (int64_t)a.M - 1);
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
            load_bytes<16>(d, px[i] + k0, left);
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
            load_bytes<4 * BITS>(c.w[g], pq + k0 * BITS / 8,
                                 (min(max(left - 32 * h, 0), 32) * BITS + 7) / 8);
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

template <int BM, int NW, int BITS, int MW = 2>
hipError_t launch_wide(const PackedLinear &a, hipStream_t s) {
    const int64_t tm = ((int64_t)a.M + BM - 1) / BM, tn = ((int64_t)a.N + 32 * NW - 1) / (32 * NW);
    if (tm * tn * 64 * NW > UINT32_MAX) return hipErrorInvalidValue;
    return launch(packed_wide_kernel<BM, NW, BITS, MW>, dim3((unsigned)(tm * tn)), dim3(64 * NW), s, a,
                  (int)tm);
}

template <int BM, int BN, int WR, int WC, int KS, int BITS>
hipError_t launch_tiles(const PackedLinear &a, hipStream_t s) {
    const int64_t tm = ((int64_t)a.M + BM - 1) / BM, tn = ((int64_t)a.N + BN - 1) / BN;
    constexpr int THREADS = 64 * WR * WC * KS;
    if (tm * tn * THREADS > UINT32_MAX) return hipErrorInvalidValue;
    return launch(packed_tile_kernel<BM, BN, WR, WC, KS, BITS>, dim3((unsigned)(tm * tn)),
                  dim3(THREADS), s, a, (int)tm);
}

template <int BITS>
hipError_t launch_bits(const PackedLinear &a, int num_cus, hipStream_t s) {
    const auto count = [&](int bm, int bn) {
        return (((int64_t)a.M + bm - 1) / bm) * (((int64_t)a.N + bn - 1) / bn);
    };
    const int64_t cus = num_cus;
    // Up to 16 rows.  Runs of k per column set by what fills the CUs: 4 where
    // there is a workgroup per CU (one row, 4 bits, 12288 x 1536: 5.6 us in 4,
    // 6.9 in 8, 7.5 in 16), else as many as the rows are long enough for (1536 x
    // 12288: 12.3 us in 4, 11.6 in 8, 9.8 in 16; 768 x 768: 3.4, 3.3, 3.6).
    // With an output in 8 bits there are two column sets (12288 x 1536: 6.6 us
    // in 2, 6.3 in 4, 7.5 in 8; 1536 x 12288: 22, 24, 16).
    if (a.M <= 16) {
        const bool lengthy = a.K >= 4096;
        if (a.Y8)
            return count(16, 32) < cus && lengthy ? launch_rows<BITS, 2, 8>(a, s)
                                                  : launch_rows<BITS, 2, 4>(a, s);
        if (count(16, 16) >= cus) return launch_rows<BITS, 1, 4>(a, s);
        return lengthy ? launch_rows<BITS, 1, 16>(a, s) : launch_rows<BITS, 1, 8>(a, s);
    }
    // More rows, by how the tiles fill the CUs (4 bits, us):
    //  - a wave per 32 columns, 128 x 256 tiles, where a round of them leaves at
    //    most a fifth of the CUs idle: 2048 x 4096 x 4096 89 against 107 in
    //    64 x 128 tiles and 156 in 64 x 64;
    //  - 32 x 64 tiles in four k-groups where they fit one per CU: 128 x 4096 x
    //    4096 18.5 against 22.7 in 64 x 64;
    //  - 64 x 64 in four k-groups, one per CU (64 x 12288 x 1536 12.6 against
    //    13.2 in two and 17 in one; 500 x 1536 x 12288 56 / 70 / 103), in two at
    //    two per CU (128 x 12288 x 1536 18.6 against 22.7 in four, and 19.9 in
    //    64 x 128 with a wave per 32 columns);
    //  - else 64 x 128 with a wave per 32 columns (256 x 12288 x 1536 25.8
    //    against 26.8 in 64 x 64; 500 x 12288 x 1536 36.3 against 47).
    const int64_t big = count(128, 256), mid = count(64, 64);
    if (big >= cus && 4 * ((big + cus - 1) / cus * cus) <= 5 * big)
        return launch_wide<128, 8, BITS, 2>(a, s);
    if (count(32, 64) <= cus) return launch_tiles<32, 64, 1, 2, 4, BITS>(a, s);
    if (mid <= cus) return launch_tiles<64, 64, 2, 2, 4, BITS>(a, s);
    if (mid <= 2 * cus) return launch_tiles<64, 64, 2, 2, 2, BITS>(a, s);
    return launch_wide<64, 4, BITS, 3>(a, s);
}

}  // namespace

hipError_t launch_packed_linear(int bits, const PackedLinear &a, int num_cus, hipStream_t s) {
    return bits == 2 ? launch_bits<2>(a, num_cus, s) : launch_bits<4>(a, num_cus, s);
}

}  // namespace gg
