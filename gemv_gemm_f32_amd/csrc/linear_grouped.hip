// linear_grouped.hip -- the fp32 dense layer on rows grouped by expert, and its
// gradients:
//
//   Z_i = X[rows_i] . op(W_e) + b_e,  Y = act(Z)     (i in group e)
//   dZ = dY * act'(Z)
//   dX_i = dZ_i . op(W_e)^T,  dW_e = X_e^T . dZ_e (or its transpose),
//   db_e = sum of dZ_e's rows
//
// The tiles are those of gemm_f32_tile.hpp (bound by the fp32 matrix unit), in
// one launch for all experts: tiles never span two groups (groups.hpp), and
// the operands' addresses are those of the tile's expert.  Offsets within an
// operand are 32 bits wide and counted from the tile (or, along k, from the
// slab), so only the rows that `rows` picks have to lie within 2 GiB.
//
// X is read through `rows` on its way into LDS, where each lane computes its
// own address in any case; a copy of X in grouped order is never made.
#include <hip/hip_runtime.h>

#include <climits>

#include "gemm_f32_tile.hpp"
#include "groups.hpp"
#include "kernels.hpp"
#include "linear_few.hpp"

namespace gg {
namespace {

// An operand's slabs from an address that moves along k; offsets within a
// slab are 32 bits.
template <class OP, bool XMAJOR>
struct NearSlabs {
    using Place = unsigned;
    OP op;
    const float *P;      // x-major: the tile's first row; k-major: its first column
    int64_t ld, X, K;    // x-major: rows from P on; k-major: columns
    __device__ __forceinline__ void start(int) {}
    __device__ __forceinline__ void issue(char *stage, int k0, int, int wave) {
        const float *p = P + (XMAJOR ? (int64_t)k0 : k0 * ld);
        const int64_t words = XMAJOR ? (X - 1) * ld + K - k0 : (min(K - k0, (int64_t)32) - 1) * ld + X;
        op.issue(stage, p, (int)(words * 4), 0, 0, wave);
    }
};

// A k-major operand whose row k is row rows[k] of P.  The next slab's row
// numbers are fetched with each slab, so that no load waits for them.
template <class OP>
struct PickedSlabs {
    using Place = unsigned;
    OP op;
    const float *P;
    int64_t ld, X;
    const int32_t *rows;
    int K, T;
    unsigned column[OP::NI];   // bytes
    int next[OP::NI];

    __device__ __forceinline__ void init(int X, int lane, int wave) {
        op.init(0, 0, X, lane, wave);
#pragma unroll
        for (int j = 0; j < OP::NI; ++j) column[j] = op.voff[j];
    }
    __device__ __forceinline__ void start(int k0) {
#pragma unroll
        for (int j = 0; j < OP::NI; ++j)
            next[j] = rows[min((unsigned)k0 + op.kof[j], (unsigned)K - 1)];
    }
    __device__ __forceinline__ void issue(char *stage, int, int k_next, int wave) {
#pragma unroll
        for (int j = 0; j < OP::NI; ++j)
            op.voff[j] = column[j] + (unsigned)((int64_t)min((unsigned)next[j], (unsigned)T - 1) * ld * 4);
        op.issue(stage, P, (int)(((int64_t)(T - 1) * ld + X) * 4), 0, 0, wave);
        start(k_next);
    }
};

// A tile's rows of an output, one float of each row per lane: buffer accesses,
// which leave out what lies behind the last row by themselves.  (With a branch and
// a 64-bit address for each row tiles spent a tenth of their time storing.)
constexpr int64_t NEAR_LD = 1 << 22;                  // 64 such rows are 1 GiB
struct TileRows {
#if defined(__HIP_DEVICE_COMPILE__)
    __amdgpu_buffer_rsrc_t rsrc;
#endif
    unsigned ld;         // bytes
    __device__ __forceinline__ TileRows(float *C, int64_t ldc, int rows) : ld((unsigned)ldc * 4) {
#if defined(__HIP_DEVICE_COMPILE__)
        rsrc = __builtin_amdgcn_make_buffer_rsrc(C, (short)0, (int)(min(rows, 64) * ld), 0x00020000);
#endif
    }
    __device__ __forceinline__ unsigned at(int row, int col) const { return (unsigned)row * ld + 4 * (unsigned)col; }
    __device__ __forceinline__ void store(unsigned at, float x) const {
#if defined(__HIP_DEVICE_COMPILE__)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x), rsrc, at, 0, 0);
#endif
    }
    __device__ __forceinline__ float load(unsigned at) const {
#if defined(__HIP_DEVICE_COMPILE__)
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsrc, at, 0, 0));
#else
        return 0.f;
#endif
    }
};

// C = acc, or C += acc.
struct Store {
    int accumulate;      // (a bool would be kept in scratch memory)

    template <int N>
    struct Fetched {};
    template <int N, class Row, class Mine>
    __device__ __forceinline__ void fetch(Fetched<N> &, int, int, int, Row, Mine) const {}
    template <int NS, class Acc, class Row, class Mine>
    __device__ __forceinline__ void block(const Acc &acc, const Fetched<NS> &, int col, int M,
                                          float *C, int64_t ldc, Row row, Mine mine) const {
        const TileRows c(C, ldc, M);
        const unsigned first = c.at(row(0), col);
        if (accumulate) {
            float old[NS];
#pragma unroll
            for (int r = 0; r < NS; ++r) old[r] = mine(r) ? c.load(first + c.at(row(r) - row(0), 0)) : 0.f;
#pragma unroll
            for (int r = 0; r < NS; ++r)
                if (mine(r)) c.store(first + c.at(row(r) - row(0), 0), old[r] + acc[r]);
        } else {
#pragma unroll
            for (int r = 0; r < NS; ++r)
                if (mine(r)) c.store(first + c.at(row(r) - row(0), 0), acc[r]);
        }
    }
};

// Z = acc + bias (unless NULL), C = act(Z).
struct TileLayer {
    const float *bias;   // NULL: none
    float *Z;
    int64_t ldz;
    int act;

    template <int N>
    struct Fetched {
        float bias;
    };
    template <int NS, class Row, class Mine>
    __device__ __forceinline__ void fetch(Fetched<NS> &f, int col, int, int N, Row, Mine) const {
        f.bias = bias && col < N ? bias[col] : 0.f;
    }
    template <int NS, class Acc, class Row, class Mine>
    __device__ __forceinline__ void block(const Acc &acc, const Fetched<NS> &f, int col, int M,
                                          float *C, int64_t ldc, Row row, Mine mine) const {
        float z[NS];
#pragma unroll
        for (int r = 0; r < NS; ++r) z[r] = acc[r] + f.bias;
        if (Z) {
            const TileRows kept(Z, ldz, M);
            const unsigned first = kept.at(row(0), col);
#pragma unroll
            for (int r = 0; r < NS; ++r)
                if (mine(r)) kept.store(first + kept.at(row(r) - row(0), 0), z[r]);
        }
        const TileRows c(C, ldc, M);
        const unsigned first = c.at(row(0), col);
        with_act(act, [&](auto a) {
#pragma unroll
            for (int r = 0; r < NS; ++r)
                if (mine(r)) c.store(first + c.at(row(r) - row(0), 0), act_value<decltype(a)::value>(z[r]));
        });
    }
};

// The same for outputs whose rows lie further apart.
struct FarStore : Store {
    template <int NS, class Acc, class Row, class Mine>
    __device__ __forceinline__ void block(const Acc &acc, const Fetched<NS> &, int col, int M,
                                          float *C, int64_t ldc, Row row, Mine mine) const {
#pragma unroll
        for (int r = 0; r < NS; ++r) {
            if (!mine(r) || row(r) >= M) continue;
            float *c = C + (int64_t)row(r) * ldc + col;
            *c = accumulate ? *c + acc[r] : acc[r];
        }
    }
};
struct FarLayer : Layer {};

// The epilogue of a group's tile at (row, n) of the output, with the group's
// bias `bias` floats on.
__device__ __forceinline__ Store at_tile(const Store &s, int64_t, int64_t, int64_t) { return s; }
__device__ __forceinline__ TileLayer at_tile(const Layer &l, int64_t bias, int64_t row, int64_t n) {
    return {l.bias ? l.bias + bias + n : nullptr, l.Z ? l.Z + row * l.ldz + n : nullptr, l.ldz, l.act};
}
__device__ __forceinline__ FarStore at_tile(const FarStore &s, int64_t, int64_t, int64_t) { return s; }
__device__ __forceinline__ Layer at_tile(const FarLayer &l, int64_t bias, int64_t row, int64_t n) {
    const TileLayer t = at_tile(static_cast<const Layer &>(l), bias, row, n);
    return {t.bias, nullptr, 0, t.Z, t.ldz, t.act};
}
inline FarStore far(const Store &s) { return {s}; }
inline FarLayer far(const Layer &l) { return {l}; }
inline bool is_far(const Store &, int64_t ldc) { return ldc > NEAR_LD; }
inline bool is_far(const Layer &l, int64_t ldc) { return ldc > NEAR_LD || l.ldz > NEAR_LD; }

// Rows of a grouped product: C_i = A[rows_i] . B_e.
struct GroupedRows {
    Groups g;
    int N, K, T;                   // T: rows of A where rows picks them
    const float *A, *B;
    const int32_t *rows;           // NULL: A_i
    float *C;
    int64_t lda, ldb, strideb, ldc, ldbias;
};

template <int BM, int BN, bool BX, int KS, int WPG, bool KT, class E>
__global__ __launch_bounds__(64 * WPG * KS) void grouped_rows_kernel(GroupedRows a, E epi, int most) {
    using S = TileShape<BM, BN, true, BX, KS, WPG, KT, 32>;
    const int tiles_n = tiles_of(a.N, BN);
    GroupTiles<BM> tiles(a.g, most);
    const int64_t bid = group_number(), n = (int64_t)tiles.number * tiles_n;
    if (bid >= n) return;
    const int lane = threadIdx.x & 63;
    const int wq = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % WPG;
    int tm, tn;
    tile_at(xcd_run((int)bid, (int)n), tiles.number, tiles_n, tm, tn);
    const GroupTile t = tiles[tm];
    const int n0 = tn * BN, left = min(t.left, BM), cols = a.N - n0;

    NearSlabs<typename S::OA, true> sa{{}, a.A, a.lda, left, a.K};
    if (a.rows) {
        const int32_t *rows = a.rows + t.row;
        sa.X = a.T;
        sa.op.init(a.lda, 0, left, lane, wq, [&](int row) {
            return (int)min((unsigned)rows[min(row, left - 1)], (unsigned)a.T - 1);
        });
    } else {
        sa.P += t.row * a.lda;
        sa.op.init(a.lda, 0, left, lane, wq);
    }
    NearSlabs<typename S::OB, BX> sb{{}, a.B + t.e * a.strideb + (BX ? n0 * a.ldb : n0), a.ldb,
                                     BX ? min(cols, BN) : cols, a.K};
    sb.op.init(a.ldb, 0, cols, lane, wq);
    direct_tile<BM, BN, true, BX, KS, WPG, KT, 32>(left, cols, a.K, sa, sb, a.C + t.row * a.ldc + n0,
                                                     a.ldc, at_tile(epi, t.e * a.ldbias, t.row, n0), 0, 0);
}

// The same on few rows per group: tiles of MB rows, as linear_f32.hip's kernels
// for few rows.
template <int MB, bool BX, int KW, int ROWS>
__global__ __launch_bounds__(64 * KW * ROWS) void grouped_few_kernel(GroupedRows a, Layer epi, int most) {
    constexpr int COLS = BX ? ROWS : 32;
    const int tiles_n = tiles_of(a.N, COLS);
    GroupTiles<MB> tiles(a.g, most);
    const int64_t bid = group_number();
    if (bid >= (int64_t)tiles.number * tiles_n) return;
    const GroupTile t = tiles[(int)(bid / tiles_n)];
    const int64_t n0 = bid % tiles_n * COLS;
    const int left = min(t.left, MB);
    const int32_t *rows = a.rows ? a.rows + t.row : nullptr;
    const float *A = a.rows ? a.A : a.A + t.row * a.lda;
    const auto x = [&](int m) {
        return A + (rows ? (int64_t)min((unsigned)rows[m], (unsigned)a.T - 1) : (int64_t)m) * a.lda;
    };
    const float *W = a.B + t.e * a.strideb;
    const TileLayer l = at_tile(epi, t.e * a.ldbias, t.row, 0);
    const Layer e{l.bias, nullptr, 0, l.Z, l.ldz, l.act};
    float *Y = a.C + t.row * a.ldc;
    if constexpr (BX) few_nk<MB, KW, ROWS>(left, a.N, a.K, x, W, a.ldb, Y, a.ldc, e, n0);
    else few_kn<MB, KW>(left, a.N, a.K, x, W, a.ldb, Y, a.ldc, e, n0);
}

// Gradients of the weights and, of the tiles of DZ_ROWS rows that the element pass
// summed, of the biases.
constexpr int DZ_ROWS = 128;

// db_e: a wave adds 64 columns' sums over its group's tiles, in 8 interleaved runs.
struct BiasSums {
    const float *partial;          // most x N
    float *db;                     // NULL: not wanted
    int64_t lddb;
    int N, most, accumulate;
    __host__ __device__ int64_t waves(int E) const { return db ? ((int64_t)N + 63) / 64 * E : 0; }
    __device__ __forceinline__ void columns(const Groups &g, int64_t wave) const {
        if (wave >= waves(g.E)) return;
        const int64_t blocks = ((int64_t)N + 63) / 64;
        const int e = (int)(wave / blocks);
        const int from = (int)min(tiles_before<DZ_ROWS>(g, e), (int64_t)most);
        int first, count;
        group_rows(g, e, first, count);
        const int end = (int)min((int64_t)from + tiles_in<DZ_ROWS>(count), (int64_t)most);
        const int64_t col = wave % blocks * 64 + (threadIdx.x & 63);
        if (col >= N) return;
        float run[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int i = from; i < end; i += 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = partial[(int64_t)min(i + u, end - 1) * N + col];
#pragma unroll
            for (int u = 0; u < 8; ++u) run[u] += i + u < end ? v[u] : 0.f;
        }
        float sum = run[0];
#pragma unroll
        for (int u = 1; u < 8; ++u) sum += run[u];
        float *to = db + e * lddb + col;
        *to = accumulate ? *to + sum : sum;
    }
};

// dW_e = A_e^T . B_e over the rows of group e, A and B stored row by row; PICK:
// which of them is read through `rows`.
enum Pick { NEITHER, PICK_A, PICK_B };
struct GroupedWeights {
    Groups g;
    int M, N, T;                   // output M x N
    const float *A, *B;
    const int32_t *rows;
    float *C;
    int64_t lda, ldb, ldc, stridec;
    bool by_size;                  // the largest groups first
    BiasSums bias;                 // what the first workgroups do, if anything
    int bias_groups;
};

template <int BM, int BN, int KS, int WPG, Pick PICK, class E>
__global__ __launch_bounds__(64 * WPG * KS) void grouped_weights_kernel(GroupedWeights a, E epi) {
    using S = TileShape<BM, BN, false, false, KS, WPG, false, 32>;
    const int tiles_m = tiles_of(a.M, BM), tiles_n = tiles_of(a.N, BN), per = tiles_m * tiles_n;
    const int64_t bid = group_number() - a.bias_groups, n = (int64_t)per * a.g.E;
    if (bid >= n) return;
    if (bid < 0) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        return a.bias.columns(a.g, group_number() * (KS * WPG) + wave);
    }
    // every XCD takes a part of each expert: groups differ in size, so that an
    // expert per XCD would leave most of them waiting for the largest
    const OneGroup g = group_at(a.g, (int)(bid / per), a.by_size, a.g.M / a.g.E);
    const int e = g.e, first = g.first, count = g.count, place = xcd_run((int)(bid % per), per);
    if (count == 0 && epi.accumulate) return;
    const int lane = threadIdx.x & 63;
    const int wq = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % WPG;
    int tm, tn;
    tile_at(place, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    float *C = a.C + e * a.stridec + m0 * a.ldc + n0;
    const auto near = [&](auto op, const float *P, int64_t ld, int X) {
        NearSlabs<decltype(op), false> s{op, P + first * ld, ld, X, count};
        s.op.init(ld, 0, X, lane, wq);
        return s;
    };
    const auto picked = [&](auto op, const float *P, int64_t ld, int X) {
        PickedSlabs<decltype(op)> s;
        s.op = op, s.P = P, s.ld = ld, s.X = X, s.rows = a.rows + first, s.K = count, s.T = a.T;
        s.init(X, lane, wq);
        return s;
    };
    const auto product = [&](auto sa, auto sb) {
        direct_tile<BM, BN, false, false, KS, WPG, false, 32>(a.M - m0, a.N - n0, count, sa, sb, C, a.ldc, epi, 0, 0);
    };
    const typename S::OA oa{};
    const typename S::OB ob{};
    if constexpr (PICK == PICK_A) product(picked(oa, a.A + m0, a.lda, a.M - m0), near(ob, a.B + n0, a.ldb, a.N - n0));
    else if constexpr (PICK == PICK_B) product(near(oa, a.A + m0, a.lda, a.M - m0), picked(ob, a.B + n0, a.ldb, a.N - n0));
    else product(near(oa, a.A + m0, a.lda, a.M - m0), near(ob, a.B + n0, a.ldb, a.N - n0));
}

// ---------------------------------------------------------------------------
// dZ = dY * act'(Z) and the column sums of each tile of DZ_ROWS rows, as the
// dense layer's element pass (linear_bwd.hip): 64 columns per workgroup, 16
// lanes of 4 columns by 16 rows at a time.

__global__ __launch_bounds__(256) void grouped_dz_kernel(Groups g, int act, int N, const float *dY,
                                                         int64_t lddy, const float *Z, int64_t ldz,
                                                         float *dZ, int64_t lddz, float *partial, int most) {
    __shared__ v4f red[256];
    const int tiles_n = tiles_of(N, 64);
    GroupTiles<DZ_ROWS> tiles(g, most);
    const int64_t bid = group_number();
    if (bid >= (int64_t)tiles.number * tiles_n) return;
    const int tm = (int)(bid / tiles_n);
    const GroupTile t = tiles[tm];
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const int64_t col = bid % tiles_n * 64 + 4 * tx;
    const int live = (int)min(max(N - col, (int64_t)0), (int64_t)4);   // columns of this thread that exist
    const int64_t end = (int64_t)t.row + min(t.left, DZ_ROWS);
    v4f sum = {0.f, 0.f, 0.f, 0.f};
    with_act(act, [&](auto a) {
        constexpr int ACT = decltype(a)::value;
#pragma unroll 4
        for (int64_t r = t.row + ty; r < end; r += 16) {
            const float *pd = dY + r * lddy + col;
            const float *pz = Z + r * ldz + col;
            v4f d = {0.f, 0.f, 0.f, 0.f}, z = d;
            if (live == 4) {
                d = *reinterpret_cast<const v4f_any *>(pd);
                if (ACT != GG_ACT_NONE) z = *reinterpret_cast<const v4f_any *>(pz);
            } else {
#pragma unroll
                for (int c = 0; c < 3; ++c) {
                    if (c >= live) continue;
                    d[c] = pd[c];
                    if (ACT != GG_ACT_NONE) z[c] = pz[c];
                }
            }
            if constexpr (ACT != GG_ACT_NONE) {
                float *po = dZ + r * lddz + col;
#pragma unroll
                for (int c = 0; c < 4; ++c) d[c] *= act_slope<ACT>(z[c]);
                if (live == 4) {
                    *reinterpret_cast<v4f_any *>(po) = d;
                } else {
#pragma unroll
                    for (int c = 0; c < 3; ++c)
                        if (c < live) po[c] = d[c];
                }
            }
            sum += d;
        }
    });
    if (partial == nullptr) return;                   // uniform
    red[threadIdx.x] = sum;
    __syncthreads();
    if (ty == 0) {
#pragma unroll
        for (int y = 1; y < 16; ++y) sum += red[y * 16 + tx];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < live) partial[(int64_t)tm * N + col + c] = sum[c];
    }
}

__global__ __launch_bounds__(256) void grouped_bias_kernel(Groups g, BiasSums b) {
    b.columns(g, group_number() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
}

// ---------------------------------------------------------------------------

template <int BM, int BN, bool BX, int KS, int WPG, class E>
hipError_t rows_tiles(const GroupedRows &a, const E &epi, hipStream_t s) {
    const int64_t most = tiles_most(a.g.M, a.g.E, BM), n = most * (((int64_t)a.N + BN - 1) / BN);
    if (n > INT_MAX) return hipErrorInvalidConfiguration;
    // (K a multiple of 4 apart: 8192 x 2048 x 1024 3.6% faster without the code for
    // chunks that K cuts)
    return a.K % 4 ? launch(grouped_rows_kernel<BM, BN, BX, KS, WPG, true, E>, grid_of(n), dim3(64 * WPG * KS), s, a, epi, (int)most)
                   : launch(grouped_rows_kernel<BM, BN, BX, KS, WPG, false, E>, grid_of(n), dim3(64 * WPG * KS), s, a, epi, (int)most);
}

template <int MB, bool BX, int KW, int ROWS>
hipError_t few_tiles(const GroupedRows &a, const Layer &epi, hipStream_t s) {
    constexpr int COLS = BX ? ROWS : 32;
    const int64_t most = tiles_most(a.g.M, a.g.E, MB), n = most * (((int64_t)a.N + COLS - 1) / COLS);
    if (n > INT_MAX) return hipErrorInvalidConfiguration;
    return launch(grouped_few_kernel<MB, BX, KW, ROWS>, grid_of(n), dim3(64 * KW * ROWS), s, a, epi, (int)most);
}

// The tile of a product of grouped rows, by how many there are likely to be.
// Tiles of 32 rows throughout: a group leaves 16 rows of its last tile empty on
// average, with 64 rows 32, and the last round of tiles is shorter.  (2048 x 1024,
// us in 32 x 64 against 64 x 64, both in 2 k-groups, for groups of like, not the
// same size: 2,048 rows of 8 groups 83 / 89, 4,096 153 / 157, 8,192 of 8 284 / 290,
// of 64 342 / 375, of one 286 / 279.)  The k-groups by how many tiles a CU holds at
// once (us, K = 768, groups of like size):
//
//   rows, groups, N    32 x 64 in 1   in 2   in 4   32 x 32 in 8
//     64,  8,  768         17.1       11.0   10.2        7.3
//    256,  8, 2304         27.0       17.2   20.8       26.6
//    768,  8, 2304         30.6       35.4   38.5       50.6
//   1536, 32,  768         29.9       31.8   40.1       44.5
//     64, 128, 768         28.5       24.9   34.0       43.1
//    128, 128, 768         32.6       40.3   47.5       60.6
//
// One 32 x 32 tile in 8 k-groups, or one 32 x 64 in 4, fills a CU's LDS; 3 in 2
// k-groups and 6 in 1 do.  Longer grids run in 2 as fast as in 1 or faster where K
// is long enough for its tiles' ends not to matter (8192 rows of 8 groups, 2048
// outputs: K = 256 93 against 84, 512 157 / 151, 768 221 / 218, 1024 282 / 285, 2048
// 544 / 557; 4096 rows, 1024 outputs, K = 512 45.6 / 46.6, 2048 151 / 167).
template <bool BX, class E>
hipError_t rows_product(const GroupedRows &a, const E &epi, int num_cus, hipStream_t s) {
    const int64_t rows = tiles_likely(a.g.M, a.g.E, 32), cus = num_cus;
    const int64_t quarters = rows * (((int64_t)a.N + 31) / 32), tiles = rows * (((int64_t)a.N + 63) / 64);
    const int slabs = slabs_of<32>(a.K);              // a k-group should have one at least
    if (is_far(epi, a.ldc)) return rows_tiles<32, 64, BX, 1, 2>(a, far(epi), s);
    if (slabs >= 8 && quarters <= cus) return rows_tiles<32, 32, BX, 8, 1>(a, epi, s);
    if (slabs >= 8 && tiles <= cus) return rows_tiles<32, 64, BX, 4, 2>(a, epi, s);
    if (slabs >= 4 && (tiles <= 3 * cus || (4 * tiles > 19 * cus && slabs >= 20)))
        return rows_tiles<32, 64, BX, 2, 2>(a, epi, s);
    return rows_tiles<32, 64, BX, 1, 2>(a, epi, s);
}

// Up to 16 rows, where groups have one or two at most: a kernel that reads each
// group's matrix once, without tiles (us, 8 groups of N x K = 2304 x 768 /
// 768 x 2304, against the best tile):
//   W stored K x N   2 rows 5.1 / 7.7 against 7.5 / 13.5, 4 rows 6.5 / 7.9 against
//                    11.1 / 14.1, 8 rows 10.9 / 11.3 against 12.4 / 14.5, 16 rows 11.0 /
//                    13.0 against 12.3 / 14.5, 32 rows 17.5 / 16.7 against 16.8 / 15.3
//   W stored N x K   2 rows 4.4 / 3.9 against 7.2 / 12.9, 8 rows 10.0 / 8.8 against
//                    13.1 / 14.2, 16 rows 13.4 / 10.0 against 13.0 / 14.1
// K x N: 16 waves per 32 columns where that is a workgroup per CU at most, else 8 (2
// rows, 2304 x 768: 5.1 against 5.3; 4 rows 7.0 / 6.5).  N x K: one row at a time
// where few groups have more (2 rows 4.4 against 4.8 and 3.9 / 4.5, 8 rows 11.1 /
// 10.0 and 8.3 / 8.8).  Its workgroups have 4 or 32 columns: outputs of so many that
// a grid does not hold them go to the tiles, of 32 rows by 32 columns at least.
inline bool few_rows(const GroupedRows &a, bool nk) {
    const int64_t M = a.g.M, E = a.g.E;
    if (M * tiles_of(a.N, nk ? 4 : 32) > INT_MAX) return false;      // a row per group at most
    return M <= 16 && (M <= E || (M <= 2 * E && (!nk || a.N <= 2048)));
}

template <bool BX>
hipError_t few_product(const GroupedRows &a, const Layer &epi, int num_cus, hipStream_t s) {
    if constexpr (BX) {
        return 2 * (int64_t)a.g.M <= a.g.E ? few_tiles<1, true, 1, 4>(a, epi, s) : few_tiles<2, true, 1, 4>(a, epi, s);
    } else {
        const int64_t M = a.g.M, slabs = ((int64_t)a.N + 31) / 32;
        const bool wide = M * slabs <= num_cus;
        if (M <= a.g.E) return wide ? few_tiles<1, false, 16, 1>(a, epi, s) : few_tiles<1, false, 8, 1>(a, epi, s);
        return wide ? few_tiles<2, false, 16, 1>(a, epi, s) : few_tiles<2, false, 8, 1>(a, epi, s);
    }
}

template <bool BX>
hipError_t layer_product(const GroupedRows &a, const Layer &epi, int num_cus, hipStream_t s) {
    return few_rows(a, BX) ? few_product<BX>(a, epi, num_cus, s) : rows_product<BX>(a, epi, num_cus, s);
}

template <int KS, Pick PICK, class E>
hipError_t weights_tiles(GroupedWeights a, const E &epi, int64_t n, hipStream_t s) {
    a.bias_groups = (int)((a.bias.waves(a.g.E) + 4 * KS - 1) / (4 * KS));
    return launch(grouped_weights_kernel<64, 64, KS, 4, PICK, E>, grid_of(a.bias_groups + n), dim3(256 * KS), s, a, epi);
}

// 64 x 64 tiles, four workgroups of which share a CU, the largest groups' first
// (4096 rows in 8 groups of 36 to 1632, 2048 x 1024: 160 us, in the groups' order
// 205); only where a CU has one or
// two and they walk far, in 4 k-groups (us in 1 / 4, for groups of like size):
//   4096 rows of one group, 768 x 768 (144 tiles)     104 / 83
//   16384 of 2, 768 x 768 (288)                       323 / 290, 4096 of 2: 85 / 86
//   65536 of 8, 512 x 512 (512)                       330 / 304
//   1000 of 2, 2048 x 1024 (1,024)                    43 / 63,   8192 of 2: 288 / 300
//   300 of 3, 230 x 230 (48)                          6.8 / 11.4
// In 2 k-groups no size gained over the better of the two, and tiles of 128 x 64
// and 128 x 128 took longer but in the largest products (16384 rows of 8, 2048 x
// 1024: 573, 565 and 577).
template <Pick PICK>
hipError_t weights_product(const GroupedWeights &a, const Store &epi, int num_cus, hipStream_t s) {
    const int64_t per = (((int64_t)a.M + 63) / 64) * (((int64_t)a.N + 63) / 64), n = per * a.g.E;
    if (per > INT_MAX / a.g.E) return hipErrorInvalidConfiguration;
    const int rows = a.g.M / a.g.E;
    if (is_far(epi, a.ldc)) return weights_tiles<1, PICK>(a, far(epi), n, s);
    if ((n <= num_cus && rows >= 1024) || (n <= 2 * (int64_t)num_cus && rows >= 4096))
        return weights_tiles<4, PICK>(a, epi, n, s);
    return weights_tiles<1, PICK>(a, epi, n, s);
}

}  // namespace

int64_t grouped_dz_tiles(int64_t M, int64_t E) { return tiles_most(M, E, DZ_ROWS); }

hipError_t launch_linear_grouped(const LinearGrouped &a, int num_cus, hipStream_t s) {
    const GroupedRows r{{a.offsets, a.E, a.M}, a.N, a.K, a.T, a.X, a.W, a.rows, a.Y,
                        a.ldx, a.ldw, a.stridew, a.ldy, a.ldb};
    const Layer e{a.bias, nullptr, 0, a.Z, a.ldz, a.act};
    return a.trans_w ? layer_product<true>(r, e, num_cus, s) : layer_product<false>(r, e, num_cus, s);
}

hipError_t launch_linear_grouped_bwd(const LinearGroupedBwd &a, int num_cus, hipStream_t s) {
    const Groups g{a.offsets, a.E, a.M};
    hipError_t e = hipSuccess;
    const float *dZ = a.dY;
    int64_t lddz = a.lddy;
    BiasSums bias{};
    if (a.N > 0 && (a.act != GG_ACT_NONE || a.db != nullptr)) {
        const int64_t most = grouped_dz_tiles(a.M, a.E), cols = ((int64_t)a.N + 63) / 64;
        float *out = a.ws, *partial = a.ws;
        if (a.act != GG_ACT_NONE) {
            lddz = dz_stride(a.N);
            partial = a.ws + (int64_t)a.M * lddz;
            dZ = out;
        }
        if (most * cols > INT_MAX || cols * a.E > INT_MAX) return hipErrorInvalidConfiguration;
        if (most > 0)
            e = launch(grouped_dz_kernel, grid_of(most * cols), dim3(256), s, g, a.act, a.N, a.dY, a.lddy, a.Z, a.ldz,
                       out, lddz, a.db ? partial : nullptr, (int)most);
        if (e != hipSuccess) return e;
        // in the launch of dW where there is one (all gradients of 64 rows of 8 groups, 768
        // x 768: 21.2 us, 23.3 in one of its own)
        if (a.db) bias = {partial, a.db, a.lddb, a.N, (int)most, a.accumulate ? 1 : 0};
        if (a.db && !a.dW)
            e = launch(grouped_bias_kernel, grid_of((bias.waves(a.E) + 3) / 4), dim3(256), s, g, bias);
        if (e != hipSuccess) return e;
    }
    if (a.dX) {
        const GroupedRows r{g, a.K, a.N, 0, dZ, a.W, nullptr, a.dX, lddz, a.ldw, a.stridew, a.lddx, 0};
        e = a.trans_w ? rows_product<false>(r, Store{0}, num_cus, s)
                      : rows_product<true>(r, Store{0}, num_cus, s);
        if (e != hipSuccess) return e;
    }
    if (a.dW) {
        // finding the order takes 2 to 4% where groups are of like size (64 rows each of
        // 64, 1024 x 1024: 143 against 137 us; 512 each of 8, 2048 x 1024: 162 / 161)
        const bool by_size = a.M >= 128 * (int64_t)a.E;
        GroupedWeights w{g, a.K, a.N, a.T, a.X, dZ, a.rows, a.dW, a.ldx, lddz, a.lddw, a.stridedw, by_size, bias, 0};
        if (a.trans_w) w = {g, a.N, a.K, a.T, dZ, a.X, a.rows, a.dW, lddz, a.ldx, a.lddw, a.stridedw, by_size, bias, 0};
        const Store st{a.accumulate ? 1 : 0};
        e = !a.rows ? weights_product<NEITHER>(w, st, num_cus, s)
            : a.trans_w ? weights_product<PICK_B>(w, st, num_cus, s) : weights_product<PICK_A>(w, st, num_cus, s);
    }
    return e;
}

}  // namespace gg
