// linear_mx8_grouped.hip -- the packed layers on rows grouped by expert: the
// tiles of linear_mx8_tile.hpp, each within one group (groups.hpp), on that
// expert's codes, scales and bias, in one launch for all experts.  The rows of
// X that a group picks are found as its tile loads them; no copy in grouped
// order is made.
#include <hip/hip_runtime.h>

#include <climits>

#include "groups.hpp"
#include "kernels.hpp"
#include "linear_mx8_tile.hpp"

namespace gg {
namespace {

// The layer of tile t of BM rows at most, its row 0 the tile's first row.
template <int BM>
__device__ __forceinline__ PackedLinear layer_of(const PackedGrouped &a, const GroupTile &t) {
    PackedLinear p = a.layer;
    p.M = min(t.left, BM);
    p.Q += t.e * a.strideq;
    p.S += t.e * a.strides;
    if (p.bias) p.bias += t.e * a.ldb;
    if (p.Y) p.Y += t.row * p.ldy;
    if (p.Y8) {
        p.Y8 += t.row * p.ldy8;
        p.YE += t.row * p.ldye;
    }
    return p;
}

// The rows of X that feed a tile's rows.
struct PickedRow {
    const int32_t *rows;
    int first, T;
    __device__ __forceinline__ PickedRow(const PackedGrouped &a, const GroupTile &t)
        : rows(a.rows), first(t.row), T(a.T) {}
    __device__ __forceinline__ int64_t operator()(int64_t m) const {
        return rows ? (int64_t)min((unsigned)rows[first + m], (unsigned)T - 1) : first + m;
    }
};

// Workgroup -> (tile of rows, tile of columns): runs of neighbouring tiles per
// XCD, rows first.  False for workgroups past the end.
template <int BM>
__device__ __forceinline__ bool find_tile(const PackedGrouped &a, int bn, int most, GroupTile &t, int64_t &n0) {
    const Groups g{a.offsets, a.E, a.layer.M};
    GroupTiles<BM> tiles(g, most);
    const int tiles_n = tiles_of(a.layer.N, bn);
    const int64_t bid = group_number(), n = (int64_t)tiles.number * tiles_n;
    if (bid >= n) return false;
    const int tb = xcd_run((int)bid, (int)n);
    t = tiles[tb % tiles.number];
    n0 = (int64_t)(tb / tiles.number) * bn;
    return true;
}

template <int BITS, int NH, int KW>
__global__ __launch_bounds__(64 * NH * KW) void packed_rows_grouped(PackedGrouped a, int most) {
    GroupTile t;
    int64_t n0;
    if (!find_tile<16>(a, 16 * NH, most, t, n0)) return;
    packed_rows<BITS, NH, KW>(layer_of<16>(a, t), n0, PickedRow(a, t));
}

template <int KW, int BITS, int MW>
__global__ __launch_bounds__(64 * KW, MW) void packed_block_grouped(PackedGrouped a, int most) {
    GroupTile t;
    int64_t n0;
    if (!find_tile<32>(a, 32, most, t, n0)) return;
    packed_block<KW, BITS>(layer_of<32>(a, t), 0, n0, PickedRow(a, t));
}

template <int BM, int NW, int BITS, int MW>
__global__ __launch_bounds__(64 * NW, MW) void packed_wide_grouped(PackedGrouped a, int most) {
    __shared__ __attribute__((aligned(16))) char smem[wide_bytes<BM, NW>()];
    GroupTile t;
    int64_t n0;
    if (!find_tile<BM>(a, 32 * NW, most, t, n0)) return;
    const PackedLinear p = layer_of<BM>(a, t);
    const PickedRow x(a, t);
    // what a group's last tile needs no more than half of runs as one of half
    // the rows
    if constexpr (BM == 64 && NW == 4)
        if (t.left <= 32) {
            packed_wide<32, NW, BITS>(p, 0, n0, x, smem);
            return;
        }
    packed_wide<BM, NW, BITS>(p, 0, n0, x, smem);
}

template <class Kernel>
hipError_t launch_tiles(Kernel kernel, const PackedGrouped &a, int bm, int bn, int threads, hipStream_t s) {
    const int64_t most = tiles_most(a.layer.M, a.E, bm), n = most * (((int64_t)a.layer.N + bn - 1) / bn);
    if (n > INT_MAX) return hipErrorInvalidConfiguration;
    return launch(kernel, grid_of(n), dim3(threads), s, a, (int)most);
}

template <int BITS, int NH, int KW>
hipError_t launch_rows(const PackedGrouped &a, hipStream_t s) {
    return launch_tiles(packed_rows_grouped<BITS, NH, KW>, a, 16, 16 * NH, 64 * NH * KW, s);
}

template <int KW, int BITS, int MW>
hipError_t launch_block(const PackedGrouped &a, hipStream_t s) {
    return launch_tiles(packed_block_grouped<KW, BITS, MW>, a, 32, 32, 64 * KW, s);
}

template <int BM, int NW, int BITS, int MW>
hipError_t launch_wide(const PackedGrouped &a, hipStream_t s) {
    return launch_tiles(packed_wide_grouped<BM, NW, BITS, MW>, a, BM, 32 * NW, 64 * NW, s);
}

// The shape by the rows per group and by how many tiles there are likely to be (us,
// 2 bits; 4 bits ask for the same):
//  - few rows per group: the kernel of few rows.  Where rows of W are short, that is
//    up to 8 in up to 12 tiles of 16 x 16 per CU (8 rows of 64 groups, 1536 x 1536:
//    5.2, in 32 x 128 tiles 10.3; 64 of 64, 15 per CU: 16.0 / 14.9); where they are
//    long, up to 4 (64 of 64, 1536 x 12288: 82 / 90; 256 of 32, 1536 x 8192: 62, in
//    32 x 32 cells 53) or, in a tile per CU, 16 (16 rows, 4096 x 4096: 6.7 / 9.0).  A
//    tile's k in 4 runs, but 16 (8 with an output in 8 bits) for long rows and a
//    tile per CU (8 rows, 4096 x 4096: 5.9 / 6.2 in 4) and 1 (2) for short ones and
//    many tiles (32 of 16, 2304 x 768: 7.1 / 7.6 in 4; but 16 of 16, 1536 x 1536: 6.8
//    / 5.8).
//  - up to 8 cells of 32 x 32 per CU and long rows, 4 and 1536 columns: a wave per run
//    of k in each (256 rows of 8 groups, 1536 x 12288: 45, in 32 x 128 66; 512 of 16,
//    4096 x 4096, 12 per CU: 58 / 54; 256 of 16, 1536 x 1536: 9.4 / 10.6).
//  - less than 16 rows per group, or up to 2.5 tiles of 64 x 128 per CU: 32 x 128 (1024
//    rows of 32 groups, 2304 x 2304: 28, in 64 x 128 38; 512 of 16, 2304 x 768: 9.7 /
//    13.6; 512 of 16, 4096 x 4096: 54 / 50).
//  - 128 x 256 for large groups and products (4,096 rows of 8 groups, 4096 x 4096:
//    201 / 217 at 4 bits, 210 / 234 in 64 x 128).
//  - else 64 x 128, a last tile of up to 32 rows as 32 x 128 (1,000 rows of 16 groups,
//    12288 x 1536: 78, all in 64 x 128 89, all in 32 x 128 88).
template <int BITS>
hipError_t launch_bits(const PackedGrouped &a, int num_cus, hipStream_t s) {
    const int64_t M = a.layer.M, E = a.E, N = a.layer.N, K = a.layer.K, cus = num_cus;
    const auto tiles = [&](int bm, int bn) { return tiles_likely(M, E, bm) * ((N + bn - 1) / bn); };
    const bool lengthy = K >= 4096;
    const int64_t sixteens = tiles(16, 16);
    // (4,096 per CU is out of reach but for huge outputs, which need a grid of larger tiles)
    const bool few = lengthy ? (M <= 4 * E && sixteens <= 4096 * cus) || (M <= 16 * E && sixteens <= cus)
                             : M <= 8 * E && sixteens <= 12 * cus;
    if (few) {
        const bool one_run = K < 1536 && sixteens > 4 * cus, most_runs = lengthy && sixteens <= cus;
        if (a.layer.Y8)
            return one_run ? launch_rows<BITS, 2, 2>(a, s)
                   : most_runs ? launch_rows<BITS, 2, 8>(a, s) : launch_rows<BITS, 2, 4>(a, s);
        return one_run ? launch_rows<BITS, 1, 1>(a, s)
               : most_runs ? launch_rows<BITS, 1, 16>(a, s) : launch_rows<BITS, 1, 4>(a, s);
    }
    if (K >= 1536 && tiles(32, 32) <= (lengthy ? 8 : 4) * cus) return launch_block<4, BITS, 3>(a, s);
    if (M < 16 * E || 2 * tiles(64, 128) <= 5 * cus) return launch_wide<32, 4, BITS, 3>(a, s);
    if (M >= 256 * E && tiles(128, 256) >= 2 * cus) return launch_wide<128, 8, BITS, 2>(a, s);
    return launch_wide<64, 4, BITS, 3>(a, s);
}

}  // namespace

hipError_t launch_packed_grouped(int bits, const PackedGrouped &a, int num_cus, hipStream_t s) {
    return bits == 2 ? launch_bits<2>(a, num_cus, s) : launch_bits<4>(a, num_cus, s);
}

}  // namespace gg
