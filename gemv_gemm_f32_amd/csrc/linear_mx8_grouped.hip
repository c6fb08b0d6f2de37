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
    const int tiles_m = min(tiles_before<BM>(g, g.E), most), tiles_n = (a.layer.N + bn - 1) / bn;
    const int64_t bid = group_number(), n = (int64_t)tiles_m * tiles_n;
    if (bid >= n) return false;
    const int tb = xcd_run((int)bid, (int)n);
    t = tile_of_groups<BM>(g, tb % tiles_m);
    n0 = (int64_t)(tb / tiles_m) * bn;
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
    GroupTile t;
    int64_t n0;
    if (!find_tile<BM>(a, 32 * NW, most, t, n0)) return;
    packed_wide<BM, NW, BITS>(layer_of<BM>(a, t), 0, n0, PickedRow(a, t));
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

template <int BITS>
hipError_t launch_bits(const PackedGrouped &a, int num_cus, hipStream_t s) {
    const int64_t per_group = a.layer.M / a.E;
    if (per_group <= 8) {
        if (a.layer.Y8) return launch_rows<BITS, 2, 4>(a, s);
        return launch_rows<BITS, 1, 4>(a, s);
    }
    if (per_group <= 32) return launch_block<4, BITS, 3>(a, s);
    return launch_wide<64, 4, BITS, 3>(a, s);
}

}  // namespace

hipError_t launch_packed_grouped(int bits, const PackedGrouped &a, int num_cus, hipStream_t s) {
    return bits == 2 ? launch_bits<2>(a, num_cus, s) : launch_bits<4>(a, num_cus, s);
}

}  // namespace gg
