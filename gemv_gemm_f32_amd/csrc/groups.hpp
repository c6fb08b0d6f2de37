// groups.hpp -- rows grouped by expert: group e is the rows offsets[e] ..
// offsets[e + 1] - 1 of M, and a workgroup finds its tile among tiles that
// never span two groups.
//
// Only the device knows the groups' sizes, so a launch has as many workgroups
// as any sizes could need (tiles_most) and those past the end return at once.
// Each wave finds its tile by itself, without a barrier: a lane per group, the
// groups' tile counts summed over the lanes, 64 groups at a time.  The offsets
// are bounded to 0 .. M as they are read, so whatever they hold, no row
// outside of the M is touched.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wave.hpp"

namespace gg {

struct Groups {
    const int32_t *offsets;   // E + 1
    int E, M;
};

// Tiles of BM rows that M rows in E groups can need at most.
inline int64_t tiles_most(int64_t M, int64_t E, int64_t BM) {
    const int64_t n = (M + E * (BM - 1)) / BM;
    return n < M ? n : M;
}

// The rows of group e, for e < E; none for others.  Whatever the offsets hold,
// 0 <= first <= first + count <= M.
__host__ __device__ inline void group_rows(const Groups &g, int e, int &first, int &count) {
    first = count = 0;
    if (e < g.E) {
        const int from = g.offsets[e], to = g.offsets[e + 1];
        first = from < 0 ? 0 : from < g.M ? from : g.M;
        const int end = to < g.M ? to : g.M;
        count = end > first ? end - first : 0;
    }
}

template <int BM>
__device__ __forceinline__ int tiles_in(int count) { return count / BM + (count % BM != 0); }

// Tiles of all groups, and, with `upto` groups, of the first ones.
template <int BM>
__device__ __forceinline__ int tiles_before(const Groups &g, int upto) {
    const int lane = threadIdx.x & 63;
    int sum = 0;
    for (int c = 0; c < upto; c += 64) {
        int first, count;
        group_rows(g, c + lane < upto ? c + lane : g.E, first, count);
        sum += __builtin_amdgcn_readlane(wave64_scan(tiles_in<BM>(count)), 63);
    }
    return sum;
}

// Tile number t of all (t below their number): its group, the tile's first
// row and how many of the group's rows there are from there on.
struct GroupTile {
    int e, row, left;
};
template <int BM>
__device__ __forceinline__ GroupTile tile_of_groups(const Groups &g, int t) {
    const int lane = threadIdx.x & 63;
    for (int c = 0; c < g.E; c += 64) {
        int first, count;
        group_rows(g, c + lane, first, count);
        const int n = tiles_in<BM>(count), incl = wave64_scan(n);
        const uint64_t past = __ballot(incl > t);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            const int skip = (t - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(n, l))) * BM;
            return {c + l, __builtin_amdgcn_readlane(first, l) + skip,
                    __builtin_amdgcn_readlane(count, l) - skip};
        }
        t -= __builtin_amdgcn_readlane(incl, 63);
    }
    return {0, 0, 0};
}

// Workgroups in a grid of up to 65,535 x 2^20, and one's number.
__device__ __forceinline__ int64_t group_number() {
    return (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

// The place in the tile order of workgroup `bid` of n: workgroups are handed to
// the 8 XCDs in turn, so that each XCD gets a run of neighbouring tiles.
__host__ __device__ inline int xcd_run(int bid, int n) {
    const int x = bid & 7, left = n & 7;
    return x * (n >> 3) + (x < left ? x : left) + (bid >> 3);
}

inline dim3 grid_of(int64_t n) {
    const int64_t most = 1 << 20;
    return n <= most ? dim3((unsigned)n) : dim3((unsigned)most, (unsigned)((n + most - 1) / most));
}

}  // namespace gg
