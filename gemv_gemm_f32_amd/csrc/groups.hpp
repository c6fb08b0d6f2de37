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

#include <cmath>

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

// And how many they are likely to need: one for each group that holds any, which
// rows on groups at random leave, or a half-empty one for each beside the full
// tiles.
inline int64_t tiles_likely(int64_t M, int64_t E, int64_t BM) {
    const int64_t some = E ? (int64_t)std::ceil((double)E * -std::expm1(-(double)M / (double)E)) : 0;
    const int64_t full = M / BM + some / 2;
    return some > full ? some : full;
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

// Tiles of `size` that n rows or columns need, for any n below 2^31 (n + size - 1 may
// lie past it).
__host__ __device__ inline int tiles_of(int n, int size) {
    return (int)(((unsigned)n + (unsigned)size - 1) / (unsigned)size);
}

template <int BM>
__device__ __forceinline__ int tiles_in(int count) { return tiles_of(count, BM); }

// Tiles of the first `upto` groups, of 128 rows or so: 64 groups' then fit 32
// bits even where offsets that are not in order count rows more than once.
template <int BM>
__device__ __forceinline__ int64_t tiles_before(const Groups &g, int upto) {
    static_assert(BM >= 64, "64 groups of 2^31 rows");
    const int lane = threadIdx.x & 63;
    int64_t sum = 0;
    for (int c = 0; c < upto; c += 64) {
        int first, count;
        group_rows(g, c + lane < upto ? c + lane : g.E, first, count);
        sum += (unsigned)__builtin_amdgcn_readlane(wave64_scan(tiles_in<BM>(count)), 63);
    }
    return sum;
}

// Tile number t of all: its group, the tile's first row and how many of the
// group's rows there are from there on.
struct GroupTile {
    int e, row, left;
};

// Tiles of all groups, at most `most`, and then one of them.  Up to 64 groups'
// offsets are read once, by the constructor.
template <int BM>
struct GroupTiles {
    const Groups &g;
    int first, count, incl, number;
    __device__ __forceinline__ GroupTiles(const Groups &groups, int most) : g(groups) {
        round(0);
        number = __builtin_amdgcn_readlane(incl, 63);
        for (int c = 64; c < g.E; c += 64) {
            round(c);
            number += __builtin_amdgcn_readlane(incl, 63);
        }
        number = __builtin_amdgcn_readfirstlane(min(number, most));
    }
    // t below number
    __device__ __forceinline__ GroupTile operator[](int t) {
        if (g.E <= 64) return within(0, t);
        for (int c = 0;; c += 64) {
            round(c);
            const int here = __builtin_amdgcn_readlane(incl, 63);
            if (t < here || c + 64 >= g.E) return within(c, t);
            t -= here;
        }
    }

private:
    // a lane per group from c on: its rows, and tiles up to its end
    __device__ __forceinline__ void round(int c) {
        group_rows(g, c + (int)(threadIdx.x & 63), first, count);
        incl = wave64_scan(tiles_in<BM>(count));
    }
    // (The same in every lane, and made so: addresses that the compiler takes for
    // a lane's own cost each load a loop over the lanes: 10 to 15% of the fp32
    // products.)
    __device__ __forceinline__ GroupTile within(int c, int t) const {
        const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(incl > t)) - 1);
        const int rows = __builtin_amdgcn_readlane(count, l);
        const int skip = (t - (__builtin_amdgcn_readlane(incl, l) - tiles_in<BM>(rows))) * BM;
        // Offsets that are not in order can make the sum pass 32 bits.
        if (skip < 0 || skip >= rows) return {0, 0, 1};
        return {__builtin_amdgcn_readfirstlane(c + l),
                __builtin_amdgcn_readfirstlane(__builtin_amdgcn_readlane(first, l) + skip),
                __builtin_amdgcn_readfirstlane(rows - skip)};
    }
};

// Group number r (below E), or number r when of each 64 groups those of at
// least four times `mean` rows come first, then those of at least twice and once
// that and then the others: where the groups' work is as uneven as they are, the
// long ones should not be the last to start.
struct OneGroup {
    int e, first, count;
};
__device__ __forceinline__ OneGroup group_at(const Groups &g, int r, bool by_size, int mean) {
    int first, count;
    if (!by_size) {
        group_rows(g, r, first, count);
        return {r, __builtin_amdgcn_readfirstlane(first), __builtin_amdgcn_readfirstlane(count)};
    }
    const int c = r & ~63, lane = threadIdx.x & 63;
    group_rows(g, c + lane, first, count);
    uint64_t among = __ballot(c + lane < g.E);
    r -= c;
#pragma unroll
    for (int shift = 2; shift >= 0; --shift) {
        const uint64_t large = among & __ballot(count >> shift >= mean);
        const int n = __popcll(large);
        among = r < n ? large : among & ~large;
        r -= r < n ? 0 : n;
    }
    const int before = __builtin_amdgcn_mbcnt_hi((unsigned)(among >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)among, 0));
    const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)(among & __ballot(before == r))) - 1);
    return {c + l, __builtin_amdgcn_readlane(first, l), __builtin_amdgcn_readlane(count, l)};
}

// The run of J entries behind the one at j0, of k entries; k behind the last one (j0 +
// J may lie past 2^31).
template <int J>
__host__ __device__ __forceinline__ int next_run(int j0, int k) { return k - j0 > J ? j0 + J : k; }

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
