// linear_mx8.hip -- the packed layers on rows in 8 bits: launches of the tiles
// of linear_mx8_tile.hpp and the choice among them.
#include <hip/hip_runtime.h>

#include "kernels.hpp"
#include "linear_mx8_tile.hpp"

namespace gg {
namespace {

// row m of Y is fed by row m of X
struct SameRow {
    __device__ __forceinline__ int64_t operator()(int64_t m) const { return m; }
};

// Workgroup -> tile: runs of neighbouring tiles per XCD, rows first.
__device__ __forceinline__ int tile_number() {
    int tb = blockIdx.x;
    if ((gridDim.x & 7) == 0) tb = (tb & 7) * (gridDim.x >> 3) + (tb >> 3);
    return tb;
}

template <int BITS, int NH, int KW>
__global__ __launch_bounds__(64 * NH * KW) void packed_rows_kernel(PackedLinear a) {
    packed_rows<BITS, NH, KW>(a, (int64_t)blockIdx.x * 16 * NH, SameRow{});
}

template <int KW, int BITS, int MW>
__global__ __launch_bounds__(64 * KW, MW) void packed_block_kernel(PackedLinear a, int tiles_m) {
    const int tb = tile_number();
    packed_block<KW, BITS>(a, (int64_t)(tb % tiles_m) * 32, (int64_t)(tb / tiles_m) * 32, SameRow{});
}

template <int BM, int NW, int BITS, int MW = 2>
__global__ __launch_bounds__(64 * NW, MW) void packed_wide_kernel(PackedLinear a, int tiles_m) {
    __shared__ __attribute__((aligned(16))) char smem[wide_bytes<BM, NW>()];
    const int tb = tile_number();
    packed_wide<BM, NW, BITS>(a, (int64_t)(tb % tiles_m) * BM, (int64_t)(tb / tiles_m) * 32 * NW, SameRow{},
                              smem);
}

// A launch has fewer than 2^32 threads: with `threads` for each bm x bn tile,
// larger outputs are cut into rectangles (from multiples of 256, so that
// blocks of 32 columns stay whole), and one(rectangle) launches each.
template <class One>
hipError_t in_parts(const PackedLinear &a, int bm, int bn, int threads, One one) {
    int64_t rows = a.M, cols = a.N;
    while (((rows + bm - 1) / bm) * ((cols + bn - 1) / bn) * threads > UINT32_MAX) {
        int64_t &longer = rows >= cols ? rows : cols;
        longer = ((longer + 1) / 2 + 255) & ~int64_t(255);
    }
    for (int64_t m = 0; m < a.M; m += rows)
        for (int64_t n = 0; n < a.N; n += cols) {
            PackedLinear p = a;
            p.M = (int)(a.M - m < rows ? a.M - m : rows);
            p.N = (int)(a.N - n < cols ? a.N - n : cols);
            p.X += m * a.ldx;
            p.XE += m * a.ldxe;
            p.Q += n * a.ldq;
            p.S += n * a.lds;
            if (a.bias) p.bias += n;
            if (a.R) p.R += m * a.ldr + n;
            if (a.Y) p.Y += m * a.ldy + n;
            if (a.Y8) {
                p.Y8 += m * a.ldy8 + n;
                p.YE += m * a.ldye + n / 32;
            }
            const hipError_t e = one(p);
            if (e != hipSuccess) return e;
        }
    return hipSuccess;
}

template <int BITS, int NH, int KW>
hipError_t launch_rows(const PackedLinear &a, hipStream_t s) {
    constexpr int COLS = 16 * NH, THREADS = 64 * NH * KW;
    return in_parts(a, 16, COLS, THREADS, [s](const PackedLinear &p) {
        const int64_t nb = ((int64_t)p.N + COLS - 1) / COLS;
        return launch(packed_rows_kernel<BITS, NH, KW>, dim3((unsigned)nb), dim3(THREADS), s, p);
    });
}

template <int KW, int BITS, int MW>
hipError_t launch_block(const PackedLinear &a, hipStream_t s) {
    const int64_t tm = ((int64_t)a.M + 31) / 32, tn = ((int64_t)a.N + 31) / 32;
    return launch(packed_block_kernel<KW, BITS, MW>, dim3((unsigned)(tm * tn)), dim3(64 * KW), s, a, (int)tm);
}

template <int BM, int NW, int BITS, int MW = 2>
hipError_t launch_wide(const PackedLinear &a, hipStream_t s) {
    return in_parts(a, BM, 32 * NW, 64 * NW, [s](const PackedLinear &p) {
        const int64_t tm = ((int64_t)p.M + BM - 1) / BM, tn = ((int64_t)p.N + 32 * NW - 1) / (32 * NW);
        return launch(packed_wide_kernel<BM, NW, BITS, MW>, dim3((unsigned)(tm * tn)), dim3(64 * NW), s, p,
                      (int)tm);
    });
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
    // More rows (2 bits / 4 bits, us):
    //  - 32 x 32 cells with a wave per run of k, up to 6 workgroups per CU: 256 x
    //    4096 x 4096 23.7 / 26.4 against 27.0 / 36.5 in the best shape of the other
    //    kernel, 384 x 4096 x 4096 32.5 / 35.7 against 33.7 / 37.3, but 512 x 4096 x
    //    4096 41.0 / 45.4 against 36.3 / 39.7.  Eight runs instead of four where
    //    there is at most one workgroup per CU and k is long: 64 x 1536 x 12288
    //    17.2 / 19.1 against 18.7 / 21.1; 128 x 2304 x 768 7.6 / 8.1 against 5.7 / 6.2.
    //  - else a wave per 32 columns: 128 x 256 tiles where a round of them leaves
    //    at most a fifth of the CUs idle (2048 x 4096 x 4096 77 / 82 against 99 /
    //    108 in 64 x 128); 64 x 256 where they fit one per CU and 64 x 128 do not
    //    (1024 x 4096 x 4096 48.4 / 53.0 against 52.0 / 56.6; 512 x 4096 x 4096 42.6 /
    //    47.6 against 36.5 / 39.7); else 64 x 128 (500 x 12288 x 1536 32.2 / 35.0
    //    against 38.1 / 41.8 in 64 x 256).
    const int64_t cells = count(32, 32), big = count(128, 256);
    if (cells <= 6 * cus)
        return cells <= cus && a.K >= 4096 ? launch_block<8, BITS, 2>(a, s) : launch_block<4, BITS, 3>(a, s);
    if (big >= cus && 4 * ((big + cus - 1) / cus * cus) <= 5 * big)
        return launch_wide<128, 8, BITS, 2>(a, s);
    if (count(64, 128) > cus && count(64, 256) <= cus) return launch_wide<64, 8, BITS, 2>(a, s);
    return launch_wide<64, 4, BITS, 3>(a, s);
}

}  // namespace

hipError_t launch_packed_linear(int bits, const PackedLinear &a, int num_cus, hipStream_t s) {
    return bits == 2 ? launch_bits<2>(a, num_cus, s) : launch_bits<4>(a, num_cus, s);
}

}  // namespace gg
