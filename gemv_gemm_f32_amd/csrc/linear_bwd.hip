// linear_bwd.hip -- gradients of the fp32 dense layer Y = act(Z) + R,
// Z = X.op(W) + b:
//
//   dZ = dY * act'(Z)           (element by element)
//   dX = dZ . op(W)^T,  dW = X^T . dZ  (or its transpose),  db = sum_rows dZ
//
// One pass over dY and Z makes dZ (in the workspace, where the activation is
// not the identity; else dZ is dY itself) and, while the values are in
// registers, the column sums of each chunk of rows; the chunks' sums are then
// added in order by a second, small kernel.  The two products are those of
// gemm_f32_tile.hpp.
//
// The element pass is bound by memory: it reads dY and Z and writes dZ.  A
// workgroup takes 64 columns by one chunk of rows, 16 lanes of 4 columns by
// 16 rows at a time, so a row's part is 256 contiguous bytes.
#include <hip/hip_runtime.h>

#include "activation.hpp"
#include "kernels.hpp"

namespace gg {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef v4f v4f_any __attribute__((aligned(4)));   // rows may start at any float

constexpr int COLS = 64;             // columns per workgroup
constexpr int LANES = COLS / 4;      // threads along a row
constexpr int ROWS = 256 / LANES;    // rows at a time

__global__ __launch_bounds__(256) void dz_kernel(int act, int M, int N, int chunk,
                                                 const float *dY, int64_t lddy, const float *Z,
                                                 int64_t ldz, float *dZ, int64_t lddz,
                                                 float *partial) {
    __shared__ v4f red[256];
    const int tx = threadIdx.x % LANES, ty = threadIdx.x / LANES;
    const RowRange rows = dz_rows(M, chunk, blockIdx.y);
    for (int64_t c0 = (int64_t)blockIdx.x * COLS; c0 < N; c0 += (int64_t)gridDim.x * COLS) {
        const int64_t col = c0 + 4 * tx;
        const int live = (int)min(max(N - col, (int64_t)0), (int64_t)4);   // columns of this thread that exist
        v4f sum = {0.f, 0.f, 0.f, 0.f};
        with_act(act, [&](auto a) {
            constexpr int ACT = decltype(a)::value;
            for (int64_t r = rows.first + ty; r < rows.end; r += ROWS) {
                const float *pd = dY + r * lddy + col;
                const float *pz = Z + r * ldz + col;
                float *po = dZ + r * lddz + col;
                v4f d = {0.f, 0.f, 0.f, 0.f}, z = d;
                if (live == 4) {
                    d = *reinterpret_cast<const v4f_any *>(pd);
                    if (ACT != GG_ACT_NONE) z = *reinterpret_cast<const v4f_any *>(pz);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (c >= live) continue;
                        d[c] = pd[c];
                        if (ACT != GG_ACT_NONE) z[c] = pz[c];
                    }
                }
                if constexpr (ACT != GG_ACT_NONE) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) d[c] *= act_slope<ACT>(z[c]);
                    if (live == 4) {
                        *reinterpret_cast<v4f_any *>(po) = d;
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (c < live) po[c] = d[c];
                    }
                }
                sum += d;
            }
        });
        if (partial == nullptr) continue;             // uniform
        red[threadIdx.x] = sum;
        __syncthreads();
        if (ty == 0) {
#pragma unroll
            for (int y = 1; y < ROWS; ++y) sum += red[y * LANES + tx];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c < live) partial[(int64_t)blockIdx.y * N + col + c] = sum[c];
        }
        __syncthreads();
    }
}

// out[c] = (accumulate ? out[c] : 0) + sum over i of partial[i][c]: 16
// interleaved runs of rows per column, each added in order with 8 loads in
// flight, then the runs in order.
constexpr int RUNS = 16, INFLIGHT = 8;

__global__ __launch_bounds__(64 * RUNS) void column_sum_kernel(int n, int N, const float *partial,
                                                               int accumulate, float *out) {
    __shared__ float red[RUNS][64];
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < N; c0 += (int64_t)gridDim.x * 64) {
        const int64_t col = c0 + tx;
        float sum = 0.f;
        if (col < N) {
            const float *p = partial + col;
            for (int i = ty; i < n; i += RUNS * INFLIGHT) {
                float v[INFLIGHT];
#pragma unroll
                for (int u = 0; u < INFLIGHT; ++u)
                    v[u] = i + RUNS * u < n ? p[(int64_t)(i + RUNS * u) * N] : 0.f;
#pragma unroll
                for (int u = 0; u < INFLIGHT; ++u) sum += v[u];
            }
        }
        red[ty][tx] = sum;
        __syncthreads();
        if (ty == 0 && col < N) {
#pragma unroll
            for (int y = 1; y < RUNS; ++y) sum += red[y][tx];
            out[col] = accumulate ? out[col] + sum : sum;
        }
        __syncthreads();
    }
}

inline unsigned blocks(int64_t n, int64_t per, int64_t most) {
    const int64_t b = (n + per - 1) / per;
    return (unsigned)(b < most ? b : most);
}

}  // namespace

hipError_t launch_column_sum(int n, int N, const float *partial, bool accumulate, float *out,
                             hipStream_t s) {
    return launch(column_sum_kernel, dim3(blocks(N, 64, 1 << 20)), dim3(64 * RUNS), s, n, N, partial,
                  accumulate ? 1 : 0, out);
}

hipError_t launch_linear_bwd(bool trans_w, int act, bool accumulate, int M, int N, int K,
                             const float *dY, int64_t lddy, const float *Z, int64_t ldz,
                             const float *X, int64_t ldx, const float *W, int64_t ldw, float *dX,
                             int64_t lddx, float *dW, int64_t lddw, float *db, float *ws,
                             int num_cus, hipStream_t s) {
    hipError_t e = hipSuccess;
    const float *dZ = dY;
    int64_t lddz = lddy;
    if (M > 0 && N > 0 && (act != GG_ACT_NONE || db != nullptr)) {
        float *out = ws, *partial = ws;
        if (act != GG_ACT_NONE) {
            lddz = dz_stride(N);
            partial = ws + (int64_t)M * lddz;
            dZ = out;
        }
        const int chunk = dz_chunk(M), chunks = dz_chunks(M);
        const dim3 grid(blocks(N, COLS, 1 << 17), chunks);
        e = launch(dz_kernel, grid, dim3(256), s, act, M, N, chunk,
                   dY, lddy, Z, ldz, out, lddz, db ? partial : nullptr);
        if (e != hipSuccess) return e;
        if (db) e = launch_column_sum(chunks, N, partial, accumulate, db, s);
    } else if (db && N > 0) {
        e = launch_column_sum(0, N, nullptr, accumulate, db, s);
    }
    if (e != hipSuccess) return e;
    if (dX && M > 0 && K > 0) {
        e = launch_gemm(true, !trans_w, M, K, N, 1.f, dZ, lddz, W, ldw, 0.f, dX, lddx, num_cus, s);
        if (e != hipSuccess) return e;
    }
    if (dW && N > 0 && K > 0) {
        const float beta = accumulate ? 1.f : 0.f;
        e = trans_w ? launch_gemm(false, false, N, K, M, 1.f, dZ, lddz, X, ldx, beta, dW, lddw, num_cus, s)
                    : launch_gemm(false, false, K, N, M, 1.f, X, ldx, dZ, lddz, beta, dW, lddw, num_cus, s);
    }
    return e;
}

}  // namespace gg
