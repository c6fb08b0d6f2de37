// kernels.hpp -- launch functions exported by the kernel translation units to
// the C entry points (api.hip).  Internal to libgemvgemm.so.
//
// Each launcher assumes its arguments were validated by the caller: sizes in
// [0, 2^31), non-null aligned pointers for non-empty operands, leading
// dimensions at least the row width, output not aliasing an input.  It only
// picks a compile-time specialisation and a grid, and launches.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <tuple>
#include <utility>

namespace gg {

// Launches kernel<<<grid, block, 0, s>>>(args...) and returns that launch's
// own status from hipLaunchKernel, so an error left pending by an earlier,
// unrelated HIP call is neither reported as ours nor cleared.  The arguments
// are converted to the kernel's parameter types first.
template <typename... P, size_t... I>
hipError_t launch_args(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t s,
                       std::tuple<P...> &args, std::index_sequence<I...>) {
    void *ptrs[sizeof...(P) + 1] = {static_cast<void *>(&std::get<I>(args))..., nullptr};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), grid, block, ptrs, 0, s);
}

template <typename... P, typename... A>
hipError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t s, A &&...a) {
    static_assert(sizeof...(P) == sizeof...(A), "kernel argument count");
    std::tuple<P...> args(std::forward<A>(a)...);
    return launch_args(kernel, grid, block, s, args, std::index_sequence_for<P...>{});
}

// C = alpha * op(A).op(B) + beta * C (C not read when beta == 0).
// ax: A stored M x K (else K x M, i.e. op(A) = A^T); bx: B stored N x K
// (op(B) = B^T, else K x N).  num_cus is the device's compute-unit count (it
// picks the tile shape).  K = 0 writes beta * C (zeros for beta = 0).
hipError_t launch_gemm(bool ax, bool bx, int M, int N, int K, float alpha, const float *A,
                       int64_t lda, const float *B, int64_t ldb, float beta, float *C,
                       int64_t ldc, int num_cus, hipStream_t stream);

// y_b = W_b.x_b for b < count, fp32; the pointer arrays are host arrays of
// device pointers.  More than F32_MAX_BATCH products take several launches
// in order; if one of them is rejected the earlier ones stay queued.
constexpr int F32_MAX_BATCH = 64;
hipError_t launch_gemv_f32(int count, int M, int K, const float *const *W, int64_t ldw,
                           const float *const *x, float *const *y, hipStream_t stream);

// y_b = W_b.x_b for b < count, W_b as 2-bit (q2) or 4-bit (q4) codes with
// one binary16 scale per 64 columns; the pointer arrays are host arrays of
// device pointers.  More than PACKED_MAX_BATCH products take several
// launches in order; if one of them is rejected the earlier ones stay
// queued.
constexpr int PACKED_MAX_BATCH = 64;
// ws: NULL, or a workspace of gemv_q2_workspace_floats(count, M, K) floats
// that batches of long rows use for partial sums (rows cut into slices);
// without it they take a kernel that needs none.
hipError_t launch_gemv_q2(int count, int M, int K, const uint8_t *const *Q, int64_t ldq,
                          const uint16_t *const *S, int64_t lds, const float *const *x,
                          float *const *y, float *ws, hipStream_t stream);
// Batches of 2-bit products whose rows are long cut them into slices of
// SLICE_K columns, each written to the workspace as partial row sums, when
// a workspace is given: rows of 4 to SLICED_MAX slices, at least
// SLICED_MIN_COUNT products (at 1,536 x 12,288, µs per product sliced
// against whole: 4 products 2.46 / 2.39, 8: 1.67 / 1.77, 16: 1.32 / 1.49,
// 40: 1.08 / 1.33).  Slices of
// SLICE_K/512 waves each, as the integer-dot kernel is tuned for.
constexpr int SLICE_K = 1536;
constexpr int SLICED_MIN_COUNT = 8;
constexpr int SLICED_MAX = 1024;

// Slices per row for a batch of this shape, 0 where it is not cut.
inline int64_t sliced_count(int64_t count, int64_t M, int64_t K) {
    if (count < SLICED_MIN_COUNT || M < 1 || K % SLICE_K != 0) return 0;
    const int64_t n = K / SLICE_K;
    return n >= 4 && n <= SLICED_MAX ? n : 0;
}

// The fixed per-device scratch buffer of the allocation-free entry point
// (noalloc.hip): its size, and its device address on the current device
// (found on first use there), or NULL if it cannot be had.
constexpr int64_t SCRATCH_BYTES = int64_t(4) << 20;
float *device_scratch();

// Floats of workspace a 2-bit batch of this shape uses, 0 if none: one
// launch's partial sums (the next launch of a batch over PACKED_MAX_BATCH
// products reuses them).
inline int64_t gemv_q2_workspace_floats(int64_t count, int64_t M, int64_t K) {
    const int64_t n = sliced_count(count, M, K);
    return n ? (count < PACKED_MAX_BATCH ? count : PACKED_MAX_BATCH) * n * M : 0;
}
hipError_t launch_gemv_q4(int count, int M, int K, const uint8_t *const *Q, int64_t ldq,
                          const uint16_t *const *S, int64_t lds, const float *const *x,
                          float *const *y, hipStream_t stream);

// Y = act(X.op(W) + bias) + R, fp32; op(W) = W^T with W stored N x K when
// trans_w, else W stored K x N.  Z (may be NULL) receives the pre-activation.
hipError_t launch_linear(bool trans_w, int act, int M, int N, int K, const float *X, int64_t ldx,
                         const float *W, int64_t ldw, const float *bias, const float *R,
                         int64_t ldr, float *Z, int64_t ldz, float *Y, int64_t ldy, int num_cus,
                         hipStream_t stream);

// Its gradients; each of dX, dW and db may be NULL.  ws holds
// linear_bwd_workspace_floats floats.
hipError_t launch_linear_bwd(bool trans_w, int act, bool accumulate, int M, int N, int K,
                             const float *dY, int64_t lddy, const float *Z, int64_t ldz,
                             const float *X, int64_t ldx, const float *W, int64_t ldw, float *dX,
                             int64_t lddx, float *dW, int64_t lddw, float *db, float *ws,
                             int num_cus, hipStream_t stream);
// Row stride of dZ in the workspace, and the rows of one chunk of column
// sums: at most 64 chunks, of a multiple of 16 rows.
inline int64_t dz_stride(int64_t N) { return (N + 3) & ~int64_t(3); }
inline int dz_chunk(int M) { return (int)((((int64_t)M + 63) / 64 + 15) & ~int64_t(15)); }
inline int dz_chunks(int M) { return (int)(((int64_t)M + dz_chunk(M) - 1) / dz_chunk(M)); }
// Rows [first, end) of chunk i.  64 bits: chunks of 2^25 rows end at 2^31.
struct RowRange {
    int64_t first, end;
};
__host__ __device__ inline RowRange dz_rows(int M, int chunk, int64_t i) {
    const int64_t first = i * chunk, end = first + chunk;
    return {first, end < M ? end : M};
}
inline unsigned __int128 linear_bwd_workspace_floats(bool identity, int64_t M, int64_t N) {
    return (identity ? 0 : (unsigned __int128)M * dz_stride(N)) + (unsigned __int128)64 * N;
}

// out[c] = (accumulate ? out[c] : 0) + the n partial sums of column c < N.
hipError_t launch_column_sum(int n, int N, const float *partial, bool accumulate, float *out,
                             hipStream_t stream);

// S = X + R (R may be NULL); y = S * rstd * gamma with rstd = 1 / sqrt(mean
// of S^2 over the row + eps), as fp32 in Y or as e4m3 bytes in Q with e8m0
// bytes in E (mx8.hpp).  S, gamma and rstd may be NULL; S may be X or R.
struct RmsNorm {
    int M, K;
    const float *X, *R, *gamma;
    float *S, *Y, *rstd;
    uint8_t *Q, *E;
    int64_t ldx, ldr, lds, ldy, ldq, lde;
    float eps;
};
hipError_t launch_rmsnorm(const RmsNorm &a, hipStream_t stream);

// dX = rstd * (gamma * dY - xhat * mean(gamma * dY * xhat)) + dS with xhat =
// S * rstd, and dgamma = sum over rows of dY * xhat.  gamma, dS, dX and
// dgamma may be NULL; dX may be dS.  ws holds rmsnorm_bwd_workspace_floats
// floats where dgamma is wanted.
struct RmsNormBwd {
    int M, K;
    const float *dY, *S, *gamma, *rstd, *dS;
    float *dX, *dgamma, *ws;
    int64_t lddy, lds, ldds, lddx;
    bool accumulate;
};
hipError_t launch_rmsnorm_bwd(const RmsNormBwd &a, hipStream_t stream);
// Partial sums of dgamma: one row of K per workgroup.
constexpr int RMSNORM_BWD_GROUPS = 512;
inline int64_t rmsnorm_bwd_workspace_floats(int64_t M, int64_t K) {
    return (M < RMSNORM_BWD_GROUPS ? M : RMSNORM_BWD_GROUPS) * K;
}

// Y = act(X8.W^T + bias) + R with X8 in 8 bits (mx8.hpp) and W (N x K) as
// 2-bit or 4-bit codes with one binary16 scale per 64 columns; to fp32 Y, or
// to 8 bits (Y8, YE), or both.
struct PackedLinear {
    int act, M, N, K;
    const uint8_t *X, *XE, *Q;
    const uint16_t *S;
    const float *bias, *R;
    float *Y;
    uint8_t *Y8, *YE;
    int64_t ldx, ldxe, ldq, lds, ldr, ldy, ldy8, ldye;
};
hipError_t launch_packed_linear(int bits, const PackedLinear &a, int num_cus, hipStream_t stream);

}  // namespace gg
