// api_experts.hip -- the C entry points of the layer with experts and of the
// norms around a block (declared in gemvgemm.h): argument checks as in api.hip,
// before any HIP call and before anything is written, then the launchers of
// kernels.hpp.  Nothing here allocates, so no exception can arise.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/gemvgemm.h"
#include "checks.hpp"
#include "kernels.hpp"

using namespace gg;

namespace {

hipStream_t hip_stream(gg_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

// The grouped kernels count tiles of 32 rows by 32 columns in 32 bits and
// offsets within 64 rows of an fp32 operand in 31.
constexpr int64_t kMaxGroupedLd = int64_t(1) << 22;
bool bad_experts(int64_t E) { return E < 0 || E > MAX_EXPERTS; }
bool bad_tiles(int64_t M, int64_t N, int64_t E) {
    return (unsigned __int128)(M / 32 + E) * (uint64_t)((N + 31) / 32) > (uint64_t)kMaxDim;
}
// Rows that are picked have to lie within 2 GiB: T rows of K elements.
bool bad_pick(int64_t T, int64_t K, int64_t ld, int64_t elem) {
    return T < 1 || extent_bytes(T, K, ld, elem) >= (uint64_t)1 << 31;
}

int packed_grouped(int bits, int act, int64_t M, int64_t N, int64_t K, int64_t E, int64_t T,
                   const uint8_t *X8, int64_t ldx, const uint8_t *XE, int64_t ldxe, const int32_t *rows,
                   const int32_t *offsets, const uint8_t *Q, int64_t ldq, int64_t strideq,
                   const uint16_t *S, int64_t lds, int64_t strides, const float *bias, int64_t ldb,
                   float *Y, int64_t ldy, uint8_t *Y8, int64_t ldy8, uint8_t *YE, int64_t ldye,
                   gg_stream_t stream) {
    if (bad_act(act) || bad_size(M) || bad_size(N) || bad_size(K) || bad_experts(E) || (rows && bad_size(T)))
        return GG_ERR_INVALID_ARG;
    if (M == 0 || N == 0 || E == 0) return GG_OK;
    if ((Y8 == nullptr) != (YE == nullptr) || (Y == nullptr && Y8 == nullptr) || (rows && T < 1) ||
        bad_tiles(M, N, E))
        return GG_ERR_INVALID_ARG;
    const int64_t per_byte = 8 / bits, from = rows ? T : M;
    Operands o;
    o.in(X8, from, K, ldx, 1).in(XE, from, (K + 31) / 32, ldxe, 1).in(offsets, 1, E + 1, E + 1);
    if (rows) o.in(rows, 1, M, M);
    o.in_each(Q, E, strideq, N, (K + per_byte - 1) / per_byte, ldq, 1).in_each(S, E, strides, N, (K + 63) / 64, lds, 2);
    if (bias) o.in(bias, E, N, ldb);
    if (Y) o.out(Y, M, N, ldy);
    if (Y8) o.out(Y8, M, N, ldy8, 1).out(YE, M, (N + 31) / 32, ldye, 1);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const PackedGrouped a{{act, (int)M, (int)N, (int)K, X8, XE, Q, S, bias, nullptr, Y, Y8, YE, ldx, ldxe, ldq, lds, 0,
                           Y ? ldy : 0, Y8 ? ldy8 : 0, YE ? ldye : 0},
                          rows, offsets, (int)E, (int)T, strideq, strides, bias ? ldb : 0};
    return launch_status(launch_packed_grouped(bits, a, cus, hip_stream(stream)));
}

// The norms with their output in fp32 (Q null) or in 8 bits (Y null).
int block_norm(int64_t M, int64_t K, const float *U, int64_t ldu, const float *X, int64_t ldx,
               const float *gamma_u, const float *gate, int64_t ldgate, float alpha, const float *gamma_s,
               float eps, float *S, int64_t lds, float *Y, int64_t ldy, uint8_t *Q, int64_t ldq, uint8_t *E,
               int64_t lde, bool mx8, float *rstd_u, float *rstd_s, gg_stream_t stream) {
    if (bad_size(M) || bad_size(K) || !(eps >= 0.f) || std::isinf(eps) || !std::isfinite(alpha))
        return GG_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return GG_OK;
    const bool own = gate && ldgate != 0;
    Operands o;
    o.in(U, M, K, ldu).replaced(X, M, K, ldx);
    if (gamma_u) o.in(gamma_u, 1, K, K);
    if (gate) o.in(gate, own ? M : 1, K, own ? ldgate : K);
    if (gamma_s) o.in(gamma_s, 1, K, K);
    o.onto(S, M, K, lds);
    if (mx8) o.out(Q, M, K, ldq, 1).out(E, M, (K + 31) / 32, lde, 1);
    else o.out(Y, M, K, ldy);
    if (rstd_u) o.out(rstd_u, 1, M, M);
    if (rstd_s) o.out(rstd_s, 1, M, M);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const BlockNorm a{(int)M, (int)K, U, X, gamma_u, gate, gamma_s, S, Y, rstd_u, rstd_s, Q, E,
                      ldu, ldx, own ? ldgate : 0, lds, ldy, ldq, lde, alpha, eps};
    return launch_status(launch_block_norm(a, hip_stream(stream)));
}

}  // namespace

extern "C" {

int expert_groups(int64_t T, int64_t k, int64_t E, const int32_t *ids, int64_t ldi, int32_t *offsets,
                  int32_t *rows, int32_t *pos, int64_t ldp, gg_stream_t stream) {
    if (bad_size(T) || bad_size(k) || bad_experts(E) || bad_size(T * k)) return GG_ERR_INVALID_ARG;
    Operands o;
    o.in(ids, T, k, ldi).out(offsets, 1, E + 1, E + 1);
    if (T * k > 0) o.out(rows, 1, T * k, T * k);
    o.out(pos, T, k, ldp);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const ExpertGroups a{(int)T, (int)k, (int)E, ids, offsets, rows, pos, ldi, ldp};
    return launch_status(launch_expert_groups(a, hip_stream(stream)));
}

int expert_combine(int64_t T, int64_t k, int64_t M, int64_t K, const float *Y, int64_t ldy,
                   const int32_t *pos, int64_t ldp, const float *weights, int64_t ldw, const float *R,
                   int64_t ldr, float *out, int64_t ldo, gg_stream_t stream) {
    if (bad_size(T) || bad_size(k) || bad_size(M) || bad_size(K)) return GG_ERR_INVALID_ARG;
    if (T == 0 || K == 0) return GG_OK;
    Operands o;
    o.in(Y, M, K, ldy).in(pos, T, k, ldp);
    if (weights) o.in(weights, T, k, ldw);
    if (R) o.replaced(R, T, K, ldr);
    o.onto(out, T, K, ldo);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const ExpertCombine a{(int)T, (int)k, (int)M, (int)K, Y, weights, R, pos, out, ldy,
                          weights ? ldw : 0, ldp, R ? ldr : 0, ldo};
    return launch_status(launch_expert_combine(a, hip_stream(stream)));
}

int expert_combine_bwd(int64_t T, int64_t k, int64_t M, int64_t K, const float *dO, int64_t lddo,
                       const float *Y, int64_t ldy, const int32_t *pos, int64_t ldp, const float *weights,
                       int64_t ldw, float *dY, int64_t lddy, float *dw, int64_t lddw, gg_stream_t stream) {
    if (bad_size(T) || bad_size(k) || bad_size(M) || bad_size(K)) return GG_ERR_INVALID_ARG;
    const bool gy = dY != nullptr && M > 0 && K > 0, gw = dw != nullptr;
    if (T == 0 || k == 0 || (!gy && !gw)) return GG_OK;
    Operands o;
    o.in(dO, T, K, lddo).in(pos, T, k, ldp);
    if (weights) o.in(weights, T, k, ldw);
    if (gy) o.out(dY, M, K, lddy);
    if (gw) o.in(Y, M, K, ldy).out(dw, T, k, lddw);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const ExpertCombineBwd a{(int)T, (int)k, (int)M, (int)K, dO, Y, weights, pos, gy ? dY : nullptr,
                             gw ? dw : nullptr, lddo, gw ? ldy : 0, weights ? ldw : 0, ldp, gy ? lddy : 0,
                             gw ? lddw : 0};
    return launch_status(launch_expert_combine_bwd(a, hip_stream(stream)));
}

int linear_f32_grouped(int trans_w, int act, int64_t M, int64_t N, int64_t K, int64_t E, int64_t T,
                       const float *X, int64_t ldx, const int32_t *rows, const int32_t *offsets,
                       const float *W, int64_t ldw, int64_t stridew, const float *bias, int64_t ldb,
                       float *Z, int64_t ldz, float *Y, int64_t ldy, gg_stream_t stream) {
    if ((trans_w != 0 && trans_w != 1) || bad_act(act) || bad_size(M) || bad_size(N) || bad_size(K) ||
        bad_experts(E) || (rows && bad_size(T)))
        return GG_ERR_INVALID_ARG;
    if (M == 0 || N == 0 || E == 0) return GG_OK;
    if (bad_tiles(M, N, E) || (K > 0 && (ldx > kMaxGroupedLd || ldw > kMaxGroupedLd)) ||
        (rows && bad_pick(T, K, ldx, 4)))
        return GG_ERR_INVALID_ARG;
    Operands o;
    o.in(X, rows ? T : M, K, ldx).in(offsets, 1, E + 1, E + 1);
    if (rows) o.in(rows, 1, M, M);
    o.in_each(W, E, stridew, trans_w ? N : K, trans_w ? K : N, ldw);
    if (bias) o.in(bias, E, N, ldb);
    if (Z) o.out(Z, M, N, ldz);
    o.out(Y, M, N, ldy);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const LinearGrouped a{trans_w == 1, act, (int)M, (int)N, (int)K, (int)E, (int)T, X, W, bias, rows, offsets, Z, Y,
                          ldx, ldw, stridew, bias ? ldb : 0, Z ? ldz : 0, ldy};
    return launch_status(launch_linear_grouped(a, cus, hip_stream(stream)));
}

int64_t linear_f32_grouped_bwd_ws_size(int act, int64_t M, int64_t N, int64_t E) {
    if (bad_act(act) || bad_size(M) || bad_size(N) || bad_experts(E)) return GG_ERR_INVALID_ARG;
    if (M == 0 || N == 0 || E == 0) return 0;
    const unsigned __int128 bytes = 4 * linear_grouped_bwd_workspace_floats(act == GG_ACT_NONE, M, N, E);
    return bytes > ((unsigned __int128)1 << 62) ? GG_ERR_INVALID_ARG : (int64_t)bytes;
}

int linear_f32_grouped_bwd(int trans_w, int act, int accumulate, int64_t M, int64_t N, int64_t K, int64_t E,
                           int64_t T, const float *dY, int64_t lddy, const float *Z, int64_t ldz,
                           const float *X, int64_t ldx, const int32_t *rows, const int32_t *offsets,
                           const float *W, int64_t ldw, int64_t stridew, float *dX, int64_t lddx, float *dW,
                           int64_t lddw, int64_t stridedw, float *db, int64_t lddb, void *workspace,
                           int64_t workspace_bytes, gg_stream_t stream) {
    if ((trans_w != 0 && trans_w != 1) || (accumulate != 0 && accumulate != 1) || bad_act(act) || bad_size(M) ||
        bad_size(N) || bad_size(K) || bad_experts(E) || (rows && bad_size(T)))
        return GG_ERR_INVALID_ARG;
    const int64_t w_rows = trans_w ? N : K, w_cols = trans_w ? K : N;
    // operands of the outputs that are wanted and not empty
    const bool gx = dX != nullptr && M > 0 && K > 0 && E > 0;
    const bool gw = dW != nullptr && N > 0 && K > 0 && E > 0;
    const bool gb = db != nullptr && N > 0 && E > 0;
    if (!gx && !gw && !gb) return GG_OK;
    const bool read_x = gw && M > 0, read_w = gx && N > 0;
    if ((gx && bad_tiles(M, K, E)) || (gw && bad_tiles(E * ((w_rows + 31) / 32) * 32, w_cols, 0)) ||
        bad_tiles(M, N, E) || (read_w && ldw > kMaxGroupedLd) || (read_x && ldx > kMaxGroupedLd) ||
        ((gx || gw) && M > 0 && N > 0 && (lddy > kMaxGroupedLd || N > kMaxGroupedLd)) ||
        (read_x && rows && bad_pick(T, K, ldx, 4)))
        return GG_ERR_INVALID_ARG;
    Operands o;
    o.in(dY, M, N, lddy).in(offsets, 1, E + 1, E + 1);
    if (act != GG_ACT_NONE) o.in(Z, M, N, ldz);
    if (read_w) o.in_each(W, E, stridew, w_rows, w_cols, ldw);
    if (gx) o.out(dX, M, K, lddx);
    if (read_x) o.in(X, rows ? T : M, K, ldx);
    if (read_x && rows) o.in(rows, 1, M, M);
    if (gw) o.out_each(dW, E, stridedw, w_rows, w_cols, lddw);
    if (gb) o.out(db, E, N, lddb);
    o.workspace(workspace, workspace_bytes,
                M && N ? 4 * linear_grouped_bwd_workspace_floats(act == GG_ACT_NONE, M, N, E) : 0);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const LinearGroupedBwd a{trans_w == 1, accumulate == 1, act, (int)M, (int)N, (int)K, (int)E, (int)T, dY, Z, X, W,
                             rows, offsets, gx ? dX : nullptr, gw ? dW : nullptr, gb ? db : nullptr,
                             static_cast<float *>(workspace), lddy, act != GG_ACT_NONE ? ldz : 0, ldx, ldw, stridew,
                             lddx, lddw, stridedw, gb ? lddb : 0};
    return launch_status(launch_linear_grouped_bwd(a, cus, hip_stream(stream)));
}

int linear_q4_mx8_grouped(int act, int64_t M, int64_t N, int64_t K, int64_t E, int64_t T, const uint8_t *X8,
                          int64_t ldx, const uint8_t *XE, int64_t ldxe, const int32_t *rows,
                          const int32_t *offsets, const uint8_t *Q, int64_t ldq, int64_t strideq,
                          const uint16_t *S, int64_t lds, int64_t strides, const float *bias, int64_t ldb,
                          float *Y, int64_t ldy, uint8_t *Y8, int64_t ldy8, uint8_t *YE, int64_t ldye,
                          gg_stream_t stream) {
    return packed_grouped(4, act, M, N, K, E, T, X8, ldx, XE, ldxe, rows, offsets, Q, ldq, strideq, S, lds, strides,
                          bias, ldb, Y, ldy, Y8, ldy8, YE, ldye, stream);
}

int linear_q2_mx8_grouped(int act, int64_t M, int64_t N, int64_t K, int64_t E, int64_t T, const uint8_t *X8,
                          int64_t ldx, const uint8_t *XE, int64_t ldxe, const int32_t *rows,
                          const int32_t *offsets, const uint8_t *Q, int64_t ldq, int64_t strideq,
                          const uint16_t *S, int64_t lds, int64_t strides, const float *bias, int64_t ldb,
                          float *Y, int64_t ldy, uint8_t *Y8, int64_t ldy8, uint8_t *YE, int64_t ldye,
                          gg_stream_t stream) {
    return packed_grouped(2, act, M, N, K, E, T, X8, ldx, XE, ldxe, rows, offsets, Q, ldq, strideq, S, lds, strides,
                          bias, ldb, Y, ldy, Y8, ldy8, YE, ldye, stream);
}

int block_norm_f32(int64_t M, int64_t K, const float *U, int64_t ldu, const float *X, int64_t ldx,
                   const float *gamma_u, const float *gate, int64_t ldgate, float alpha, const float *gamma_s,
                   float eps, float *S, int64_t lds, float *Y, int64_t ldy, float *rstd_u, float *rstd_s,
                   gg_stream_t stream) {
    return block_norm(M, K, U, ldu, X, ldx, gamma_u, gate, ldgate, alpha, gamma_s, eps, S, lds, Y, ldy, nullptr, 0,
                      nullptr, 0, false, rstd_u, rstd_s, stream);
}

int block_norm_mx8(int64_t M, int64_t K, const float *U, int64_t ldu, const float *X, int64_t ldx,
                   const float *gamma_u, const float *gate, int64_t ldgate, float alpha, const float *gamma_s,
                   float eps, float *S, int64_t lds, uint8_t *Q, int64_t ldq, uint8_t *E, int64_t lde,
                   gg_stream_t stream) {
    return block_norm(M, K, U, ldu, X, ldx, gamma_u, gate, ldgate, alpha, gamma_s, eps, S, lds, nullptr, 0, Q, ldq, E,
                      lde, true, nullptr, nullptr, stream);
}

int64_t block_norm_f32_bwd_ws_size(int64_t M, int64_t K) {
    if (bad_size(M) || bad_size(K)) return GG_ERR_INVALID_ARG;
    return 4 * block_norm_bwd_workspace_floats(M, K);
}

int block_norm_f32_bwd(int accumulate, int64_t M, int64_t K, const float *dY, int64_t lddy, const float *U,
                       int64_t ldu, const float *S, int64_t lds, const float *gamma_u, const float *gate,
                       int64_t ldgate, float alpha, const float *gamma_s, const float *rstd_u,
                       const float *rstd_s, const float *dS, int64_t ldds, float *dU, int64_t lddu, float *dX,
                       int64_t lddx, float *dgamma_u, float *dgamma_s, float *dgate, int64_t lddgate,
                       void *workspace, int64_t workspace_bytes, gg_stream_t stream) {
    if ((accumulate != 0 && accumulate != 1) || bad_size(M) || bad_size(K) || !std::isfinite(alpha) ||
        (dgate && !gate))
        return GG_ERR_INVALID_ARG;
    const bool own = gate && ldgate != 0;
    const bool gu = dU != nullptr && M > 0, gx = dX != nullptr && M > 0, gg_own = dgate && own && M > 0;
    const bool sums = dgamma_u || dgamma_s || (dgate && !own);
    if (K == 0 || (!gu && !gx && !gg_own && !sums)) return GG_OK;
    Operands o;
    o.in(dY, M, K, lddy).in(U, M, K, ldu).in(S, M, K, lds);
    if (M > 0) o.in(rstd_u, 1, M, M).in(rstd_s, 1, M, M);
    if (gamma_u) o.in(gamma_u, 1, K, K);
    if (gamma_s) o.in(gamma_s, 1, K, K);
    if (gate) o.in(gate, own ? M : 1, K, own ? ldgate : K);
    if (dS) o.replaced(dS, M, K, ldds);
    if (gu) o.out(dU, M, K, lddu);
    if (gx) o.onto(dX, M, K, lddx);
    if (dgamma_u) o.out(dgamma_u, 1, K, K);
    if (dgamma_s) o.out(dgamma_s, 1, K, K);
    if (gg_own) o.out(dgate, M, K, lddgate);
    else if (dgate && !own) o.out(dgate, 1, K, K);
    if (sums) o.workspace(workspace, workspace_bytes, 4 * (unsigned __int128)block_norm_bwd_workspace_floats(M, K));
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const BlockNormBwd a{(int)M, (int)K, dY, U, S, gamma_u, gate, gamma_s, rstd_u, rstd_s, dS, gu ? dU : nullptr,
                         gx ? dX : nullptr, dgamma_u, dgamma_s, own && M == 0 ? nullptr : dgate,
                         sums ? static_cast<float *>(workspace) : nullptr, lddy, ldu, lds, own ? ldgate : 0,
                         dS ? ldds : 0, lddu, lddx, own ? lddgate : 0, alpha, own, accumulate == 1};
    return launch_status(launch_block_norm_bwd(a, hip_stream(stream)));
}

}  // extern "C"
