// api_layers.hip -- the C entry points of the dense layers and the norm
// (declared in gemvgemm.h): argument checks as in api.hip, before any HIP
// call and before anything is written, then the launchers of kernels.hpp.
// Nothing here allocates, so no exception can arise.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/gemvgemm.h"
#include "checks.hpp"
#include "kernels.hpp"

using namespace gg;

namespace {

int packed_linear(int bits, int act, int64_t M, int64_t N, int64_t K, const uint8_t *X8,
                  int64_t ldx, const uint8_t *XE, int64_t ldxe, const uint8_t *Q, int64_t ldq,
                  const uint16_t *S, int64_t lds, const float *bias, const float *R, int64_t ldr,
                  float *Y, int64_t ldy, uint8_t *Y8, int64_t ldy8, uint8_t *YE, int64_t ldye,
                  gg_stream_t stream) {
    if (bad_act(act) || bad_size(M) || bad_size(N) || bad_size(K)) return GG_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GG_OK;
    if ((Y8 == nullptr) != (YE == nullptr) || (Y == nullptr && Y8 == nullptr))
        return GG_ERR_INVALID_ARG;
    const int64_t per_byte = 8 / bits;
    Operands o;
    o.in(X8, M, K, ldx, 1).in(XE, M, (K + 31) / 32, ldxe, 1);
    o.in(Q, N, (K + per_byte - 1) / per_byte, ldq, 1).in(S, N, (K + 63) / 64, lds, 2);
    if (bias) o.in(bias, 1, N, N);
    if (R) o.replaced(R, M, N, ldr);
    if (Y) o.onto(Y, M, N, ldy);
    if (Y8) o.out(Y8, M, N, ldy8, 1).out(YE, M, (N + 31) / 32, ldye, 1);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const PackedLinear a{act, (int)M, (int)N, (int)K, X8, XE, Q, S, bias, R, Y, Y8, YE,
                         ldx, ldxe, ldq, lds, R ? ldr : 0, Y ? ldy : 0, Y8 ? ldy8 : 0, YE ? ldye : 0};
    return launch_status(launch_packed_linear(bits, a, cus, reinterpret_cast<hipStream_t>(stream)));
}

// The norm with its output in fp32 (Q null) or in 8 bits (Y null).
int rmsnorm(int64_t M, int64_t K, const float *X, int64_t ldx, const float *R, int64_t ldr,
            const float *gamma, float eps, float *S, int64_t lds, float *Y, int64_t ldy,
            uint8_t *Q, int64_t ldq, uint8_t *E, int64_t lde, bool mx8, float *rstd,
            gg_stream_t stream) {
    if (bad_size(M) || bad_size(K) || !(eps >= 0.f) || std::isinf(eps)) return GG_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return GG_OK;
    Operands o;
    o.replaced(X, M, K, ldx);
    if (R) o.replaced(R, M, K, ldr);
    if (gamma) o.in(gamma, 1, K, K);
    if (S) o.onto(S, M, K, lds);
    if (mx8) o.out(Q, M, K, ldq, 1).out(E, M, (K + 31) / 32, lde, 1);
    else o.out(Y, M, K, ldy);
    if (rstd) o.out(rstd, 1, M, M);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const RmsNorm a{(int)M, (int)K, X, R, gamma, S, Y, rstd, Q, E, ldx, R ? ldr : 0,
                    S ? lds : 0, ldy, ldq, lde, eps};
    return launch_status(launch_rmsnorm(a, reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

int linear_f32(int trans_w, int act, int64_t M, int64_t N, int64_t K, const float *X, int64_t ldx,
               const float *W, int64_t ldw, const float *bias, const float *R, int64_t ldr,
               float *Z, int64_t ldz, float *Y, int64_t ldy, gg_stream_t stream) {
    if ((trans_w != 0 && trans_w != 1) || bad_act(act) || bad_size(M) || bad_size(N) || bad_size(K))
        return GG_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GG_OK;
    Operands o;
    o.in(X, M, K, ldx);
    if (trans_w) o.in(W, N, K, ldw);
    else o.in(W, K, N, ldw);
    if (bias) o.in(bias, 1, N, N);
    if (R) o.replaced(R, M, N, ldr);
    if (Z) o.out(Z, M, N, ldz);
    o.onto(Y, M, N, ldy);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    return launch_status(launch_linear(trans_w == 1, act, (int)M, (int)N, (int)K, X, ldx, W, ldw,
                                       bias, R, R ? ldr : 0, Z, Z ? ldz : 0, Y, ldy, cus,
                                       reinterpret_cast<hipStream_t>(stream)));
}

int64_t linear_f32_bwd_ws_size(int act, int64_t M, int64_t N) {
    if (bad_act(act) || bad_size(M) || bad_size(N)) return GG_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return 0;
    const unsigned __int128 bytes = 4 * linear_bwd_workspace_floats(act == GG_ACT_NONE, M, N);
    return bytes > ((unsigned __int128)1 << 62) ? GG_ERR_INVALID_ARG : (int64_t)bytes;
}

int linear_f32_bwd(int trans_w, int act, int accumulate, int64_t M, int64_t N, int64_t K,
                   const float *dY, int64_t lddy, const float *Z, int64_t ldz, const float *X,
                   int64_t ldx, const float *W, int64_t ldw, float *dX, int64_t lddx, float *dW,
                   int64_t lddw, float *db, void *workspace, int64_t workspace_bytes,
                   gg_stream_t stream) {
    if ((trans_w != 0 && trans_w != 1) || (accumulate != 0 && accumulate != 1) || bad_act(act) ||
        bad_size(M) || bad_size(N) || bad_size(K))
        return GG_ERR_INVALID_ARG;
    const int64_t w_rows = trans_w ? N : K, w_cols = trans_w ? K : N;
    // operands of the outputs that are wanted and not empty
    const bool gx = dX != nullptr && M > 0 && K > 0;
    const bool gw = dW != nullptr && N > 0 && K > 0;
    const bool gb = db != nullptr && N > 0;
    if (!gx && !gw && !gb) return GG_OK;
    Operands o;
    o.in(dY, M, N, lddy);
    if (act != GG_ACT_NONE) o.in(Z, M, N, ldz);
    if (gx) o.in(W, w_rows, w_cols, ldw).out(dX, M, K, lddx);
    if (gw) o.in(X, M, K, ldx).out(dW, w_rows, w_cols, lddw);
    if (gb) o.out(db, 1, N, N);
    o.workspace(workspace, workspace_bytes,
                M && N ? 4 * linear_bwd_workspace_floats(act == GG_ACT_NONE, M, N) : 0);
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    return launch_status(launch_linear_bwd(
        trans_w == 1, act, accumulate == 1, (int)M, (int)N, (int)K, dY, lddy, Z,
        act != GG_ACT_NONE ? ldz : 0, X, ldx, W, ldw, gx ? dX : nullptr, lddx, gw ? dW : nullptr,
        lddw, gb ? db : nullptr, static_cast<float *>(workspace), cus,
        reinterpret_cast<hipStream_t>(stream)));
}

int rmsnorm_f32(int64_t M, int64_t K, const float *X, int64_t ldx, const float *R, int64_t ldr,
                const float *gamma, float eps, float *S, int64_t lds, float *Y, int64_t ldy,
                float *rstd, gg_stream_t stream) {
    return rmsnorm(M, K, X, ldx, R, ldr, gamma, eps, S, lds, Y, ldy, nullptr, 0, nullptr, 0, false,
                   rstd, stream);
}

int rmsnorm_mx8(int64_t M, int64_t K, const float *X, int64_t ldx, const float *R, int64_t ldr,
                const float *gamma, float eps, float *S, int64_t lds, uint8_t *Q, int64_t ldq,
                uint8_t *E, int64_t lde, gg_stream_t stream) {
    return rmsnorm(M, K, X, ldx, R, ldr, gamma, eps, S, lds, nullptr, 0, Q, ldq, E, lde, true,
                   nullptr, stream);
}

int64_t rmsnorm_f32_bwd_ws_size(int64_t M, int64_t K) {
    if (bad_size(M) || bad_size(K)) return GG_ERR_INVALID_ARG;
    return 4 * rmsnorm_bwd_workspace_floats(M, K);
}

int rmsnorm_f32_bwd(int accumulate, int64_t M, int64_t K, const float *dY, int64_t lddy,
                    const float *S, int64_t lds, const float *gamma, const float *rstd,
                    const float *dS, int64_t ldds, float *dX, int64_t lddx, float *dgamma,
                    void *workspace, int64_t workspace_bytes, gg_stream_t stream) {
    if ((accumulate != 0 && accumulate != 1) || bad_size(M) || bad_size(K)) return GG_ERR_INVALID_ARG;
    const bool gx = dX != nullptr && M > 0;
    if (K == 0 || (!gx && dgamma == nullptr)) return GG_OK;
    Operands o;
    o.in(dY, M, K, lddy).in(S, M, K, lds);
    if (M > 0) o.in(rstd, 1, M, M);
    if (gamma) o.in(gamma, 1, K, K);
    if (gx && dS) o.replaced(dS, M, K, ldds);
    if (gx) o.onto(dX, M, K, lddx);
    if (dgamma) o.out(dgamma, 1, K, K);
    if (dgamma) o.workspace(workspace, workspace_bytes, 4 * (unsigned __int128)rmsnorm_bwd_workspace_floats(M, K));
    if (int st = o.status()) return st;
    int cus = 0;
    if (int st = check_device(&cus)) return st;
    const RmsNormBwd a{(int)M, (int)K, dY, S, gamma, rstd, gx ? dS : nullptr, gx ? dX : nullptr,
                       dgamma, static_cast<float *>(workspace), lddy, lds, gx && dS ? ldds : 0,
                       gx ? lddx : 0, accumulate == 1};
    return launch_status(launch_rmsnorm_bwd(a, reinterpret_cast<hipStream_t>(stream)));
}

int linear_q4_mx8(int act, int64_t M, int64_t N, int64_t K, const uint8_t *X8, int64_t ldx,
                  const uint8_t *XE, int64_t ldxe, const uint8_t *Q, int64_t ldq,
                  const uint16_t *S, int64_t lds, const float *bias, const float *R, int64_t ldr,
                  float *Y, int64_t ldy, uint8_t *Y8, int64_t ldy8, uint8_t *YE, int64_t ldye,
                  gg_stream_t stream) {
    return packed_linear(4, act, M, N, K, X8, ldx, XE, ldxe, Q, ldq, S, lds, bias, R, ldr, Y, ldy,
                         Y8, ldy8, YE, ldye, stream);
}

int linear_q2_mx8(int act, int64_t M, int64_t N, int64_t K, const uint8_t *X8, int64_t ldx,
                  const uint8_t *XE, int64_t ldxe, const uint8_t *Q, int64_t ldq,
                  const uint16_t *S, int64_t lds, const float *bias, const float *R, int64_t ldr,
                  float *Y, int64_t ldy, uint8_t *Y8, int64_t ldy8, uint8_t *YE, int64_t ldye,
                  gg_stream_t stream) {
    return packed_linear(2, act, M, N, K, X8, ldx, XE, ldxe, Q, ldq, S, lds, bias, R, ldr, Y, ldy,
                         Y8, ldy8, YE, ldye, stream);
}

}  // extern "C"
