// etp_dense_api.hip -- the C ABI declared in include/etp_dense.h: host-side
// argument validation and dispatch to the launchers.
#include <cmath>

#include "../../include/etp_dense.h"
#include "etp_dense.hpp"

namespace {

constexpr int kMaxWidth = 65536;

etp_status status_of(hipError_t e) { return e == hipSuccess ? ETP_OK : ETP_ERR_HIP; }

bool misaligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Sizes and storage type of a call over rows.
etp_status check_sizes(int64_t n_rows, int32_t w0, int32_t w1, int32_t dtype)
{
    if (n_rows < 0 || w0 < 1 || w1 < 1 || (dtype != ETP_F32 && dtype != ETP_BF16))
        return ETP_ERR_INVALID_ARGUMENT;
    if (n_rows >= (int64_t{1} << 31) || w0 > kMaxWidth || w1 > kMaxWidth)
        return ETP_ERR_UNSUPPORTED;
    return ETP_OK;
}

// A feature matrix [n_rows][width] of the given element size; null is
// allowed where `optional`.
etp_status check_rows(const void *p, int64_t ld, int32_t width, size_t elem, bool optional)
{
    if (!p)
        return optional ? ETP_OK : ETP_ERR_INVALID_ARGUMENT;
    if (ld < width || misaligned(p, elem))
        return ETP_ERR_INVALID_ARGUMENT;
    return ld >= (int64_t{1} << 31) ? ETP_ERR_UNSUPPORTED : ETP_OK;
}

etp_status check_ws(const void *ws, size_t have, size_t need)
{
    return need == 0 || (ws && !misaligned(ws, 16) && have >= need) ? ETP_OK : ETP_ERR_WORKSPACE;
}

bool positive_finite(float v) { return std::isfinite(v) && v > 0.f; }

#define ETP_TRY(expr)                  \
    do {                               \
        const etp_status st_ = (expr); \
        if (st_ != ETP_OK)             \
            return st_;                \
    } while (0)

}  // namespace

extern "C" {

etp_status etp_linear(int64_t n_rows, int32_t n_in, int32_t n_out, int32_t dtype, const void *x, int64_t ldx,
                      const void *W, const float *bias, int32_t activation, const void *residual, int64_t ldr,
                      void *y, int64_t ldy, void *z, int64_t ldz, void *stream)
{
    ETP_TRY(check_sizes(n_rows, n_in, n_out, dtype));
    if (activation < ETP_ACT_NONE || activation > ETP_ACT_GELU)
        return ETP_ERR_INVALID_ARGUMENT;
    if (n_rows == 0)
        return ETP_OK;
    const size_t e = dtype == ETP_BF16 ? 2 : 4;
    ETP_TRY(check_rows(x, ldx, n_in, e, false));
    ETP_TRY(check_rows(W, n_out, n_out, e, false));
    ETP_TRY(check_rows(y, ldy, n_out, e, false));
    ETP_TRY(check_rows(residual, ldr, n_out, e, true));
    ETP_TRY(check_rows(z, ldz, n_out, e, true));
    if (misaligned(bias, 4))
        return ETP_ERR_INVALID_ARGUMENT;
    const etp::LinearArgs a{n_rows, n_in, n_out, dtype == ETP_BF16, x,   ldx, W, bias, activation,
                            residual, ldr, y, ldy, z, ldz};
    return status_of(etp::launch_linear(a, static_cast<hipStream_t>(stream)));
}

etp_status etp_linear_vjp_workspace(int64_t n_rows, int32_t n_in, int32_t n_out, int32_t dtype, size_t *bytes)
{
    if (!bytes)
        return ETP_ERR_INVALID_ARGUMENT;
    ETP_TRY(check_sizes(n_rows, n_in, n_out, dtype));
    *bytes = etp::linear_vjp_workspace_bytes(n_rows, n_in, n_out, dtype == ETP_BF16);
    return ETP_OK;
}

etp_status etp_linear_vjp(int64_t n_rows, int32_t n_in, int32_t n_out, int32_t dtype, const void *x, int64_t ldx,
                          const void *W, const void *z, int64_t ldz, int32_t activation, const void *grad_y,
                          int64_t ldgy, void *grad_x, int64_t ldgx, float *grad_W, float *grad_b, uint32_t flags,
                          void *ws, size_t ws_bytes, void *stream)
{
    ETP_TRY(check_sizes(n_rows, n_in, n_out, dtype));
    if (activation < ETP_ACT_NONE || activation > ETP_ACT_GELU)
        return ETP_ERR_INVALID_ARGUMENT;
    if (flags & ~static_cast<uint32_t>(ETP_FLAG_ACCUMULATE))
        return ETP_ERR_INVALID_ARGUMENT;
    const size_t e = dtype == ETP_BF16 ? 2 : 4;
    if (n_rows > 0) {
        ETP_TRY(check_rows(x, ldx, n_in, e, !grad_W));
        ETP_TRY(check_rows(W, n_out, n_out, e, !grad_x));
        ETP_TRY(check_rows(z, ldz, n_out, e, activation == ETP_ACT_NONE));
        ETP_TRY(check_rows(grad_y, ldgy, n_out, e, !grad_x && !grad_W && !grad_b));
        ETP_TRY(check_rows(grad_x, ldgx, n_in, e, true));
    }
    if (misaligned(grad_W, 4) || misaligned(grad_b, 4))
        return ETP_ERR_INVALID_ARGUMENT;
    const bool bf = dtype == ETP_BF16;
    if (grad_W || grad_b)
        ETP_TRY(check_ws(ws, ws_bytes, etp::linear_vjp_workspace_bytes(n_rows, n_in, n_out, bf)));
    const etp::LinearVjpArgs a{n_rows, n_in, n_out, bf, (flags & ETP_FLAG_ACCUMULATE) != 0, x, ldx, W, z, ldz,
                               activation, grad_y, ldgy, grad_x, ldgx, grad_W, grad_b, ws};
    return status_of(etp::launch_linear_vjp(a, static_cast<hipStream_t>(stream)));
}

etp_status etp_layer_norm(int64_t n_rows, int32_t n_cols, int32_t dtype, const void *x, int64_t ldx,
                          const float *gamma, const float *beta, float eps, void *y, int64_t ldy, float *mean,
                          float *rstd, void *stream)
{
    ETP_TRY(check_sizes(n_rows, n_cols, 1, dtype));
    if (!positive_finite(eps))
        return ETP_ERR_INVALID_ARGUMENT;
    if (n_rows == 0)
        return ETP_OK;
    const size_t e = dtype == ETP_BF16 ? 2 : 4;
    ETP_TRY(check_rows(x, ldx, n_cols, e, false));
    ETP_TRY(check_rows(y, ldy, n_cols, e, false));
    if (misaligned(gamma, 4) || misaligned(beta, 4) || misaligned(mean, 4) || misaligned(rstd, 4))
        return ETP_ERR_INVALID_ARGUMENT;
    const etp::NormArgs a{n_rows, n_cols, dtype == ETP_BF16, x, ldx, gamma, beta, eps, y, ldy, mean, rstd};
    return status_of(etp::launch_layer_norm(a, static_cast<hipStream_t>(stream)));
}

etp_status etp_layer_norm_vjp_workspace(int64_t n_rows, int32_t n_cols, int32_t dtype, size_t *bytes)
{
    if (!bytes)
        return ETP_ERR_INVALID_ARGUMENT;
    ETP_TRY(check_sizes(n_rows, n_cols, 1, dtype));
    *bytes = etp::layer_norm_vjp_workspace_bytes(n_rows, n_cols, dtype == ETP_BF16);
    return ETP_OK;
}

etp_status etp_layer_norm_vjp(int64_t n_rows, int32_t n_cols, int32_t dtype, const void *x, int64_t ldx,
                              const float *gamma, const float *mean, const float *rstd, const void *grad_y,
                              int64_t ldgy, void *grad_x, int64_t ldgx, float *grad_gamma, float *grad_beta,
                              uint32_t flags, void *ws, size_t ws_bytes, void *stream)
{
    ETP_TRY(check_sizes(n_rows, n_cols, 1, dtype));
    if (flags & ~static_cast<uint32_t>(ETP_FLAG_ACCUMULATE))
        return ETP_ERR_INVALID_ARGUMENT;
    const size_t e = dtype == ETP_BF16 ? 2 : 4;
    if (n_rows > 0) {
        if (!mean || !rstd)
            return ETP_ERR_INVALID_ARGUMENT;
        ETP_TRY(check_rows(x, ldx, n_cols, e, false));
        ETP_TRY(check_rows(grad_y, ldgy, n_cols, e, false));
        ETP_TRY(check_rows(grad_x, ldgx, n_cols, e, true));
    }
    if (misaligned(gamma, 4) || misaligned(mean, 4) || misaligned(rstd, 4) || misaligned(grad_gamma, 4) ||
        misaligned(grad_beta, 4))
        return ETP_ERR_INVALID_ARGUMENT;
    const bool bf = dtype == ETP_BF16;
    if (grad_gamma || grad_beta)
        ETP_TRY(check_ws(ws, ws_bytes, etp::layer_norm_vjp_workspace_bytes(n_rows, n_cols, bf)));
    const etp::NormVjpArgs a{n_rows, n_cols, bf, (flags & ETP_FLAG_ACCUMULATE) != 0, x, ldx, gamma, mean, rstd,
                             grad_y, ldgy, grad_x, ldgx, grad_gamma, grad_beta, ws};
    return status_of(etp::launch_layer_norm_vjp(a, static_cast<hipStream_t>(stream)));
}

static etp_status check_mats(int32_t n_mats, int32_t rows, int32_t cols, int32_t dtype)
{
    if (n_mats < 0)
        return ETP_ERR_INVALID_ARGUMENT;
    ETP_TRY(check_sizes(0, rows, cols, dtype));
    return n_mats >= 65536 ? ETP_ERR_UNSUPPORTED : ETP_OK;
}

etp_status etp_orthogonalize_workspace(int32_t n_mats, int32_t rows, int32_t cols, int32_t dtype, size_t *bytes)
{
    if (!bytes)
        return ETP_ERR_INVALID_ARGUMENT;
    ETP_TRY(check_mats(n_mats, rows, cols, dtype));
    *bytes = n_mats ? etp::orthogonalize_workspace_bytes(n_mats, rows, cols) : 0;
    return ETP_OK;
}

etp_status etp_orthogonalize(int32_t n_mats, int32_t rows, int32_t cols, int32_t dtype, const void *G, int32_t steps,
                             const float *coef, float eps, void *X, void *ws, size_t ws_bytes, void *stream)
{
    ETP_TRY(check_mats(n_mats, rows, cols, dtype));
    if (steps < 1 || steps > 64 || !positive_finite(eps))
        return ETP_ERR_INVALID_ARGUMENT;
    if (coef && !(std::isfinite(coef[0]) && std::isfinite(coef[1]) && std::isfinite(coef[2])))
        return ETP_ERR_INVALID_ARGUMENT;
    if (n_mats == 0)
        return ETP_OK;
    const size_t e = dtype == ETP_BF16 ? 2 : 4;
    ETP_TRY(check_rows(G, cols, cols, e, false));
    ETP_TRY(check_rows(X, cols, cols, e, false));
    const bool bf = dtype == ETP_BF16;
    ETP_TRY(check_ws(ws, ws_bytes, etp::orthogonalize_workspace_bytes(n_mats, rows, cols)));
    etp::OrthArgs a{n_mats, rows, cols, bf, G, steps, {3.4445f, -4.7750f, 2.0315f}, eps, X, ws};
    if (coef)
        for (int i = 0; i < 3; ++i)
            a.coef[i] = coef[i];
    return status_of(etp::launch_orthogonalize(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
