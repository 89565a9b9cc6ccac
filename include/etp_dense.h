/*
 * etp_dense.h -- C ABI of libetp's dense operators: the layers of the radial
 * and node networks around the tensor product, and the update of their
 * weights, on AMD Instinct MI355X (gfx950).
 *
 * The convolution with radial weights (etp_edge_conv_fwd_radial, etp.h)
 * takes per-edge features h "from the hidden layers of a radial network" and
 * its VJP hands back grad_h. These calls are those hidden layers -- a linear
 * layer with bias, activation and residual, and the layer norm -- with their
 * VJPs, and the orthogonalised update of a weight matrix (of these layers, of
 * W_r, or of the channel-mixing blocks). There is no VJP of the VJPs here: a
 * loss on forces, which differentiates grad_x of these layers once more, needs
 * the caller's own second pass through them (etp_edge_conv_vjp2_radial is that
 * of the convolution).
 *
 * Conventions as in etp.h: statuses, streams, ownership, DEVICE pointers
 * owned by the caller, validation on the host before any launch, no
 * allocation, no synchronisation, outputs that do not alias inputs (nor each
 * other), fixed-order sums (bitwise reproducible, no atomics). Differences:
 *   - types: `dtype` (ETP_F32 or ETP_BF16) is the storage of features and of
 *     W; bias, gamma, beta, row statistics and the gradients of weights are
 *     float. bf16 outputs are rounded once (nearest even) from float.
 *   - feature matrices have a row pitch ld (elements, >= the row's length),
 *     so that one irrep row of node features can be read in place: element
 *     (r, k) of x is x[r * ldx + k]. Weights and weight gradients are dense.
 *   - pointers need the alignment of their element only (16-byte aligned
 *     rows run faster).
 *   - products are formed on the matrix cores. Float operands are split
 *     exactly into three bf16 parts each and the six leading cross products
 *     are added in float: what is dropped is at most 2^-24 of the product
 *     and of either sign, as a float product's own rounding. (Operands below
 *     2^-110 are held to 2^-134 absolutely.) A non-finite float operand makes
 *     the outputs it contributes to NaN, also where IEEE arithmetic would
 *     give an infinity; so does a bf16 one in the VJP, whose other factor d is
 *     a float.
 * Limits: n_rows < 2^31; widths (n_in, n_out, n_cols, rows, cols) in
 * [1, 65536]; a pitch below 2^31; else UNSUPPORTED (widths below 1:
 * INVALID_ARGUMENT).
 */
#ifndef ETP_DENSE_H
#define ETP_DENSE_H

#include "etp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ETP_ACT_NONE = 0,
    ETP_ACT_SILU = 1, /* z / (1 + exp(-z)) */
    ETP_ACT_GELU = 2, /* z Phi(z), Phi the normal distribution function (erf) */
} etp_activation;

/* Linear layer:
 *   z[r, j] = sum_k x[r, k] W[k, j] + bias[j],   y[r, j] = act(z[r, j]) + residual[r, j]
 * x [n_rows][n_in] pitch ldx; W [n_in][n_out]; bias float [n_out] or NULL;
 * residual [n_rows][n_out] pitch ldr, or NULL; y [n_rows][n_out] pitch ldy;
 * z NULL, or [n_rows][n_out] pitch ldz: the pre-activation, which the VJP of
 * a layer with an activation needs. n_rows = 0 does nothing. Errors:
 * INVALID_ARGUMENT (null x, W or y with n_rows > 0, negative n_rows, width
 * below 1, unknown dtype or activation, a pitch below the row length,
 * misaligned pointers), UNSUPPORTED (limits), HIP. */
ETP_API etp_status etp_linear(int64_t n_rows, int32_t n_in, int32_t n_out, int32_t dtype, const void *x, int64_t ldx,
                              const void *W, const float *bias, int32_t activation, const void *residual,
                              int64_t ldr, void *y, int64_t ldy, void *z, int64_t ldz, void *stream);

/* VJP of etp_linear: with d = grad_y * act'(z),
 *   grad_x[r, k] = sum_j d[r, j] W[k, j]      (dtype, pitch ldgx)
 *   grad_W[k, j] = sum_r x[r, k] d[r, j]      (float [n_in][n_out])
 *   grad_b[j]    = sum_r d[r, j]              (float [n_out])
 * (the residual's gradient is grad_y itself). z: what etp_linear stored, NULL
 * when the activation is NONE. Outputs may be NULL (not computed); x is
 * needed for grad_W only, W for grad_x only. d is a float (three bf16 parts)
 * also when the features are bf16; with n_in and n_out above 128 it is kept
 * once in the workspace.
 * ETP_FLAG_ACCUMULATE adds into every output given. With n_rows = 0 grad_W
 * and grad_b are zeroed (or left as they are when accumulating). ws: DEVICE,
 * 16-byte aligned, at least etp_linear_vjp_workspace() bytes (which count d
 * also for an activation of NONE, where it is grad_y itself), contents
 * undefined afterwards; needed for grad_W and grad_b. Errors: as etp_linear,
 * plus WORKSPACE (ws missing, misaligned or too small), INVALID_ARGUMENT
 * (other flags). */
ETP_API etp_status etp_linear_vjp(int64_t n_rows, int32_t n_in, int32_t n_out, int32_t dtype, const void *x,
                                  int64_t ldx, const void *W, const void *z, int64_t ldz, int32_t activation,
                                  const void *grad_y, int64_t ldgy, void *grad_x, int64_t ldgx, float *grad_W,
                                  float *grad_b, uint32_t flags, void *ws, size_t ws_bytes, void *stream);

/* Workspace (bytes) of etp_linear_vjp. Host only. Errors: INVALID_ARGUMENT
 * (null bytes, negative n_rows, width below 1, unknown dtype), UNSUPPORTED. */
ETP_API etp_status etp_linear_vjp_workspace(int64_t n_rows, int32_t n_in, int32_t n_out, int32_t dtype,
                                            size_t *bytes);

/* Layer norm over the columns of each row:
 *   mean = sum_c x[r, c] / n_cols,  rstd = 1 / sqrt(sum_c (x[r, c] - mean)^2 / n_cols + eps)
 *   y[r, c] = (x[r, c] - mean) rstd gamma[c] + beta[c]
 * x, y: dtype, pitches ldx, ldy; gamma, beta: float [n_cols] or NULL (1 and
 * 0); mean, rstd: float [n_rows], written when not NULL (the VJP needs both).
 * eps: finite, > 0. y is formed from differences that a common offset of the
 * row costs no digits; the variance is summed from them in float. Errors: as
 * etp_linear. */
ETP_API etp_status etp_layer_norm(int64_t n_rows, int32_t n_cols, int32_t dtype, const void *x, int64_t ldx,
                                  const float *gamma, const float *beta, float eps, void *y, int64_t ldy,
                                  float *mean, float *rstd, void *stream);

/* VJP of etp_layer_norm: with h = (x - mean) rstd and d = grad_y gamma,
 *   grad_x = rstd (d - sum_c d / n_cols - h sum_c d h / n_cols)   (dtype, pitch ldgx)
 *   grad_gamma[c] = sum_r grad_y h,  grad_beta[c] = sum_r grad_y  (float [n_cols])
 * mean, rstd: as etp_layer_norm wrote them. Outputs may be NULL (not
 * computed). ETP_FLAG_ACCUMULATE adds into every output given; with
 * n_rows = 0 grad_gamma and grad_beta are zeroed (or left as they are when
 * accumulating). ws: DEVICE, 16-byte aligned, at least
 * etp_layer_norm_vjp_workspace() bytes, needed for grad_gamma and grad_beta.
 * Errors: as etp_linear_vjp. */
ETP_API etp_status etp_layer_norm_vjp(int64_t n_rows, int32_t n_cols, int32_t dtype, const void *x, int64_t ldx,
                                      const float *gamma, const float *mean, const float *rstd, const void *grad_y,
                                      int64_t ldgy, void *grad_x, int64_t ldgx, float *grad_gamma, float *grad_beta,
                                      uint32_t flags, void *ws, size_t ws_bytes, void *stream);

/* Workspace (bytes) of etp_layer_norm_vjp. Host only. Errors: as
 * etp_linear_vjp_workspace. */
ETP_API etp_status etp_layer_norm_vjp_workspace(int64_t n_rows, int32_t n_cols, int32_t dtype, size_t *bytes);

/* Orthogonalised update: for each of n_mats matrices G [rows][cols] (dtype,
 * dense, back to back), X_0 = G / (|G|_F + eps) and `steps` Newton-Schulz steps
 *   X <- coef[0] X + (coef[1] A + coef[2] A^2) X,   A = X X^T
 * (on the transposed matrix when rows > cols), which drive the singular values
 * towards 1 and leave the singular vectors: the update of a weight matrix by
 * the nearest (semi-)orthogonal one. X: dtype [n_mats][rows][cols]. coef: HOST
 * float[3], or NULL for (3.4445, -4.7750, 2.0315), with which five steps take
 * singular values from 0.002 |G|_F up into about [0.7, 1.2]. |G|_F is summed
 * in double; a zero matrix gives zero. steps in [1, 64]; eps finite, > 0. ws:
 * DEVICE, 16-byte aligned, at least etp_orthogonalize_workspace() bytes.
 * Errors: INVALID_ARGUMENT (null G or X, negative n_mats, width below 1,
 * unknown dtype, steps, eps or coef not as above), UNSUPPORTED (limits;
 * n_mats >= 2^16), WORKSPACE, HIP. */
ETP_API etp_status etp_orthogonalize(int32_t n_mats, int32_t rows, int32_t cols, int32_t dtype, const void *G,
                                     int32_t steps, const float *coef, float eps, void *X, void *ws,
                                     size_t ws_bytes, void *stream);

/* Workspace (bytes) of etp_orthogonalize. Host only. Errors: INVALID_ARGUMENT
 * (null bytes, negative n_mats, width below 1, unknown dtype), UNSUPPORTED. */
ETP_API etp_status etp_orthogonalize_workspace(int32_t n_mats, int32_t rows, int32_t cols, int32_t dtype,
                                               size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* ETP_DENSE_H */
