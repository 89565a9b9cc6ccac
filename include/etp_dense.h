/*
 * etp_dense.h -- C ABI of libetp's dense operators: the layers of the radial
 * and node networks around the tensor product, and the update of their
 * weights, on AMD Instinct MI355X (gfx950).
 *
 * The convolution with radial weights (etp_edge_conv_fwd_radial, etp.h)
 * takes per-edge features h "from the hidden layers of a radial network" and
 * its VJP hands back grad_h. These calls are those hidden layers -- a linear
 * layer with bias, activation and residual, and the layer norm -- with their
 * VJPs, the linear layer with a matrix for each group of rows (an element, a
 * pair of elements), the norm of all gradients with clipping, and the
 * orthogonalised update of a weight matrix (of these layers, of
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
 *     a float (not in etp_grouped_linear_vjp without an activation, where d is
 *     a bf16 too).
 *   - sums are float. A matrix instruction drops what lies below the last place
 *     of the sum so far, always to the same side: n results on top of each
 *     other leave a sum whose terms are all alike off by up to n 2^-24 of itself
 *     (32 terms take six results of float layers, three or one of bf16 ones).
 *     This holds for the sums along a row (n_in, n_out) and for etp_linear_vjp's
 *     along the rows: 100000 alike rows of a 2048 x 2048 layer left grad_W 8e-4
 *     off. etp_grouped_linear_vjp holds n to 256 there (1.7e-5 at any number of
 *     rows, also in a single group).
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

/* Rows grouped by a type id (an atom's element, an edge's pair of elements):
 *   group_ptr[g] = the number of rows with 0 <= ids[r] < g,   g = 0 .. n_groups
 *   order[s]     = the rows by group, in row order within each (a stable sort);
 * rows whose id is none of 0 .. n_groups - 1 (padding) are in no group and come
 * behind, from group_ptr[n_groups] on. ids int32 [n_rows]; group_ptr int32
 * [n_groups + 1]; order int32 [n_rows]. For the types of a fixed structure this
 * is done once. (etp_csr_transpose groups edges by source too, in a time that
 * grows with the square of a long group.) ws: DEVICE, 16-byte aligned, at least
 * etp_group_rows_workspace() bytes (NULL where that is 0). n_rows = 0 writes
 * zeros into group_ptr. Errors: INVALID_ARGUMENT (null group_ptr, null ids or
 * order with n_rows > 0, negative n_rows, n_groups below 1, misaligned
 * pointers), UNSUPPORTED (n_rows >= 2^31, n_groups >= 2^16), WORKSPACE, HIP. */
ETP_API etp_status etp_group_rows(int64_t n_rows, int32_t n_groups, const int32_t *ids, int32_t *group_ptr,
                                  int32_t *order, void *ws, size_t ws_bytes, void *stream);

/* Workspace (bytes) of etp_group_rows. Host only. Errors: INVALID_ARGUMENT
 * (null bytes, negative n_rows, n_groups below 1), UNSUPPORTED. */
ETP_API etp_status etp_group_rows_workspace(int64_t n_rows, int32_t n_groups, size_t *bytes);

/* Linear layer with a matrix for each group of rows:
 *   z[r, j] = sum_k x[r, k] W[g, k, j] + bias[g, j],   y[r, j] = act(z[r, j]) + residual[r, j]
 * for every row r = order[s], group_ptr[g] <= s < group_ptr[g + 1] (order NULL:
 * r = s, rows that lie in groups). Features stay in the caller's row order.
 * W [n_groups][n_in][n_out]; bias float [n_groups][n_out] or NULL; everything
 * else as etp_linear. Rows in no group (before group_ptr[0], behind
 * group_ptr[n_groups]) have no effect and are not written. group_ptr, order: DEVICE
 * int32, as etp_group_rows writes them, and trusted: a row named twice is written
 * twice, in any order (an index that is no row is passed over, offsets outside [0,
 * n_rows] are held to that range). The sizes of the groups are not read back, so
 * that empty groups cost a little each and count in the choice of the kernel: 21
 * rows take 9 us in 64 groups, 11 in 5041, 82 in 65535 (of 16 x 16; of 16 x 1024
 * 1.2 ms); 100000 rows in 25 groups take up to three times as long when 5041
 * are named. Number the types that occur. Errors: as etp_linear, plus INVALID_ARGUMENT
 * (null group_ptr, n_groups below 1), UNSUPPORTED (n_groups >= 2^16). */
ETP_API etp_status etp_grouped_linear(int64_t n_rows, int32_t n_groups, const int32_t *group_ptr,
                                      const int32_t *order, int32_t n_in, int32_t n_out, int32_t dtype, const void *x,
                                      int64_t ldx, const void *W, const float *bias, int32_t activation,
                                      const void *residual, int64_t ldr, void *y, int64_t ldy, void *z, int64_t ldz,
                                      void *stream);

/* VJP of etp_grouped_linear: with d = grad_y * act'(z), for the rows of each group
 *   grad_x[r, k]    = sum_j d[r, j] W[g, k, j]         (dtype, pitch ldgx)
 *   grad_W[g, k, j] = sum_{r in g} x[r, k] d[r, j]     (float [n_groups][n_in][n_out])
 *   grad_b[g, j]    = sum_{r in g} d[r, j]             (float [n_groups][n_out])
 * Outputs, flags, z and ws as etp_linear_vjp, with
 * etp_grouped_linear_vjp_workspace() bytes (needed for grad_W and grad_b). d is a
 * float also when the features are bf16; without an activation it is grad_y as
 * stored. Gradients of groups without rows are zero (or left as they are when
 * accumulating); rows of grad_x in no group are not written. Errors: as
 * etp_linear_vjp, plus those of etp_grouped_linear. */
ETP_API etp_status etp_grouped_linear_vjp(int64_t n_rows, int32_t n_groups, const int32_t *group_ptr,
                                          const int32_t *order, int32_t n_in, int32_t n_out, int32_t dtype,
                                          const void *x, int64_t ldx, const void *W, const void *z, int64_t ldz,
                                          int32_t activation, const void *grad_y, int64_t ldgy, void *grad_x,
                                          int64_t ldgx, float *grad_W, float *grad_b, uint32_t flags, void *ws,
                                          size_t ws_bytes, void *stream);

/* Workspace (bytes) of etp_grouped_linear_vjp. Host only. Errors: as
 * etp_linear_vjp_workspace, plus n_groups as etp_grouped_linear. */
ETP_API etp_status etp_grouped_linear_vjp_workspace(int64_t n_rows, int32_t n_groups, int32_t n_in, int32_t n_out,
                                                    int32_t dtype, size_t *bytes);

/* One tensor of a list (the list is a HOST array): numel entries of dtype, dense. */
typedef struct {
    const void *data; /* DEVICE; may be NULL where numel is 0 */
    int64_t numel;
    int32_t dtype; /* etp_dtype */
} etp_tensor;

/* Norm of all tensors taken as one vector,
 *   norm = sqrt(sum_i sum_e grads[i][e]^2)
 * with squares and sums in double and one rounding to float at the end: no
 * square overflows or vanishes. norm: DEVICE float. It is not finite where an
 * entry is not (or where the norm is no float). The list is read during the call
 * only; a captured graph keeps the addresses. n_tensors = 0 gives 0. ws: DEVICE,
 * 16-byte aligned, at least etp_grad_norm_workspace() bytes. Errors:
 * INVALID_ARGUMENT (null list with n_tensors > 0, null norm, negative n_tensors
 * or numel, null data with numel > 0, unknown dtype, misaligned pointers),
 * UNSUPPORTED (a numel of 2^43 or more), WORKSPACE, HIP. */
ETP_API etp_status etp_grad_norm(int32_t n_tensors, const etp_tensor *grads, float *norm, void *ws, size_t ws_bytes,
                                 void *stream);

/* Clipping to a largest norm: with norm as above (kept in double),
 *   out[i][e] = grads[i][e] * (norm <= max_norm ? 1 : max_norm / norm)
 * where a float's product is formed in double and rounded once, and a bf16's scale
 * and product are each rounded to float before the result is to bf16. out: HOST array of
 * DEVICE pointers, each of its tensor's type, dense, equal to its tensor's data (in
 * place) or apart from every tensor of the call (which is not looked for: other
 * overlaps are races); NULL: all in place, apart from each other. In place nothing
 * is written when the norm is small enough. An infinite norm gives zeros (NaN from the
 * infinite entries), a NaN makes every entry NaN: *norm tells. norm: DEVICE float,
 * written when not NULL.
 * max_norm: finite, >= 0. ws as etp_grad_norm. Errors: as etp_grad_norm (norm may
 * be NULL), plus INVALID_ARGUMENT (max_norm, an out[i] that is null with entries
 * or misaligned). */
ETP_API etp_status etp_clip_grads(int32_t n_tensors, const etp_tensor *grads, float max_norm, void *const *out,
                                  float *norm, void *ws, size_t ws_bytes, void *stream);

/* Workspace (bytes) of etp_grad_norm and etp_clip_grads for a list; its data
 * pointers are not looked at. Host only. Errors: INVALID_ARGUMENT (null bytes,
 * otherwise as etp_grad_norm), UNSUPPORTED. */
ETP_API etp_status etp_grad_norm_workspace(int32_t n_tensors, const etp_tensor *grads, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* ETP_DENSE_H */
