/*
 * carbon_lm.h - the operators of a language model's training step around its
 * linear layers: token embedding, root-mean-square norm and the output
 * layer's softmax cross entropy, each with its gradient.  Public C ABI, part
 * of the same library and with the same conventions as carbon_gemm.h (device
 * pointers, dense row-major matrices, asynchronous on `stream`, status codes,
 * fault injection, CARBON_ERR_UNSUPPORTED off GB300).
 *
 * Determinism: no floating-point atomics; every sum has a fixed order, so
 * every result is bit-identical from run to run.  A row's result of
 * carbon_embedding_fwd, carbon_rms_norm_fwd and the dx of carbon_rms_norm_bwd,
 * and a position's loss, lse and dX of carbon_linear_xent_* (dX of
 * CARBON_REDUCE_MEAN but for the count; of CARBON_REDUCE_NONE above the smallest
 * values of G, see there), do not depend on the other rows of the call (batch
 * invariance).  Sums over tokens (the gradients of the table and of gamma)
 * depend on all of them, in a fixed order.
 *
 * Sums, norms and softmax statistics are held in fp32; each output is rounded
 * once, to nearest-even.  dtype is that of every 16- or 32-bit operand and
 * output unless a type is named.  Pointers that are not multiples of their
 * element's size: CARBON_ERR_MISALIGNED.
 *
 * Workspace: where a function takes one, the caller passes a 16-byte aligned
 * device buffer of at least the bytes that its _workspace query returns; the
 * library allocates nothing.  Its contents need not be set and mean nothing
 * afterwards; two calls that may overlap on the GPU need one each.  About:
 *   carbon_embedding_bwd     M (16 + D / 2) bytes (a histogram per 1024 or 8192
 *                            tokens more above 8192 tokens)
 *   carbon_rms_norm_bwd      at most 608 rows of D fp32 values
 *   carbon_linear_xent_fwd   M (2 D + V / 16) bytes
 *   carbon_linear_xent_bwd   M (6 D + 24576) bytes (the logits would take
 *                            4 M V), and up to 128 MiB more below about 2500
 *                            positions.  M = 8192, D = 768: 240 MB
 *
 * Indices that name no row (a token id outside [0, V); a target that is
 * neither ignore_index nor in [0, V)): the lookup gives a row of zeros, the
 * gradients leave it out, the loss treats the position as ignored, and
 * carbon_get_device_status() reports CARBON_ERR_OUT_OF_BOUNDS.
 */
#ifndef CARBON_LM_H
#define CARBON_LM_H

#include "carbon_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- token embedding -------------------------------------------------------
 *
 * table[V,D], ids[M] (int64), out[M,D]:   out[m] = scale * table[ids[m]] */
carbon_status_t carbon_embedding_fwd(void *out, const void *table, const int64_t *ids, int64_t M,
                                     int64_t V, int64_t D, float scale, carbon_dtype_t dtype,
                                     carbon_stream_t stream);

/* dtable[v] = scale * sum over m with ids[m] == v of dy[m], summed in fp32
 * over the tokens sorted by (id, position), for every row v of the table
 * (zeros where no token names v).  accumulate != 0: the sum is added to the
 * dtable already there instead (one rounding), and rows that no token names
 * are left alone -- e.g. onto the output layer's gradient of a tied table.
 * padding_idx: a row that gets no gradient, or -1.
 * Workspace: carbon_embedding_bwd_workspace bytes. */
carbon_status_t carbon_embedding_bwd(void *dtable, const void *dy, const int64_t *ids, int64_t M,
                                     int64_t V, int64_t D, float scale, int64_t padding_idx,
                                     int accumulate, void *workspace, int64_t workspace_bytes,
                                     carbon_dtype_t dtype, carbon_stream_t stream);
/* Bytes, or -1 where the sizes are invalid. */
int64_t carbon_embedding_bwd_workspace(int64_t M, int64_t V, int64_t D);

/* ---- root-mean-square norm -------------------------------------------------
 *
 *   h = x + residual            (residual may be NULL: h = x)
 *   rstd[m] = 1 / sqrt(mean_j h[m,j]^2 + eps)
 *   n = h * rstd,   y = n * gamma
 *
 * from the unrounded fp32 sum h.  h_out (may be NULL): h rounded to dtype,
 * the residual stream that goes on.  rstd (may be NULL): fp32 [M].
 * codes and scales (both or neither): an 8-bit checkpoint of n, with a scale
 * per token: scales[m] = max_j |n[m,j]| / 127, codes[m,j] = n[m,j] / scales[m]
 * to the nearest integer (n times the fp32 quotient 127 / max).  A row whose
 * maximum is below 2^-100 has scale 0 and codes 0; a row with a NaN or an
 * infinity has scale NaN and codes 0, so that it reads back as NaN.
 * y and h_out may each lie over x or residual (the same address); else no
 * operands overlap.  gamma[D].  D = 0 or M = 0: nothing to do. */
carbon_status_t carbon_rms_norm_fwd(void *y, void *h_out, float *rstd, int8_t *codes, float *scales,
                                    const void *x, const void *residual, const void *gamma,
                                    int64_t M, int64_t D, float eps, carbon_dtype_t dtype,
                                    carbon_stream_t stream);

/* Gradients, from h and rstd, or from the 8-bit checkpoint (h NULL; codes and
 * scales given; n = codes * scales):
 *
 *   dx     = rstd * (gamma*dy - n * mean_j(gamma*dy*n)) + dh     (also the gradient of residual)
 *   dgamma = sum_m dy * n
 *
 * dh: the gradient that reaches h along the residual stream, or NULL.
 * dgamma may be NULL.  y_out (may be NULL): y = n * gamma once more, e.g. for
 * the weight gradient of the linear layer that took y.  dx and y_out may not
 * overlap another operand, except dx == dh.  Workspace: carbon_rms_norm_bwd_workspace
 * bytes (the partial sums of dgamma). */
carbon_status_t carbon_rms_norm_bwd(void *dx, void *dgamma, void *y_out, const void *dy,
                                    const void *h, const int8_t *codes, const float *scales,
                                    const float *rstd, const void *gamma, const void *dh,
                                    int64_t M, int64_t D, void *workspace, int64_t workspace_bytes,
                                    carbon_dtype_t dtype, carbon_stream_t stream);
int64_t carbon_rms_norm_bwd_workspace(int64_t M, int64_t D);

/* out = codes * scales (* gamma, where it is not NULL): reads an 8-bit
 * checkpoint back. */
carbon_status_t carbon_rms_norm_expand(void *out, const int8_t *codes, const float *scales,
                                       const void *gamma, int64_t M, int64_t D,
                                       carbon_dtype_t dtype, carbon_stream_t stream);

/* ---- linear layer + softmax cross entropy over a large vocabulary ----------
 *
 * x[M,D], table[V,D] (one row per vocabulary entry, as an embedding's table
 * is stored: tied weights pass it as it is), targets[M] (int64):
 *
 *   z[m] = table . x[m],  lse[m] = log sum_v exp(z[m,v]),
 *   loss[m] = lse[m] - z[m,targets[m]]
 *
 * The logits are formed in tiles on the tensor cores and never stored.
 * Positions whose target is ignore_index cost nothing, have loss 0 and lse 0,
 * and neither they nor their x (NaN included) reach any other result.
 *
 * dtype: CARBON_BF16 or CARBON_F16 (CARBON_F32: CARBON_ERR_UNSUPPORTED, as
 * on the tensor-core tier).  x, table, dx and dtable 16-byte aligned and D a
 * multiple of 8, else CARBON_ERR_MISALIGNED.  M, V < 2^30, D <= 4194240 and fewer
 * than 2^31 tiles of 256 x 128 among the logits, else
 * CARBON_ERR_INVALID_ARG (as for V = 0 or D = 0 where M > 0). */
typedef enum {
    CARBON_REDUCE_NONE = 0,     /* a loss per position */
    CARBON_REDUCE_SUM = 1,      /* their sum */
    CARBON_REDUCE_MEAN = 2      /* their sum / max(positions that count, 1) */
} carbon_reduce_t;

/* Errors: a logit is within D 2^-23 sum_j |x_j w_j| of the exact one (exact
 * products, the tensor cores' fp32 accumulator); lse within the largest of these
 * of its row plus (16 + log2 V) 2^-23 (|lse| + |z| + 1), z the target's logit; a
 * loss within twice the former plus the latter.
 *
 * losses: fp32 [M].  total: fp32 [1], the sum or mean (fixed order), NULL for
 * CARBON_REDUCE_NONE.  lse: fp32 [M].  count: int64 [1], the number of
 * positions that count.  Workspace: carbon_linear_xent_fwd_workspace bytes. */
carbon_status_t carbon_linear_xent_fwd(float *losses, float *total, float *lse, int64_t *count,
                                       const void *x, const void *table, const int64_t *targets,
                                       int64_t M, int64_t D, int64_t V, int64_t ignore_index,
                                       carbon_reduce_t reduction, void *workspace,
                                       int64_t workspace_bytes, carbon_dtype_t dtype,
                                       carbon_stream_t stream);
int64_t carbon_linear_xent_fwd_workspace(int64_t M, int64_t D, int64_t V);

/* dx[M,D] and dtable[V,D] from grad (fp32: [M] for CARBON_REDUCE_NONE, else
 * [1]) and the forward's lse.  With g[m] the gradient of loss[m] (divided by
 * the count for CARBON_REDUCE_MEAN) and P = softmax(z):
 *
 *   G[m,v] = g[m] * (P[m,v] - [v == targets[m]]),  dx = G . table,  dtable = G^T . x
 *
 * The logits are formed again, a piece of the vocabulary at a time.  G enters
 * the tensor cores in dtype, with |g| between 1 and 2 for the largest finite
 * one (a power of two is taken out); the sums are fp32.  Entries of G then keep
 * the type's precision down to 2^-26 (CARBON_F16) or 2^-158 (CARBON_BF16) and
 * lose bits below: with CARBON_REDUCE_NONE the only way in which the gradients
 * of other positions reach a row of dx.  A g that is not finite makes its own
 * row of dx, and dtable, not finite, and no other row of dx.  dtable is written
 * whole.
 * Workspace: carbon_linear_xent_bwd_workspace bytes. */
carbon_status_t carbon_linear_xent_bwd(void *dx, void *dtable, const float *grad, const void *x,
                                       const void *table, const int64_t *targets, const float *lse,
                                       int64_t M, int64_t D, int64_t V, int64_t ignore_index,
                                       carbon_reduce_t reduction, void *workspace,
                                       int64_t workspace_bytes, carbon_dtype_t dtype,
                                       carbon_stream_t stream);
int64_t carbon_linear_xent_bwd_workspace(int64_t M, int64_t D, int64_t V);

#ifdef __cplusplus
}
#endif

#endif /* CARBON_LM_H */
