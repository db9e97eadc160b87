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
 *   carbon_linear_logp_fwd   M (2 D + 3 V / 32) bytes; with alternatives 4 M V more
 *                            up to 256 positions, above M (top + 5) V / 128 or, below
 *                            some thousand positions, up to 8 times as much
 *   carbon_linear_logp_bwd   as carbon_linear_xent_bwd
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

/* ---- log probabilities of given tokens ------------------------------------------
 *
 * x[M,D], table[V,D] and tokens[M] as x, table and targets above, and with the
 * same limits.  With z[m] = table . x[m] / temperature and P = softmax(z):
 *
 *   lse[m] = log sum_v exp z[m,v],   log_probs[m] = z[m,tokens[m]] - lse[m]
 *   entropy[m] = -sum_v P[m,v] log P[m,v]
 *
 * all fp32 [M].  top_ids (int64) and top_log_probs (fp32), [M,top]: the `top`
 * largest entries of P with their logarithms, largest first; not read or written
 * for top = 0.  top <= 28 and top <= V, temperature > 0 (and log2(e) / temperature
 * an fp32 number), else CARBON_ERR_INVALID_ARG.  Positions whose token is
 * ignore_index (or names no entry, see above) cost nothing: log_probs, entropy, lse
 * and top_log_probs 0, top_ids -1.  Places for which no logit above -infinity is
 * left: -1, -infinity.
 *
 * Order of the alternatives: the top + 4 largest logits as the tensor cores form
 * them (their error: see carbon_linear_xent_fwd), ordered by their logits as
 * sums of the exact products in about 48 bits, equal ones by the lower entry.
 * top_log_probs come from the tensor cores' logits, as log_probs do (the same bits
 * for the same entry), but are never above the one before.
 *
 * Logits are multiplied by 1 + D 2^-30, which makes up for the mean of what the
 * tensor cores' accumulator drops (sums that fp32 holds exactly are off by that much
 * instead).  carbon_linear_xent_fwd does not: its loss and -log_probs of the same
 * operands differ by about D 2^-30 of a logit.
 * Errors of log_probs and lse: those of the loss above, of z / temperature;
 * entropy: (16 + log2 V) 2^-23 (entropy + 1) and 2 (entropy + 1) times the largest
 * error of a logit, over the temperature.  log_probs and top_log_probs are formed as
 * differences to the largest logit, so what is near 0 has small errors (where the
 * logits are exact, (16 + log2 V + D / 128) 2^-23 (1 + |log_probs| + entropy)); they are never
 * above 0, and entropy never below.  A position's results do not depend on the other
 * positions. */
carbon_status_t carbon_linear_logp_fwd(float *log_probs, float *entropy, float *lse,
                                       int64_t *top_ids, float *top_log_probs, const void *x,
                                       const void *table, const int64_t *tokens, int64_t M,
                                       int64_t D, int64_t V, int64_t top, float temperature,
                                       int64_t ignore_index, void *workspace,
                                       int64_t workspace_bytes, carbon_dtype_t dtype,
                                       carbon_stream_t stream);
int64_t carbon_linear_logp_fwd_workspace(int64_t M, int64_t D, int64_t V, int64_t top);

/* dx[M,D] and dtable[V,D] from the gradients of log_probs and of entropy (fp32
 * [M], either may be NULL: zeros) and the forward's lse and entropy (entropy may
 * be NULL with grad_entropy):
 *
 *   G[m,v] = grad_log_probs[m] ([v == tokens[m]] - P[m,v])
 *            - grad_entropy[m] P[m,v] (log P[m,v] + entropy[m])
 *   dx = G . table / temperature,   dtable = G^T . x / temperature
 *
 * G is rounded to dtype as for the loss with CARBON_REDUCE_NONE, the power of two
 * being that of the largest finite |grad_log_probs| + (1 + log V) |grad_entropy|.
 * Workspace: carbon_linear_logp_bwd_workspace bytes, about those of the loss. */
carbon_status_t carbon_linear_logp_bwd(void *dx, void *dtable, const float *grad_log_probs,
                                       const float *grad_entropy, const void *x,
                                       const void *table, const int64_t *tokens, const float *lse,
                                       const float *entropy, int64_t M, int64_t D, int64_t V,
                                       float temperature, int64_t ignore_index, void *workspace,
                                       int64_t workspace_bytes, carbon_dtype_t dtype,
                                       carbon_stream_t stream);
int64_t carbon_linear_logp_bwd_workspace(int64_t M, int64_t D, int64_t V);

/* ---- linear layer with low-rank adapters ---------------------------------------
 *
 * x[M,K], w[K,N], bias[N] (may be NULL) as on the tensor-core tier; n adapters of
 * rank r, a[n,K,r] and b[n,r,N], their factors scales[n] (fp32, e.g. alpha / r);
 * adapters[M] (int64): the adapter i of each row, -1 for none.
 *
 *   u[m] = scales[i] (x[m] . a[i]),   y[m] = x[m] . w + bias + u[m] . b[i]
 *
 * in one accumulator, rounded once.  Rows of any order and mix; a row takes
 * nothing from other rows or their adapters (NaN included), and its bits do not
 * depend on them.  A row without an adapter is that of the layer alone.  Another
 * number in adapters than -1 .. n-1 counts as -1 and CARBON_ERR_OUT_OF_BOUNDS is
 * reported by carbon_get_device_status().  Rows that stand together (a request's
 * tokens) cost least: each adapter's products run for every tile of 256 rows that
 * has a row of it.
 *
 * u: carbon_lora_linear_u_elements 16-bit elements, 16-byte aligned, written by
 * the forward and read by the backward pass: [M][3][r rounded up to 16], the
 * 16-bit terms hi and lo of u (u = hi + lo to 2^-17 in bf16, 2^-22 in fp16,
 * relative, and to fp16's smallest step 2^-24), and lo times 2^11.  With fp16 a
 * |u| above 65504 is infinite.  An infinity in x (dy) goes where the formulas take it;
 * one in an adapter's b (a; for the adapters' gradients one in x or dy) may give NaN
 * in place of infinity, for it meets both terms.
 *
 * dtype: CARBON_BF16 or CARBON_F16 (CARBON_F32: CARBON_ERR_UNSUPPORTED).  K, N
 * and r multiples of 8, and y, u, x, w, a, b (dx, da, db, dy) 16-byte aligned, else
 * CARBON_ERR_MISALIGNED.  1 <= r <= 128, K, N <= 2^21, n < 2^24, M < 2^30.  M = 0:
 * nothing to do, and zeros for da and db.
 *
 * Errors: y within (K + 2 r) 2^-23 (sum |x w| + sum |u b|) and the two terms'
 * sum |u b| 2^-16 (2^-21 in fp16) of the exact value, before its rounding; u within
 * (K + 2) 2^-23 scales sum |x a|.
 * Workspace: carbon_lora_linear_fwd_workspace bytes (about 48 M). */
carbon_status_t carbon_lora_linear_fwd(void *y, void *u, const void *x, const void *w,
                                       const void *bias, const void *a, const void *b,
                                       const int64_t *adapters, const float *scales, int64_t M,
                                       int64_t K, int64_t N, int64_t n, int64_t r, void *workspace,
                                       int64_t workspace_bytes, carbon_dtype_t dtype,
                                       carbon_stream_t stream);
/* M * 3 * (r rounded up to 16), or -1 where the sizes are invalid. */
int64_t carbon_lora_linear_u_elements(int64_t M, int64_t r);
int64_t carbon_lora_linear_fwd_workspace(int64_t M, int64_t K, int64_t N, int64_t n, int64_t r);

/* Gradients, from the forward's u:
 *
 *   du[m] = scales[i] (dy[m] . b[i]^T),   dx[m] = dy[m] . w^T + du[m] . a[i]^T
 *   da[i] = sum over the rows m of adapter i of x[m]^T . du[m]
 *   db[i] = sum over them of u[m]^T . dy[m]
 *
 * da and db (both or neither may be NULL) are written whole, zeros for adapters
 * that no row names; dx may be NULL, then w and a may be; without da, x and u
 * may be.  Each adapter's sum takes its rows in their order, 1024 at a time, and
 * depends on them alone.
 * Workspace: carbon_lora_linear_bwd_workspace bytes: 6 M r for du, 52 M, 8 n, and
 * M / 512 partial sums of (K + N) r fp32 numbers. */
carbon_status_t carbon_lora_linear_bwd(void *dx, void *da, void *db, const void *dy, const void *x,
                                       const void *w, const void *a, const void *b,
                                       const int64_t *adapters, const float *scales, const void *u,
                                       int64_t M, int64_t K, int64_t N, int64_t n, int64_t r,
                                       void *workspace, int64_t workspace_bytes,
                                       carbon_dtype_t dtype, carbon_stream_t stream);
int64_t carbon_lora_linear_bwd_workspace(int64_t M, int64_t K, int64_t N, int64_t n, int64_t r);

/* ---- norm of all gradients, and clipping -------------------------------------
 *
 *   norm = sqrt(sum over the `count` tensors and their elements of g^2)
 *   out  = g * min(1, max_norm / (norm + eps))
 *
 * grads, out, sizes (elements) and dtypes (carbon_dtype_t) are arrays on the
 * host, read during the call; the tensors are contiguous and on the device.
 * norm: fp32 [1] on the device, may be NULL; the quotient takes the norm as it
 * is written there.  out may be NULL (the norm alone), and out[i] may be
 * grads[i] (in place: where the factor is 1 nothing is written); what is written
 * may not overlap anything else (CARBON_ERR_INVALID_ARG).  A NaN among the
 * gradients makes the norm and all of out NaN; an infinity makes the norm
 * infinite and the factor 0.  The factor is 1 for max_norm = infinity (unless the
 * norm is NaN), and where norm + eps = 0.
 *
 * Squares are summed in fp32 by 32, in float64 from there on; squares outside
 * fp32's range are scaled, so that the norm overflows only where it is no fp32
 * number itself.  An element's place in the sum depends on the sizes and the
 * order of the tensors, not on their addresses.  max_norm >= 0, eps >= 0.
 * Workspace: carbon_clip_grads_workspace bytes, 4864 for every 256 tensors. */
carbon_status_t carbon_clip_grads(float *norm, void *const *out, const void *const *grads,
                                  const int64_t *sizes, const int *dtypes, int64_t count,
                                  float max_norm, float eps, void *workspace,
                                  int64_t workspace_bytes, carbon_stream_t stream);
/* Bytes, or -1 where the sizes are invalid. */
int64_t carbon_clip_grads_workspace(const int64_t *sizes, int64_t count);

#ifdef __cplusplus
}
#endif

#endif /* CARBON_LM_H */
