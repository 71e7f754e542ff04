/*
 * libsgemm -- the operators of a language model that sit around its matrix
 * products, on one NVIDIA GB300 (sm_103a): the norms, gate and residual sum
 * between two blocks, the product with 8-bit weights, and the log
 * probabilities that the last product's logits are turned into.
 *
 * Conventions are those of sgemm.h: row-major DEVICE matrices owned by the
 * caller, a leading dimension (elements between rows) for each, every call
 * asynchronous on `stream`, no memory allocated, nothing synchronised,
 * arguments checked on the host before any CUDA call, and on any status other
 * than SGEMM_OK nothing launched.  Elements in the gap between a row's length
 * and its leading dimension are never written.  Any alignment of rows that the
 * element type allows is accepted.  The calls launch kernels only, so after
 * one call on a device they can be captured into a CUDA graph.  Results are
 * the same bits on every run.  (A backward pass over no rows, T == 0, clears the
 * gradients of the weights and the gate by cudaMemsetAsync and cudaMemset2DAsync
 * instead of a kernel.)
 */
#ifndef SGEMM_LAYERS_H
#define SGEMM_LAYERS_H

#include <stddef.h>
#include <stdint.h>

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations, logits and gradients. */
typedef enum {
    SGEMM_F32 = 0,
    SGEMM_BF16 = 1,
    SGEMM_F16 = 2
} sgemm_dtype;

/*
 * Between two blocks of a model, for each of T rows (tokens) of width D:
 *     h = y * rsqrt(mean(y^2) + eps) * w_post     the norm after a block
 *     r = x + scale * gate * h                    gate, residual scale and sum
 *     n = r * rsqrt(mean(r^2) + eps) * w_pre      the norm before the next
 * All of it is computed in FP32 from x and y; r and n are each rounded once,
 * when they are written (n comes from the unrounded r).
 *   dtype: the type of x, y, gate, r and n.
 *   w_pre, w_post: D weights each, of type wdtype (FP32, or the same as
 *       dtype).  w_post == NULL: no norm after the block, h = y.
 *   gate: gate_rows x D, where gate_rows divides T: row t uses gate row
 *       t / (T / gate_rows).  1 row: one gate for every token; T rows: one per
 *       token.  NULL (gate_rows 0): no gate.
 *   r: T x D, may be x itself (same pointer and leading dimension).
 *   n: T x D, or NULL when only the 8-bit form is wanted.
 *   q, q_scale: NULL, or n quantised per row to 8 bits as sgemm_quantize_i8
 *       does it, from the unrounded n.
 *   rstd: 2 x T FP32: rsqrt(mean(y^2) + eps) of each row (1 without w_post),
 *       then rsqrt(mean(r^2) + eps); the backward pass reads them.  May be
 *       NULL.
 * T <= 2^30, D <= 24576.  Without rows or columns (T == 0 or D == 0) nothing is
 * launched and nothing written, rstd and q_scale included.
 */
int sgemm_block_norm(int T, int D, int dtype,
                     const void *x, int ldx, const void *y, int ldy,
                     const void *w_pre, const void *w_post, int wdtype,
                     const void *gate, int ldg, int gate_rows,
                     float scale, float eps,
                     void *r, int ldr, void *n, int ldn,
                     signed char *q, int ldq, float *q_scale,
                     float *rstd, cudaStream_t stream);

/*
 * The gradient of sgemm_block_norm: dn and dr are the gradients of n and r
 * (dr NULL: zero); dx and dy (dtype), dw_pre and dw_post (wdtype) and dgate
 * (dtype, gate_rows x D) are written.  dw_post is needed exactly when w_post
 * is given, dgate exactly when gate is.  rstd is what the forward pass wrote.
 * Sums over rows are FP32, in an order fixed by the shape, and rounded once.
 * dx may be dr or dn, and dy may be dn or dr (same pointer and leading
 * dimension).
 *   workspace: sgemm_block_norm_backward_workspace_size(T, D) bytes, 16-byte
 *       aligned; its contents on entry do not matter.  Calls that share one
 *       must not overlap on the GPU.
 */
int sgemm_block_norm_backward(int T, int D, int dtype,
                              const void *x, int ldx, const void *y, int ldy,
                              const void *w_pre, const void *w_post, int wdtype,
                              const void *gate, int ldg, int gate_rows,
                              float scale, const float *rstd,
                              const void *dn, int lddn, const void *dr, int lddr,
                              void *dx, int lddx, void *dy, int lddy,
                              void *dw_pre, void *dw_post, void *dgate, int lddg,
                              void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes of sgemm_block_norm_backward on the current device (0 if
 * the device cannot be queried or T or D is 0): 16 D for each block, or for
 * narrow rows each warp, that sums over rows, of which an SM holds 1 to 16. */
size_t sgemm_block_norm_backward_workspace_size(int T, int D);

/*
 * Rows quantised to 8-bit integers: for each of M rows of K elements
 *     s = max|x| / 127,   q = rint(x * (127 / max|x|))   in [-127, 127]
 * with FP32 operations each rounded once, so q is defined to the bit.  A row
 * of zeros has s = 0 and q = 0.  A row that holds an infinity or a NaN gets
 * q = 0 and an s that is not finite, so that its products are NaN and not
 * silently wrong.  Serves for activations (a scale per token) and for weights
 * stored N x K (a scale per output channel).
 */
int sgemm_quantize_i8(int M, int K, int dtype, const void *x, int ldx,
                      signed char *q, int ldq, float *s, cudaStream_t stream);

/*
 * C = diag(a_scale) A B^T diag(b_scale) + bias, with A (M x K) and B (N x K,
 * as a linear layer stores its weights) 8-bit integers:
 *     C[m][n] = a_scale[m] * b_scale[n] * sum_k A[m][k] B[n][k] + bias[n]
 * For M <= 4 the sum is an exact integer.  For more rows it is exact while its
 * partial sums stay below 2^24 in magnitude (always for K <= 1024) and an FP32
 * sum otherwise; the scales and the bias are applied in FP32 and the result is
 * rounded once to ctype.
 *   bias: N FP32 values or NULL.  M, N <= 2^30, K <= 131071.
 *   workspace: sgemm_i8_workspace_size(M, N, K, B, ldb) bytes, 16-byte aligned,
 *       with contents that do not matter; calls that share one must not
 *       overlap on the GPU.  M <= 4 and K == 0 need none; rows of B that are not
 *       16-byte aligned need N K bytes of it.
 * K == 0: every sum is empty (C = bias, or 0, whatever the scales).
 * The kernel for more than four rows waits for its own copies, with a limit:
 * one that runs out is reported by sgemm_device_status, and C is unspecified.
 */
int sgemm_i8(int M, int N, int K,
             const signed char *A, int lda, const float *a_scale,
             const signed char *B, int ldb, const float *b_scale,
             const float *bias, void *C, int ldc, int ctype,
             void *workspace, size_t workspace_bytes, cudaStream_t stream);

size_t sgemm_i8_workspace_size(int M, int N, int K, const signed char *B, int ldb);

/*
 * The linear layer with 8-bit weights on activations that are not quantised
 * yet: sgemm_quantize_i8 of the M x K rows of X (xtype), then sgemm_i8.
 */
int sgemm_linear_i8(int M, int N, int K, int xtype, const void *X, int ldx,
                    const signed char *B, int ldb, const float *b_scale,
                    const float *bias, void *C, int ldc, int ctype,
                    void *workspace, size_t workspace_bytes, cudaStream_t stream);

size_t sgemm_linear_i8_workspace_size(int M, int N, int K, const signed char *B, int ldb);

/*
 * For each of T rows of V logits z, the distribution p = softmax(scale * z)
 * over the columns that the mask allows:
 *     lse      = log sum_j exp(scale z_j)
 *     logprob  = scale z_target - lse
 *     entropy  = -sum_j p_j log p_j
 *     top      the `top` most likely columns, most likely first, equal logits
 *              by the lowest column, with their log probabilities
 * read from the logits in one pass.
 *   scale: > 0 and at most 2^127 (one over the temperature).
 *   mask: mask_rows x ceil(V / 32) words, bit j % 32 of word j / 32 set where
 *       column j is allowed; mask_rows is T or 1 (one mask for all rows), ldm
 *       words between rows.  NULL (mask_rows 0): every column is allowed.  What
 *       a masked logit holds (NaN and infinities too) does not matter.
 *   target: T columns.  target < 0: the row is not scored and its logprob is
 *       0.  A target that the mask leaves out has logprob -infinity; one that
 *       is not below V has NaN.
 *   logprob, entropy, lse: T each, FP32; any of them may be NULL (target may be
 *       NULL with logprob).
 *   top: 0 .. 32; top_logprob (FP32) and top_id (32-bit) are T x top, dense.
 *       Columns that cannot occur (masked, or with logit -infinity) are no
 *       alternatives: where fewer than `top` are left, the rest have id -1 and
 *       log probability -infinity.
 * A row without any allowed finite column has lse -infinity, entropy 0 and
 * logprob -infinity.  A row whose allowed logits hold a NaN or +infinity has
 * NaN for all its numbers and -1 for its alternatives.  A row that is not
 * scored has logprob 0 in either case.
 */
int sgemm_logprobs(int T, int V, int dtype, const void *logits, int ldz, float scale,
                   const int32_t *mask, int ldm, int mask_rows, const int64_t *target,
                   float *logprob, float *entropy, float *lse,
                   int top, float *top_logprob, int32_t *top_id, cudaStream_t stream);

/*
 * The gradient of sgemm_logprobs' logprob and entropy with respect to the
 * logits:
 *     dz_j = scale * (g_logprob ([j = target] - p_j) - g_entropy p_j (log p_j + entropy))
 * for the columns that the mask allows, and 0 for the others.
 *   lse, entropy: what the forward pass wrote (entropy may be NULL when
 *       g_entropy is NULL).  g_entropy NULL: no gradient reaches the entropy.
 *       lse is FP32, so beside everything else p_j is off by 2^-24 |lse| relative.
 *       Rows with target < 0 have no gradient from logprob.
 *   dz: T x V, of the logits' type; may be the logits themselves (same pointer
 *       and leading dimension).
 * A row without any allowed finite column has gradient 0; one with a target
 * that is not below V, or whose lse is NaN, has NaN.
 */
int sgemm_logprobs_backward(int T, int V, int dtype, const void *logits, int ldz, float scale,
                            const int32_t *mask, int ldm, int mask_rows, const int64_t *target,
                            const float *lse, const float *entropy,
                            const float *g_logprob, const float *g_entropy,
                            void *dz, int lddz, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif
