/*
 * libsgemm -- the operators of a language model that sit around its matrix
 * products, on one NVIDIA GB300 (sm_103a): the norms, gate and residual sum
 * between two blocks, the products with 8-bit and 4-bit weights, and the log
 * probabilities, or the steps of beam search, that the last product's logits
 * are turned into.
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
 * gradients of the weights, the bias and the gate by cudaMemsetAsync and
 * cudaMemset2DAsync instead of a kernel; rows of no columns quantised to 4 bits
 * have their scales cleared so.)
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
 * The norm of rows about their mean, of T rows of width D, after an optional sum:
 *     r = x + add                                  (r = x without add)
 *     n = (r - mean) rstd w + b,   mean = mean(r), rstd = rsqrt(mean((r - mean)^2) + eps)
 * The sum is rounded to dtype, once, and what is normalised is the r that is written,
 * so the backward pass needs r alone; everything else is FP32, and n is rounded once.
 * The squares are summed about means of parts of the row, so no difference of large numbers
 * is taken for the deviation; the mean is an FP32 sum, off by up to about 50 2^-24 of the row's
 * mean magnitude, which shifts the whole row.
 *   dtype: the type of x, add, r and n.  r is needed exactly when add is given; it may be
 *       x or add (same pointer and leading dimension).
 *   w, b: D weights each, of type wdtype (FP32, or the same as dtype); b may be NULL (0).
 *   stats: 2 x T FP32, the means, then the rstd of all rows, for the backward pass.  May be
 *       NULL.
 * T <= 2^30, D <= 24576.  Without rows or columns nothing is launched and nothing written.
 */
int sgemm_layer_norm(int T, int D, int dtype,
                     const void *x, int ldx, const void *add, int lda,
                     const void *w, const void *b, int wdtype, float eps,
                     void *r, int ldr, void *n, int ldn, float *stats, cudaStream_t stream);

/*
 * The gradient of sgemm_layer_norm with respect to r, whose gradient add and the forward
 * pass's x share, to w and to b.  With h = (x - mean) rstd and u = dn w, of each row:
 *     dx = dr + rstd (u - mean(u) - h mean(u h)),   dw = sum dn h,   db = sum dn
 *   x: the r of the forward pass (its x, where nothing was added).  stats: what the forward
 *       pass wrote.  dn, dr: the gradients of n and of r (dr NULL: zero).
 *   dx (dtype) may be dn, dr or x (same pointer and leading dimension); dw and db have
 *       type wdtype; db NULL: not wanted.
 * Sums over rows are FP32, in an order fixed by the shape, and rounded once.
 *   workspace: sgemm_layer_norm_backward_workspace_size(T, D) bytes, 16-byte aligned; its
 *       contents on entry do not matter.  Calls that share one must not overlap on the
 *       GPU.
 * Over no rows (T == 0) dw and db are cleared.
 */
int sgemm_layer_norm_backward(int T, int D, int dtype,
                              const void *x, int ldx, const void *w, int wdtype, const float *stats,
                              const void *dn, int lddn, const void *dr, int lddr,
                              void *dx, int lddx, void *dw, void *db,
                              void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes of sgemm_layer_norm_backward on the current device (0 if the device
 * cannot be queried or T or D is 0): 8 D for each block that sums over rows, of which an SM
 * holds 1 to 16, for the type and alignment that has the most. */
size_t sgemm_layer_norm_backward_workspace_size(int T, int D);

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

/*
 * Rows quantised to 4-bit floating point.  A code is a sign bit and three bits
 * for 0, 0.5, 1, 1.5, 2, 3, 4, 6 (e2m1); `block` columns share a scale:
 *   block 16: each row has a scale S = max|row| / 2688 (FP32), each block one of
 *       8 bits, s = e4m3(max|y| / 6) with y = x (2688 / max|row|); the codes are
 *       e2m1(y (1 / s)), and a column stands for code * s * S.
 *   block 32: each block has a power of two, s = the smallest with
 *       max|x| / s <= 6, as its exponent + 127 in 8 bits (e8m0); the codes are
 *       e2m1(x / s), a column stands for code * s, and there is no row scale
 *       (scale is NULL).  (The microscaling formats' own rule, the exponent of the largest
 *       less 2, would let magnitudes above 6 s saturate; the products take scales of
 *       either rule.)
 * All by FP32 operations each rounded once (1 / 6 is the FP32 number next to it), to
 * nearest with ties to even, so codes and scales are defined to the bit.  Blocks whose
 * scale comes out as 0 have codes 0.  A row (block 16), or a block (block 32), that
 * holds an infinity or a NaN gets codes 0 and a scale that is not finite, so that its
 * products are NaN and not silently wrong.
 *   q: M x ceil(K / 2) bytes, ldq bytes between rows: column k in the low half of
 *       byte k / 2 where k is even, in the high half where it is odd; the half
 *       behind an odd K is 0.  q must be 16-byte aligned and ldq a multiple of
 *       16, here and in the products.
 *   block_scale: sgemm_fp4_scales_size(M, K, block) bytes, 16-byte aligned: the
 *       blocks' scales in tiles of 128 rows by 4 blocks.  The scale of row r and
 *       block j is byte 16 (r % 32) + 4 (r / 32 % 4) + j % 4 of the 512 of tile
 *       (r / 128, j / 4); tiles of the same rows follow each other.  Scales of
 *       blocks and rows behind the matrix are 0.
 *   scale: M FP32 values (block 16).
 * M <= 2^30, K <= 2^24.  Serves for activations and for weights stored N x K.
 */
int sgemm_quantize_fp4(int M, int K, int dtype, const void *x, int ldx, int block,
                       unsigned char *q, int ldq, unsigned char *block_scale, float *scale,
                       cudaStream_t stream);

/* Bytes of the tiles that hold the blocks' scales of rows x K columns. */
size_t sgemm_fp4_scales_size(int rows, int K, int block);

/*
 * Block scales from rows of plain bytes (s: rows x ceil(K / block), lds between
 * rows) to tiles, for weights that were quantised elsewhere.
 */
int sgemm_fp4_lay_out_scales(int rows, int K, int block, const unsigned char *s, int lds,
                             unsigned char *tiles, cudaStream_t stream);

/*
 * C = A B^T + bias for the matrices that codes and scales stand for (A: M x K, B:
 * N x K, both quantised with the same block, as sgemm_quantize_fp4 lays them out):
 * the products of codes and the blocks' scales are exact, the sums over K are FP32, in
 * an order fixed by the shape; the rows' scales and the bias are applied in FP32 and the
 * result is rounded once to ctype.
 *   a_scale, b_scale: M and N FP32 values, or NULL (1).  Beside weights that were
 *       quantised elsewhere b_scale can hold whatever scale they have beyond their
 *       blocks', repeated for each row.
 *   bias: N FP32 values or NULL.  M, N <= 2^30, K <= 2^24.
 *   Scales of rows behind the matrix do not matter; those of blocks behind K must be
 *   finite.
 * K == 0: every sum is empty (C = bias, or 0, whatever the scales).
 * The kernel waits for its own copies, with a limit: one that runs out is reported by
 * sgemm_device_status, and C is unspecified.
 */
int sgemm_fp4(int M, int N, int K, int block,
              const unsigned char *A, int lda, const unsigned char *a_block, const float *a_scale,
              const unsigned char *B, int ldb, const unsigned char *b_block, const float *b_scale,
              const float *bias, void *C, int ldc, int ctype, cudaStream_t stream);

/*
 * The linear layer with 4-bit weights on activations that are not quantised yet:
 * sgemm_quantize_fp4 of the M x K rows of X (xtype), then sgemm_fp4.
 *   workspace: sgemm_linear_fp4_workspace_size(M, K, block) bytes, 16-byte aligned,
 *       with contents that do not matter; calls that share one must not overlap on
 *       the GPU.  One row of up to 90112 columns needs none.
 */
int sgemm_linear_fp4(int M, int N, int K, int xtype, const void *X, int ldx, int block,
                     const unsigned char *B, int ldb, const unsigned char *b_block, const float *b_scale,
                     const float *bias, void *C, int ldc, int ctype,
                     void *workspace, size_t workspace_bytes, cudaStream_t stream);

size_t sgemm_linear_fp4_workspace_size(int M, int K, int block);

/*
 * A step of beam search.  B groups of W beams each have logits over V columns (row
 * b W + w is beam w of group b) and a score, their log probability so far.  Of each
 * group's W V continuations, whose score is
 *     score[b][w] + log softmax(scale * logits)[column]        (over the columns that the
 *                                                               mask allows)
 * the `top` best are written, best first: their scores, their beams (0 .. W - 1) and their
 * columns.  Equal scores go by the lower beam, then the lower column.  The scores are
 * compared in 64 bits (those of one beam by their logits) and rounded once when they are
 * written; they come from FP32 sums, whose order, and so their last bit, depends on where in
 * 16 bytes a row starts.  The only continuation of a beam has the beam's score, exactly.
 *   logits, scale, mask: as in sgemm_logprobs.  score: B x W, dense.
 *   finished: B x W bytes or NULL.  A beam whose byte is not 0 has one continuation, the
 *       column `end` (>= 0) with the score it has; its logits are not read.
 *   A beam whose score is not finite takes no part (a beam that does not exist has
 *   -infinity), nor does one whose allowed logits hold a NaN or +infinity, or are all
 *   -infinity.  Columns that cannot occur are no continuations.  Where fewer than `top`
 *   are left, the rest have score -infinity, beam -1 and column -1.
 *   out_score (FP32), parent, token (32-bit): B x top, dense.
 *   workspace: sgemm_beam_step_workspace_size(B, W, top) bytes, 16-byte aligned; contents on
 *       entry do not matter.  Calls that share one must not overlap on the GPU.
 * W, top: 1 .. 32.  B W <= 2^30.
 */
int sgemm_beam_step(int B, int W, int V, int dtype, const void *logits, int ldz, float scale,
                    const int32_t *mask, int ldm, int mask_rows,
                    const float *score, const unsigned char *finished, int end,
                    int top, float *out_score, int32_t *parent, int32_t *token,
                    void *workspace, size_t workspace_bytes, cudaStream_t stream);

size_t sgemm_beam_step_workspace_size(int B, int W, int top);

/*
 * Rows of states reordered as beams were chosen: row b top + k of out becomes row
 * b W + parent[b][k] of in, for B groups.  A row is `outer` runs of `inner` bytes, in_outer
 * (out_outer) bytes apart; rows are in_row (out_row) bytes apart.  A row whose parent is
 * not 0 .. W - 1 is left as it is.
 *   out may be in (same pointer and strides, top == W): each row then becomes what its
 *       parent was before the call, and rows that are their own parent are neither read
 *       nor written for themselves.
 *   Rows of out must not overlap each other.  All sizes and strides are bytes, at most 2^44
 *   in all; any alignment is accepted (16 bytes at a time where all allow it).
 */
int sgemm_beam_reorder(int B, int W, int top, int64_t outer, int64_t inner,
                       const void *in, int64_t in_row, int64_t in_outer,
                       const int32_t *parent, void *out, int64_t out_row, int64_t out_outer,
                       cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif
