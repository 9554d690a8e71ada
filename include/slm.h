/*
 * libsgemm -- matrix products of language models for AMD Instinct MI355X
 * (gfx950), C ABI: products grouped by expert and the rows they take, the softmax cross
 * entropy of an output layer, products with weights held in 4 bits and products in 8-bit
 * integers.
 *
 * The conventions are those of include/sgemm.h: row-major matrices, element
 * (r, c) of a matrix with leading dimension ld at index r*ld + c; device
 * pointers on the current HIP device, owned by the caller; the calls queue
 * kernels on `stream` and return, and allocate, free, copy and synchronise
 * nothing, so they may be captured into a HIP graph.  Outputs must not
 * overlap inputs.  Argument errors are returned as -p (p counts the first
 * parameter as 1) before any HIP call, but for a workspace that is too small: the
 * size that it needs depends on the current device, which is asked for its compute
 * units first.  A positive value is the hipError_t of a failed HIP call.  The calls are re-entrant: they share no state but a
 * per-device cache of the compute-unit count, and workspaces are the
 * caller's, one per call in flight (also one per captured graph that may run
 * beside another).
 *
 * Extents are at most 2^31 - 1025.  A product of more than 2^24 - 1 tiles is
 * answered with hipErrorInvalidConfiguration.
 *
 * Types.  Matrices hold fp32 or bf16 values (one type per call); every sum is
 * held in fp32, and a bf16 result is rounded once, to nearest even.
 * Pointers need the alignment of their element.  Rows at 4-byte addresses
 * (always so for fp32) are loaded straight to LDS; bf16 operands with an odd leading
 * dimension, group stride or address go through registers, more slowly.
 */
#ifndef LIBSGEMM_SLM_H
#define LIBSGEMM_SLM_H

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum sgemm_type { SGEMM_TYPE_F32 = 0, SGEMM_TYPE_BF16 = 1 };

/*
 * sgemm_grouped -- for each group e, on its rows r = offsets[e] ..
 * offsets[e+1] - 1:
 *     Y[r] <- alpha * X[r] * W_e + beta * Y[r]
 *
 *   type      enum sgemm_type of X, W and Y
 *   trans     0: W_e is K x N, W_e(k, n) at W[e*stride_w + k*ldw + n];
 *             1: W_e is N x K, stored transposed, at W[e*stride_w + n*ldw + k]
 *   groups    number of groups E >= 0 (a group without rows reads no weights)
 *   rows      rows of X and Y, >= 0
 *   N, K      >= 0
 *   X, ldx    rows x K, ldx >= max(1, K)
 *   W, ldw, stride_w   ldw >= max(1, trans ? K : N); stride_w elements from
 *             one group's weights to the next (>= 0)
 *   beta      beta == 0: Y is written, not read
 *   Y, ldy    rows x N, ldy >= max(1, N)
 *   offsets   groups + 1 ints on the device, in increasing order within
 *             [0, rows].  Rows before offsets[0] and from offsets[groups] on
 *             are left as they were.  The host does not read the offsets: a
 *             value outside [0, rows] is taken as the nearest inside, and a
 *             group that ends before it begins has no rows; where groups
 *             overlap, what their rows of Y hold is not defined.
 *
 * The gradient of X is the same call with X and Y exchanged and `trans`
 * flipped: dX <- dY * W_e^T.
 *
 * alpha == 0 or K == 0: Y <- beta*Y, X and W are not read.
 * Returns -1 type, -2 trans, -3 groups < 0, -4 rows < 0, -5 N < 0 (or more
 * than 2^31 - 1 tiles), -6 K < 0, -8 X NULL (while it is read) or not aligned
 * to its type, -9 ldx, -10 W likewise, -11 ldw, -12 stride_w < 0, -14 Y, -15
 * ldy, -16 offsets NULL or not 4-byte aligned.
 *
 * Accuracy: fp32 sums of products that are exact (bf16) or fp32 (fp32), in
 * one order for given sizes: results repeat bit for bit.
 */
int sgemm_grouped(int type, int trans, int groups, int rows, int N, int K, float alpha,
                  const void *X, int ldx, const void *W, int ldw, int64_t stride_w, float beta,
                  void *Y, int ldy, const int *offsets, hipStream_t stream);

/*
 * sgemm_grouped_wgrad -- the gradient of grouped weights: for each group e,
 *     D_e <- alpha * sum over its rows r of X[r]^T * G[r] + beta * D_e
 *
 *   X, ldx    rows x M, ldx >= max(1, M)
 *   G, ldg    rows x N, ldg >= max(1, N)
 *   D, ldd, stride_d   D_e is M x N, at D[e*stride_d + m*ldd + n]; no two groups'
 *             share an element (they follow one another, or lie side by side
 *             in rows of all groups)
 * A group without rows gets D_e <- beta*D_e.  For weights stored K x N, X is
 * the product's input and G the gradient of its output (M = K); for weights
 * stored N x K, exchange the two.  Types, offsets, alpha and beta as in
 * sgemm_grouped.
 * Returns -1 type, -2 groups < 0, -3 rows < 0, -4 M < 0, -5 N < 0 (or more
 * than 2^31 - 1 tiles), -7 X, -8 ldx, -9 G, -10 ldg, -12 D, -13 ldd, -14
 * stride_d < 0 or outputs that overlap, -15 offsets.
 */
int sgemm_grouped_wgrad(int type, int groups, int rows, int M, int N, float alpha, const void *X,
                        int ldx, const void *G, int ldg, float beta, void *D, int ldd,
                        int64_t stride_d, const int *offsets, hipStream_t stream);

/*
 * sgemm_xent -- softmax cross entropy of an output layer.  With the logits
 * z[t][v] = sum_k X[t][k] W[v][k]:
 *     lse[t]  = log(sum_v exp(z[t][v]))
 *     loss[t] = lse[t] - z[t][targets[t]]
 * without keeping the logits: tiles of them are reduced to a maximum and a sum
 * of exponentials per row.  Finite logits have to lie below 2^126 in magnitude.  The
 * loss is never below 0, and its roundings are relative to the target's distance
 * from the row's largest logit, not to lse.
 *
 *   rows, vocab, K   >= 0 (rows tokens, K hidden values; vocab >= 1 if rows > 0)
 *   X, ldx    rows x K of `type`;  W, ldw: vocab x K of `type`
 *   targets   rows int64; a value outside [0, vocab) marks a row that does
 *             not count: its loss is 0 (its lse is computed all the same)
 *   loss, lse rows floats each
 *   ws, ws_bytes   workspace, 16-byte aligned, of at least
 *             sgemm_xent_workspace(type, rows, vocab, K, 0) bytes
 *
 * Returns -1 type, -2 rows < 0, -3 vocab (< 0, 0 with rows, or too many
 * tiles), -4 K < 0, -5 X, -6 ldx, -7 W, -8 ldw, -9 targets (NULL or not 8-byte
 * aligned), -10 loss, -11 lse, -12 ws (NULL or not 16-byte aligned), -13
 * ws_bytes too small.
 */
int sgemm_xent(int type, int rows, int vocab, int K, const void *X, int ldx, const void *W, int ldw,
               const int64_t *targets, float *loss, float *lse, void *ws, int64_t ws_bytes,
               hipStream_t stream);

/*
 * sgemm_xent_backward -- gradients of sum_t dloss[t] * loss[t]: with
 *     d[t][v] = dloss[t] * (exp(z[t][v] - lse[t]) - [v == targets[t]])
 * (0 in rows that do not count, whatever z holds):
 *     dX[t][k] = sum_v d[t][v] W[v][k]      dW[v][k] = sum_t d[t][v] X[t][k]
 * The logits are computed again, a piece of the vocabulary at a time; d is
 * held in `type` for one piece (bf16 rounds each d once, by at most 2^-8 of
 * itself, as a stored gradient of that type would; with up to 128 rows what that leaves
 * over is kept beside it, so that d has 16 bits), and both products sum in fp32 over
 * all pieces.  These roundings need not average out: with the same dloss in every
 * row, the derivatives at the targets, all close to -dloss, round the same way.  A row that does not count adds 0 *
 * X[t][k] to dW: X must be finite there.
 *
 *   lse       as sgemm_xent gave it (its rounding, 2^-24 of lse, is one of
 *             every exp(z - lse))
 *   dloss     rows floats, the gradient of each row's loss
 *   dX, lddx  rows x K of `type`, or NULL: not computed
 *   dW, lddw  vocab x K of `type`, or NULL: not computed
 *   ws, ws_bytes   as above, sgemm_xent_workspace(type, rows, vocab, K, 1)
 *
 * Returns -1 .. -9 as sgemm_xent, -10 lse, -11 dloss, -12 dX, -13 lddx, -14
 * dW, -15 lddw, -16 ws, -17 ws_bytes.
 */
int sgemm_xent_backward(int type, int rows, int vocab, int K, const void *X, int ldx, const void *W,
                        int ldw, const int64_t *targets, const float *lse, const float *dloss,
                        void *dX, int lddx, void *dW, int lddw, void *ws, int64_t ws_bytes,
                        hipStream_t stream);

/* Bytes of workspace for sgemm_xent (backward 0) or sgemm_xent_backward
 * (backward 1) on the current device; -1 .. -4 for invalid sizes, -5 for
 * another `backward`. */
int64_t sgemm_xent_workspace(int type, int rows, int vocab, int K, int backward);

/*
 * sgemm_q4_matvec -- rows times weights held in 4 bits: for each group e, on
 * its rows r,
 *     Y[r][n] <- sum_k X[r][k] * (q_e[n][k] - z_e[n][b]) * s_e[n][b],  b = k / block
 * One pass over the weights serves up to 64 bf16 or 24 fp32 rows together (with
 * offsets, no more than twice a group's mean), so this is meant for single tokens and
 * short batches; any number of rows is computed, in passes of so many.
 *
 *   type      enum sgemm_type of X, S and Y
 *   groups    sets of weights (1 when offsets is NULL), at most 65535
 *   rows, N, K   K even, at most 2^27
 *   block     weights along K that share a scale and a zero: 32, 64 or 128; the
 *             last block of a row may be short
 *   X, ldx    rows x K
 *   Q         groups x N x K/2 bytes, packed: weight k of a row is the low (k
 *             even) or high (k odd) four bits of byte k/2, 0 .. 15
 *   S         groups x N x ceil(K/block) scales, packed
 *   Z         as many zeros, one byte each (0 .. 15), or NULL: 8 everywhere
 *   Y, ldy    rows x N, written
 *   offsets   groups + 1 ints on the device, as in sgemm_grouped (rows outside
 *             every group are left as they were), or NULL: all rows, one group
 *
 * Returns -1 type, -2 groups, -3 rows < 0, -4 N < 0, -5 K < 0 or odd, -6 block,
 * -7 X, -8 ldx, -9 Q, -10 S, -12 Y, -13 ldy, -14 offsets not 4-byte aligned.
 *
 * Accuracy: fp32 rows keep their 24 bits (they are multiplied as three exact
 * bf16 parts; of values below 2^-110 in magnitude what lies under 2^-133 is lost);
 * with w the dequantised weights, sums are within about
 * 4 K 2^-24 sum_b |s| sum_k (16 + q) |x| of the exact value.  A row that holds an
 * infinity, a NaN, or a value beyond 2^118 in magnitude may come out as NaN.
 */
int sgemm_q4_matvec(int type, int groups, int rows, int N, int K, int block, const void *X, int ldx,
                    const uint8_t *Q, const void *S, const uint8_t *Z, void *Y, int ldy,
                    const int *offsets, hipStream_t stream);

/*
 * sgemm_q4_quantize -- the nearest weights of that form to W (N x K of `type`,
 * values below 2^127 in magnitude): per block, with Z: scale (max(w, 0) - min(w, 0)) / 15 and the
 * zero that makes the smallest weight 0; without (Z NULL): scale max|w| / 7
 * around 8.  The scale is rounded to `type` first; q is the nearest integer to w / scale
 * (ties to even), plus the zero, clamped to 0 .. 15.  A block whose scale
 * rounds to zero reads back as zeros.
 * Returns -1 type, -2 N < 0, -3 K < 0 or odd, -4 block, -5 W, -6 ldw, -7 Q, -8 S.
 */
int sgemm_q4_quantize(int type, int N, int K, int block, const void *W, int ldw, uint8_t *Q,
                      void *S, uint8_t *Z, hipStream_t stream);

/*
 * Rows sorted by expert, and back.  `tokens` tokens choose k experts each; slot
 * s = t * k + j is token t's choice j.
 *
 * sgemm_expert_sort -- the rows that grouped products take: a slot whose expert lies in
 * [0, groups) gets a row, by expert and, within one, by slot (a stable sort); a slot
 * whose expert lies outside is dropped, and stands behind them all, again by slot.
 *
 *   slots     tokens * k, >= 0
 *   groups    number of experts, 0 .. 4096
 *   experts   slots int64
 *   offsets   groups + 1 ints: expert e has rows offsets[e] .. offsets[e+1] - 1
 *   order     slots ints: the slot of each row, those dropped last; or NULL
 *   place     slots ints: each slot's row r; -2 - r where it is dropped (r is then one of
 *             the rows from offsets[groups] on, which no expert has)
 *   ws, ws_bytes   workspace, 16-byte aligned, of at least
 *             sgemm_expert_sort_workspace(slots, groups) bytes (NULL where that is 0)
 * Returns -1 slots, -2 groups, -3 experts (NULL with slots, or not 8-byte aligned), -4
 * offsets (NULL or not 4-byte aligned), -5 order, -6 place, -7 ws, -8 ws_bytes too small.
 */
int sgemm_expert_sort(int slots, int groups, const int64_t *experts, int *offsets, int *order,
                      int *place, void *ws, int64_t ws_bytes, hipStream_t stream);

/* Bytes of workspace for sgemm_expert_sort; -1, -2 for invalid sizes. */
int64_t sgemm_expert_sort_workspace(int slots, int groups);

/*
 * sgemm_expert_gather -- tokens to their rows: with r = place[t*k + j],
 *     R[r] <- weights[t*k + j] * X[t]
 * The products are fp32, rounded once to `type`; without weights rows are copied bit for bit.
 *
 *   type      enum sgemm_type of X and R
 *   tokens, k, H   >= 0; tokens * k at most 2^31 - 1025
 *   X, ldx    tokens x H, ldx >= max(1, H)
 *   place     tokens * k ints, as sgemm_expert_sort gives them.  Rows are taken where 0 <=
 *             r < rows; -1 means no row, and any other value is left out as well.  No
 *             two places are the same (what a row that is named twice holds is not defined)
 *   weights   tokens * k floats, or NULL: 1
 *   rows      rows of R, >= 0
 *   R, ldr    rows x H, ldr >= max(1, H)
 *   fill      0: rows without a token are left as they were; 1: the rows r of dropped
 *             slots (place -2 - r) are set to zero, so that with rows = tokens * k all
 *             of R is written
 * The gradient by X is sgemm_expert_combine of the gradient by R; that by the weights is
 * sgemm_expert_combine_backward's with X as dout and the gradient by R as R.
 * Returns -1 type, -2 tokens, -3 k (or tokens * k too large), -4 H, -5 X, -6 ldx, -7
 * place, -8 weights, -9 rows, -10 R, -11 ldr, -12 fill.
 */
int sgemm_expert_gather(int type, int tokens, int k, int H, const void *X, int ldx,
                        const int *place, const float *weights, int rows, void *R, int ldr,
                        int fill, hipStream_t stream);

/*
 * sgemm_expert_combine -- rows back to tokens:
 *     out[t] <- beta * out[t] + sum_j weights[t*k + j] * R[place[t*k + j]]
 * summed in fp32 in the order of j, rounded once.  A slot without a row adds nothing and
 * its weight is not used; a token with none gets beta * out[t].  One row may serve several slots.
 * (bf16 rows were rounded before the sum: fp32 rows, as sgemm_q8_gemm gives them too, leave one
 * rounding, of the fp32 result.)
 *
 *   R, ldr    rows x H of `type`;  place, weights as above
 *   beta      beta == 0: out is written, not read
 *   out, ldo  tokens x H, ldo >= max(1, H)
 * Returns -1 type, -2 tokens, -3 k, -4 H, -5 rows, -6 R, -7 ldr, -8 place, -9 weights,
 * -11 out, -12 ldo.
 */
int sgemm_expert_combine(int type, int tokens, int k, int H, int rows, const void *R, int ldr,
                         const int *place, const float *weights, float beta, void *out, int ldo,
                         hipStream_t stream);

/*
 * sgemm_expert_combine_backward -- gradients of sum_t <dout[t], out[t]>:
 *     dR[place[s]] <- weights[s] * dout[t]        dweights[s] <- <dout[t], R[place[s]]>
 * A slot without a row gets dweights 0.  The dot products are fp32 sums, in one order for
 * given sizes: results repeat bit for bit.
 *
 *   dout, lddo   tokens x H of `type`
 *   R, ldr    as the forward pass had it; not read where dweights is NULL
 *   weights   tokens * k floats, or NULL: 1
 *   dR, lddr  rows x H of `type`, or NULL: not computed.  No two places are the same then: a row
 *             that serves several slots gets one of their gradients, not the sum.  fill as in
 *             sgemm_expert_gather
 *   dweights  tokens * k floats, or NULL: not computed
 * Returns -1 type, -2 tokens, -3 k, -4 H, -5 rows, -6 dout, -7 lddo, -8 R, -9 ldr, -10
 * place, -11 weights, -12 dR, -13 lddr, -14 fill, -15 dweights.
 */
int sgemm_expert_combine_backward(int type, int tokens, int k, int H, int rows, const void *dout,
                                  int lddo, const void *R, int ldr, const int *place,
                                  const float *weights, void *dR, int lddr, int fill,
                                  float *dweights, hipStream_t stream);

/*
 * Products in 8-bit integers, with a scale for each row of X (token) and each column of Y
 * (channel): the value of q is q times its scale.
 *
 * sgemm_q8_quantize -- rows to 8 bits: with m the largest magnitude of row r of X,
 *     scales[r] = m * (1 / 127)        Q[r][k] = X[r][k] / scales[r]
 * (the scale in fp32, 1 / 127 and the product rounded to it once each: m / 127 or its neighbour); Q
 * rounded to the nearest integer, ties to even, of the exact quotient of the stored values.
 * A row whose scale is zero gets zeros; a row that holds an infinity or a NaN gets
 * the scale NaN and zeros, so that its products are NaN.  Weights are quantised by the same call (N x K: a
 * scale for each output channel).
 *
 *   type      enum sgemm_type of X
 *   rows      >= 0;  K 0 .. 131071;  X, ldx: rows x K
 *   k, place  NULL place and k 0: row r of X goes to row r of Q, out_rows = rows.  Otherwise
 *             row t goes to the k rows place[t*k + j], as sgemm_expert_gather sends them
 *             (rows without a token: left as they were, but those of dropped slots set
 *             to zero, with the scale 0); NULL too where rows is 0
 *   out_rows  rows of Q and scales
 *   Q, ldq    out_rows x K bytes, ldq >= max(1, K).  The products read rows at 4-byte
 *             addresses (Q and ldq multiples of 4) fastest
 *   scales    out_rows floats
 * Returns -1 type, -2 rows, -3 K, -4 X, -5 ldx, -6 k (negative, rows * k too large, or not
 * 0 without place for rows), -7 place, -8 out_rows, -9 Q, -10 ldq, -11 scales.
 */
int sgemm_q8_quantize(int type, int rows, int K, const void *X, int ldx, int k, const int *place,
                      int out_rows, int8_t *Q, int ldq, float *scales, hipStream_t stream);

/*
 * sgemm_q8_gemm -- for each group e, on its rows r = offsets[e] .. offsets[e+1] - 1,
 *     Y[r][n] <- (sum_k X[r][k] * W_e[n][k]) * x_scales[r] * w_scales[e][n]
 * The sums are exact (32-bit integers); they become fp32, are multiplied by the row's scale
 * and then the column's, and rounded to `type`.
 *
 *   type      enum sgemm_type of Y
 *   groups    sets of weights (1 when offsets is NULL)
 *   rows, N   >= 0;  K 0 .. 131071, which no sum of products of bytes overflows at
 *   X, ldx    rows x K bytes;  x_scales: rows floats
 *   W, ldw, stride_w   N x K bytes a group, ldw >= max(1, K), stride_w >= 0 bytes from one
 *             group to the next;  w_scales: groups x N floats, packed
 *   Y, ldy    rows x N, written
 *   offsets   groups + 1 ints on the device, as in sgemm_grouped, or NULL: all rows, one group
 *   fill      with offsets: 0: rows before offsets[0] and from offsets[groups] on are left as they
 *             were; 1: they are set to zero
 * X and W at 4-byte addresses with leading dimensions (and stride_w) of multiples of 4 are
 * loaded straight to LDS; others go through registers, 1.1 to 2.5 times as slowly.
 * Returns -1 type, -2 groups, -3 rows, -4 N (or rows and N of more than 2^24 - 1 tiles of 256 x 256,
 * of 128 x 128 where they go through registers; each group may add one to its rows' tiles), -5 K, -6 X, -7
 * ldx, -8 x_scales, -9 W, -10 ldw, -11 stride_w, -12 w_scales, -13 Y, -14 ldy, -15 offsets
 * not 4-byte aligned, -16 fill.
 */
int sgemm_q8_gemm(int type, int groups, int rows, int N, int K, const int8_t *X, int ldx,
                  const float *x_scales, const int8_t *W, int ldw, int64_t stride_w,
                  const float *w_scales, void *Y, int ldy, const int *offsets, int fill,
                  hipStream_t stream);

/*
 * sgemm_q8_matvec -- sgemm_q8_quantize and sgemm_q8_gemm in one launch, for a few rows of X:
 * every workgroup quantises them for itself.  One pass over the weights serves up to 16 rows
 * (fewer where K is above 6656: 104 KB of quantised rows), so this is meant for single tokens and
 * short batches; any number of rows is computed, in passes of so many.  Results
 * are those of the two calls bit for bit.
 *
 *   type      enum sgemm_type of X and Y
 *   groups, fill   as in sgemm_q8_gemm, groups at most 65535;  K at most 106496
 * Returns -1 type, -2 groups, -3 rows, -4 N, -5 K, -6 X, -7 ldx, -8 W, -9 ldw, -10
 * stride_w, -11 w_scales, -12 Y, -13 ldy, -14 offsets not 4-byte aligned, -15
 * fill.
 */
int sgemm_q8_matvec(int type, int groups, int rows, int N, int K, const void *X, int ldx,
                    const int8_t *W, int ldw, int64_t stride_w, const float *w_scales, void *Y,
                    int ldy, const int *offsets, int fill, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_SLM_H */
