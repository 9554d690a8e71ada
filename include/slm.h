/*
 * libsgemm -- matrix products of language models for AMD Instinct MI355X
 * (gfx950), C ABI: products grouped by expert, the softmax cross entropy of an
 * output layer, and products with weights held in 4 bits.
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

#ifdef __cplusplus
}
#endif

#endif /* LIBSGEMM_SLM_H */
