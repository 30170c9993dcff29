/*
 * libgemm355: operators on rows of logits -- row-wise softmax and row sum (binary32), the
 * softmax cross entropy of a projection with its gradient, and routing to experts with its
 * gradient (binary32, binary16, bfloat16).
 *
 * "Kernel optimisation guide" (section on softmax optimisation, the online algorithm)
 * computes the softmax of a vector in one pass for its statistics: a running maximum m
 * and a running sum l of exp(x - m), the sum rescaled by exp(m_old - m_new) whenever the
 * maximum rises, followed by a pass that writes exp(x_i - m) / l.  Its section on
 * warp-shuffle reduction sums a value over the lanes of a warp by exchanging registers
 * between lanes.  These entry points apply both to every row of a matrix on the GPU:
 * each row is held on chip while its statistics are reduced across the 64 lanes of a
 * wave and across the waves of a workgroup, so it is read from memory once (rows of
 * more than 32768 elements are read twice).
 *
 * Layout: X and Y are rows x cols, row-major, row strides ldx and ldy in elements
 * (element (r, c) at X[r * ldx + c]).  All pointers are device pointers owned by the
 * caller; work is enqueued on `stream` and the call returns at once.  Nothing is
 * allocated.
 *
 * Errors: argument errors are detected on the host before any HIP call and return
 * GEMM355_ERR_INVALID_ARG; a current device that is not a gfx950 returns
 * GEMM355_ERR_DEVICE; a failed launch returns GEMM355_ERR_LAUNCH.
 */
#ifndef GEMM355_SOFTMAX_H
#define GEMM355_SOFTMAX_H

#include <stddef.h>

#include "gemm355.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Y[r][c] = exp(X[r][c] - m_r) / l_r for every 0 <= r < rows, 0 <= c < cols, with
 * m_r = max_c X[r][c] and l_r = sum_c exp(X[r][c] - m_r) (the online softmax above).
 *
 * Results agree with the exact softmax of the binary32 inputs to a relative error below
 * 2^-24 (2 |X[r][c] - m_r| + 2 n + 64), n the number of elements one lane sums in
 * sequence (at most 64 for rows of up to 32768 elements, cols / 1024 beyond): the
 * rounding of X - m dominates for elements far below the maximum.  Inputs are expected finite; an infinity or NaN in a row makes
 * that row's results unspecified (other rows are unaffected).
 *
 * Arguments: 0 <= rows <= 2^30, 0 <= cols <= 2^30; ldx >= max(1, cols), ldy >= max(1, cols);
 * X and Y non-null unless rows * cols == 0; Y may equal X (in place) when ldy == ldx,
 * any other overlap of the two matrices' spans is an argument error.  rows == 0 or
 * cols == 0 is a no-op.  Elements of Y outside the rows x cols region are not written. */
gemm355_status gemm355_softmax_f32(int rows, int cols, const float *X, int ldx, float *Y,
                                   int ldy, hipStream_t stream);

/* out[r] = sum_c X[r][c] for every 0 <= r < rows (cols == 0 gives +0.0).  The lanes'
 * partial sums are combined by register exchanges within each wave, then across the
 * wave's workgroup, in a fixed order, so repeated calls give identical bits; the result
 * agrees with the exact sum to within about (cols / (64 * waves per row) + 12) * 2^-24
 * times the sum of the magnitudes (sums of small integers are exact).
 *
 * Arguments: 0 <= rows <= 2^30, 0 <= cols <= 2^30, ldx >= max(1, cols); X non-null unless
 * rows * cols == 0; out (rows binary32 values) non-null unless rows == 0, and not
 * overlapping X's span. */
gemm355_status gemm355_row_sum_f32(int rows, int cols, const float *X, int ldx, float *out,
                                   hipStream_t stream);

/*
 * Softmax cross entropy over a large vocabulary.
 *
 * Z = X.op(W) holds the logits of M rows (tokens) over N classes (the vocabulary), X an
 * M x K matrix of hidden rows and W the head's weights, K x N, or N x K with
 * GEMM355_TRANS_B (the only flag taken).  X and W are of type `dtype` (gemm355_dtype); the
 * products are exact and summed in binary32, as in the GEMM entry points.  Per row t, with
 * label y_t:
 *
 *     lse_t  = log sum_v exp(Z[t][v])           (the online softmax above)
 *     loss_t = lse_t - Z[t][y_t]
 *
 * Z is never stored whole: statistics are taken from pieces of the vocabulary.  A row
 * with y_t == ignore has loss 0 and no gradient (its lse is written as any other).  A
 * label that is neither `ignore` nor in [0, N) has loss NaN and no gradient; nothing is
 * read through it.
 *
 * `workspace` is device memory of at least gemm355_xent_workspace(...) bytes, 16-byte
 * aligned (NULL when that is 0); its contents need not be kept between calls, and calls
 * that may run at the same time (two streams, two captured graphs) need one each.
 *
 * Arguments: M, N, K >= 0 and below 2^30, N >= 1 unless M == 0; ldx >= max(1, K); ldw >=
 * max(1, N), or max(1, K) with GEMM355_TRANS_B; pointers non-null where their matrix or
 * vector has elements.  M == 0 is a no-op.  K == 0 gives Z = 0. */

/* Bytes of workspace gemm355_xent needs for these arguments (host-only; 0 for arguments
 * it refuses). */
size_t gemm355_xent_workspace(int dtype, unsigned flags, int M, int N, int K);

/* loss (M values) and lse (M values) as above; either may be NULL when not wanted.
 *
 * Error of lse_t against the exact value of the given operands: the error e of a binary32
 * dot product of length K (as for gemm_f32 and its 16-bit counterparts) plus about
 * 2^-24 (4 |lse_t| + N / 256 + 64).  A logit that is NaN, +infinity, or 2^127 or more in
 * magnitude makes its row's results NaN. */
gemm355_status gemm355_xent(int dtype, unsigned flags, int M, int N, int K, const void *X,
                            int ldx, const void *W, int ldw, const int64_t *labels,
                            int64_t ignore, float *loss, float *lse, void *workspace,
                            size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace gemm355_xent_grad needs (host-only; 0 for arguments it refuses). */
size_t gemm355_xent_grad_workspace(int dtype, unsigned flags, int M, int N, int K);

/* The gradient of sum_t dloss_t loss_t:
 *
 *     dZ[t][v] = dloss_t (exp(Z[t][v] - lse_t) - [v == y_t])      (0 without a label)
 *     dX = dZ.op(W)^T  (M x K),   dop(W) = X^T.dZ  (dW laid out as W)
 *
 * lse as gemm355_xent returned it for the same operands; dloss M binary32 values.  dX and
 * dW are of type `dtype`, row strides lddx >= max(1, K), lddw as ldw; either may be NULL
 * when not wanted.  They are overwritten, must not overlap each other or an input, and
 * nothing outside them is written.  The logits are computed again piece by piece of the
 * vocabulary and each piece of dZ is rounded to `dtype` for the two products that read it
 * (for binary16 after scaling by the power of two that puts the largest |dloss_t| in
 * [2^13, 2^14), so that small probabilities are not lost; up to 64 rows and with 256
 * classes or more, what the rounding leaves is multiplied too); the products are summed in
 * binary32 and rounded once.  Values X holds in rows without a label do not reach dW.
 * M == 0 writes dW = 0. */
gemm355_status gemm355_xent_grad(int dtype, unsigned flags, int M, int N, int K, const void *X,
                                 int ldx, const void *W, int ldw, const int64_t *labels,
                                 int64_t ignore, const float *lse, const float *dloss, void *dX,
                                 int lddx, void *dW, int lddw, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream);

/* Flags of gemm355_route and gemm355_route_grad. */
enum {
    GEMM355_ROUTE_SIGMOID = 1, /* scores are 1 / (1 + exp(-x)) instead of the row's softmax */
    GEMM355_ROUTE_RENORM = 2   /* the chosen scores are divided by their sum */
};

/* Routing to experts.  For each of `rows` rows of router logits X (rows x experts, of type
 * `dtype`), with scores s = softmax(x) or sigmoid(x):
 *
 *     c_e = s_e + bias_e                       (bias NULL: 0; for the choice only)
 *     group score = sum of the `group_top` (1 or 2) largest c_e of the group
 *     the `top_groups` groups of the largest score are kept (groups of experts / groups
 *     consecutive experts each; all are kept when groups == top_groups)
 *     ids = the k kept experts of the largest c_e, in falling order
 *     weights_i = scale * s[ids_i]             (GEMM355_ROUTE_RENORM: / sum_j s[ids_j])
 *
 * Ties go to the lowest index.  Where binary32 scores cannot tell two choices or two group
 * scores apart they are compared in binary64; without a bias experts are compared by their
 * logits.  Weights are computed in binary64 and rounded once to binary32.
 * counts[e] (experts values; NULL when not wanted) is the number of rows that chose e.
 *
 * An expert whose logit is -infinity, or whose bias is -infinity or NaN, is masked: it is
 * never chosen and adds nothing to its group's score.  A row that runs out of experts has
 * id -1 and weight 0 in its remaining places.  A row whose chosen scores sum to 0 has
 * weights 0 with GEMM355_ROUTE_RENORM.  A row with a NaN logit (or, for softmax, a logit
 * of +infinity) has ids -1 and weights NaN.
 *
 * Arguments: 0 <= rows <= 2^30; 1 <= experts <= 1024; 1 <= groups <= 64 dividing experts;
 * 1 <= top_groups <= groups; group_top 1 or 2; 1 <= k <= min(64, top_groups * experts /
 * groups); ldx >= experts; ids and weights rows x k, packed, non-null (and X) unless rows
 * == 0, and no output overlapping another or an input.  counts is written (zeros) also
 * when rows == 0. */
gemm355_status gemm355_route(int dtype, unsigned flags, int rows, int experts, int k, int groups,
                             int top_groups, int group_top, const void *X, int ldx,
                             const float *bias, float scale, int32_t *ids, float *weights,
                             int32_t *counts, hipStream_t stream);

/* The gradient of sum_{t,i} dweights[t][i] weights[t][i] with respect to X, for the given
 * choice ids (rows x k, packed; an id outside [0, experts) marks a place without an
 * expert): with q_i = scale dweights_i,
 *
 *     RENORM: S = sum_j s[ids_j],  q_i <- (q_i - sum_j q_j s[ids_j] / S) / S   (0 if S == 0)
 *     ds_e = sum_{i: ids_i = e} q_i
 *     softmax: dX_e = s_e (ds_e - sum_f ds_f s_f);   sigmoid: dX_e = ds_e s_e (1 - s_e)
 *
 * With RENORM, and with sigmoid scores, only the chosen logits of a row enter its gradient,
 * and no other is read.
 *
 * dX (rows x experts, type `dtype`, row stride lddx) may equal X when lddx == ldx; any
 * other overlap is an argument error.  Arguments as for gemm355_route. */
gemm355_status gemm355_route_grad(int dtype, unsigned flags, int rows, int experts, int k,
                                  const void *X, int ldx, const int32_t *ids,
                                  const float *dweights, float scale, void *dX, int lddx,
                                  hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM355_SOFTMAX_H */
