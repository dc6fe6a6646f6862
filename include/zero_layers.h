/*
 * zero_layers.h -- part of the C ABI of libzero_mi355x.so: token tables and
 * norms, the parameters of a transformer whose gradients are sums over rows and
 * not matrix products. The forward passes read the parameters that a step has
 * written; the backward passes write their gradients where the step reads them:
 * the bf16 or fp32 gradients of a list or of the pack, or the rank's fp32
 * accumulator, added there over micro-batches.
 *
 *   zero_embedding        rows of a token table, scaled
 *   zero_token_order      the tokens of a batch sorted by their row
 *   zero_embedding_grad   the table's gradient, or a part of it, by sorted tokens
 *   zero_norm             layer norm (or its form without mean and bias) of
 *                         rows, the residual added in the same pass
 *   zero_norm_grad        its gradient: of the rows, of weight and bias
 *
 * The conventions of zero.h hold here: caller-owned device memory, calls that
 * enqueue on the given stream without synchronising, error codes with
 * zero_last_error(), arguments checked on the host before anything is enqueued.
 * Nothing is allocated, nothing is kept between calls, every call can be captured
 * into a graph, and equal inputs give bit-identical results: sums are taken in
 * 32 bits in an order that depends on the sizes and tokens only, and a value is
 * rounded once, to the type it is stored in. Arrays may start at any address that
 * suits their element type. "Stride" is the distance of two rows in elements;
 * within a row the elements are consecutive. An output's rows do not overlap
 * (stride >= dim with more than one row); an input's may (stride 0: one row, used
 * for all). Workspaces: contents on entry do not matter, calls that may run at the
 * same time need one each, and the bytes asked for do not fall as n grows, so one
 * for the largest batch serves all.
 */
#ifndef ZERO_LAYERS_MI355X_H
#define ZERO_LAYERS_MI355X_H

#include "zero_tensors.h"   /* ZERO_BF16, ZERO_F32 */

#ifdef __cplusplus
extern "C" {
#endif

/* Types of tokens. */
#define ZERO_I32 2
#define ZERO_I64 3

/* Limits of a call: tokens, rows of activations or of a table; elements of a row;
 * elements of all rows of activations, or of a part of a table's gradient. */
#define ZERO_LAYER_ROWS 16777215
#define ZERO_LAYER_DIM 1048576
#define ZERO_LAYER_ELEMS 34359738368

/* ---------------------------------------------------------------------------
 * zero_embedding -- out[t, :] = scale * table[token[t], :].
 * A token outside [0, rows), such as -1 behind the end of a sequence, gives a
 * row of zeros. The product is formed in fp32 and rounded to out's type.
 *   tokens      n tokens, ZERO_I32 or ZERO_I64
 *   table       [rows, dim], ZERO_BF16 or ZERO_F32, rows without gaps
 *   out         [n, dim] with its stride, ZERO_BF16 or ZERO_F32
 * Errors: ZERO_EINVAL for a NULL or misaligned array (with n = 0 the arrays may
 * be NULL), an unknown type, sizes outside the limits above (rows and dim from
 * 1, n from 0), a stride below dim, a scale that is not finite, or an output that
 * overlaps an input; ZERO_EHIP if a launch fails. */
int zero_embedding(const void* tokens, int32_t token_type, int64_t n, const void* table, int32_t table_type,
                   int64_t rows, int64_t dim, double scale, void* out, int32_t out_type, int64_t out_stride,
                   hipStream_t stream);

/* ---------------------------------------------------------------------------
 * zero_token_order -- sort a batch's tokens by their row, those of a row in
 * ascending position, those outside [0, rows) left out; for one or more
 * zero_embedding_grad calls on the same tokens (parts of the table, several
 * tables with the same tokens).
 *   order       device memory of at least zero_token_order_bytes(n, rows) bytes,
 *               16-byte aligned: the sorted tokens and scratch. It holds until the next
 *               call on it
 * Errors: as zero_embedding; ZERO_EINVAL for too few bytes.
 * zero_token_order_bytes returns 0 for sizes outside the limits. */
size_t zero_token_order_bytes(int64_t n, int64_t rows);
int zero_token_order(const void* tokens, int32_t token_type, int64_t n, int64_t rows, void* order,
                     size_t order_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * zero_embedding_grad -- the table's gradient, whole or in part:
 *   G[r, :] = scale * sum of d_out[t, :] over the t with token[t] = r
 *   grad[k] = G[first + k]  or  grad[k] + G[first + k]   for k in [0, count),
 * G taken as one flat array of rows * dim elements; a part may begin and end
 * inside a row, as a shard does (zero_layout's segments: first = src_off, grad at
 * dst_off of the shard). Written, rows without a token get zeros; added, they are
 * neither read nor written.
 * A row's terms are added in fp32 in ascending position, in pieces of consecutive
 * sorted tokens whose sums are then added in order.
 *   order       as zero_token_order has written it for the same n and rows, in
 *               zero_token_order_bytes(n, rows) bytes: so many are read, which the
 *               library cannot check (the Python binding does). Other contents of a
 *               buffer of that size give other sums, of the same arrays
 *   d_out       [n, dim] with its stride, ZERO_BF16 or ZERO_F32; what the rows of
 *               tokens outside the table hold does not matter
 *   grad        the part's count elements, ZERO_BF16 or ZERO_F32
 *   workspace   at least zero_embedding_grad_workspace_bytes(n, dim) bytes,
 *               16-byte aligned
 * Errors: ZERO_EINVAL for a NULL or misaligned array (d_out may be NULL with n =
 * 0, grad with count = 0), an unknown type, sizes outside the limits, a part outside
 * the table, a scale that is not finite, a workspace that is too small, or an output
 * or workspace that overlaps another array; ZERO_EHIP if a launch fails.
 * zero_embedding_grad_workspace_bytes returns 0 for sizes outside the limits. */
size_t zero_embedding_grad_workspace_bytes(int64_t n, int64_t dim);
int zero_embedding_grad(const void* order, int64_t n, int64_t rows, int64_t dim, const void* d_out,
                        int32_t out_type, int64_t out_stride, double scale, void* grad, int32_t grad_type,
                        int64_t first, int64_t count, int32_t accumulate, void* workspace, size_t ws_bytes,
                        hipStream_t stream);

/* ---------------------------------------------------------------------------
 * zero_norm -- norm of every row of an [n, dim] array:
 *   s = x                        or  s = total = x + residual, rounded to the type
 *   mean = sum(s) / dim          (0 where rms is set)
 *   rstd = 1 / sqrt(sum((s - mean)^2) / dim + eps)
 *   y = (s - mean) * rstd * weight + bias
 * Statistics are taken in fp32, the squares after the mean, and are left in mean and
 * rstd for the backward pass. In a row whose mean is larger than sqrt(variance + eps),
 * the rounding of the first mean is taken off by the sum of the deviations from it, so
 * a row of equal values gives the bias, however large they are. A row whose squared
 * deviations add up to more than fp32 holds gets rstd = 0.
 *   type, weight_type  ZERO_BF16 or ZERO_F32: of x, residual, total and y; of weight
 *                  and bias
 *   residual, total  both or neither
 *   weight, bias   [dim]; NULL stands for ones and for zeros
 *   mean, rstd     [n], fp32; either may be NULL where it is not needed
 * y may be x itself, total may be x or residual itself (same address and stride).
 * Errors: ZERO_EINVAL for a NULL or misaligned array (with n = 0 the arrays may be
 * NULL), an unknown type, sizes outside the limits, a stride that the conventions
 * above rule out, an eps below 0 or not finite, or an output that overlaps another
 * array; ZERO_EHIP if a launch fails. */
typedef struct {
  const void* x;
  const void* residual;
  void* total;
  void* y;
  const void* weight;
  const void* bias;
  float* mean;
  float* rstd;
  int64_t n, dim;
  int64_t x_stride, residual_stride, total_stride, y_stride;
  double eps;
  int32_t type, weight_type;
  int32_t rms;
  int32_t reserved;   /* 0 */
} zero_norm_args;

int zero_norm(const zero_norm_args* args, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * zero_norm_grad -- the gradient of zero_norm from d_y and what it left:
 *   xh = (x - mean) * rstd,  g = d_y * weight
 *   d_x = rstd * (g - sum(g) / dim - xh * sum(g * xh) / dim) (+ d_total)
 *   d_weight = (d_weight +) sum over rows of d_y * xh
 *   d_bias = (d_bias +) sum over rows of d_y
 * With rms there is no mean, and sum(g) is left out. x is what was normalised: total
 * where a residual was added; d_x is then the gradient of x and of residual alike, and
 * d_total, the gradient that reaches total by the skip path, is added in fp32 before
 * the rounding.
 *   type, weight_type, grad_type  ZERO_BF16 or ZERO_F32: of d_y, x, d_total and d_x; of
 *                  weight; of d_weight and d_bias
 *   mean, rstd     [n], fp32, of zero_norm (mean is not read with rms)
 *   weight         [dim]; NULL stands for ones
 *   d_x            may be NULL (the gradients of weight and bias only)
 *   d_total, d_weight, d_bias  may be NULL; d_total needs d_x
 *   accumulate     add to d_weight and d_bias instead of writing them
 *   workspace      at least zero_norm_grad_workspace_bytes(n, dim) bytes, 16-byte
 *                  aligned; may be NULL where d_weight and d_bias are
 * d_x may be d_y, x or d_total itself (same address and stride).
 * Errors: as zero_norm; ZERO_EINVAL for a workspace that is too small, and where no
 * output is asked for. zero_norm_grad_workspace_bytes returns 0 for sizes outside the
 * limits. */
typedef struct {
  const void* d_y;
  const void* x;
  const void* d_total;
  void* d_x;
  const void* weight;
  const float* mean;
  const float* rstd;
  void* d_weight;
  void* d_bias;
  int64_t n, dim;
  int64_t d_y_stride, x_stride, d_total_stride, d_x_stride;
  int32_t type, weight_type, grad_type;
  int32_t rms;
  int32_t accumulate;
  int32_t reserved;   /* 0 */
} zero_norm_grad_args;

size_t zero_norm_grad_workspace_bytes(int64_t n, int64_t dim);
int zero_norm_grad(const zero_norm_grad_args* args, void* workspace, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_LAYERS_MI355X_H */
