/*
 * zero_tensors.h -- part of the C ABI of libzero_mi355x.so: the optimizer step
 * over a list of tensors, for a rank that holds its share of the parameters
 * tensor by tensor (every tensor cut on its own, or whole tensors) instead of
 * one flat shard.
 *
 *   zero_tensors               describe the list: per tensor the parameter, the
 *                              fp32 master, the moments, the length, the group
 *   zero_tensors_upload        write the list's table to device memory
 *   zero_tensors_sqnorm        sum of squares of the list's gradients
 *   zero_tensors_adamw_step    clip with the global norm, AdamW, parameter cast
 *   zero_tensors_state_import, zero_tensors_state_export
 *                              fp32 moments to the 8-bit form and back
 *
 * The conventions of zero.h hold here: raw bf16 bit patterns, 64-bit sizes,
 * caller-owned device memory, calls that enqueue on the given stream without
 * synchronising, error codes with zero_last_error(), arguments checked on the
 * host before anything is enqueued. Nothing is allocated on the device.
 *
 * Gradients are passed per call as a HOST array of device pointers, entry i
 * for tensor i, read during the call. A NULL entry means that the tensor has
 * no gradient this time: it adds nothing to the norm, and the step leaves its
 * parameter and state as they are. The tensors may start at any address that
 * suits their element type (2 bytes for bf16, 4 for fp32, 1 for the 8-bit
 * moments) and may have any length, 0 and 1 included.
 */
#ifndef ZERO_TENSORS_MI355X_H
#define ZERO_TENSORS_MI355X_H

#include "zero.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of a list's parameters and gradients. */
#define ZERO_BF16 0
#define ZERO_F32 1

/* Elements of one tensor that share the scales of the 8-bit moments: blocks
 * [0, 256), [256, 512), ... of each tensor, the last one shorter. */
#define ZERO_STATE8_BLOCK 256

/* Hyperparameter groups one list may have. */
#define ZERO_TENSOR_GROUPS 8

/* Tensors whose gradients one launch carries in its arguments. A list of more
 * tensors takes several launches, one after another on the stream, and so does
 * one whose gradients lie 2^32 times their common alignment or more apart. */
#define ZERO_TENSORS_PER_LAUNCH 768

/* One tensor of a list; device pointers.
 *   param    the parameter, bf16 or fp32 (the list's param_type); written by
 *            the step. fp32 parameters are their own master weights.
 *   master   fp32 master weights; NULL when the parameters are fp32
 *   m, v     32-bit state: fp32 moments. 8-bit state: one byte per element,
 *            OCP e4m3 values of m and of sqrt(v)
 *   m_scale, v_scale  8-bit state: one fp32 per block of ZERO_STATE8_BLOCK
 *            elements: m = value * m_scale, sqrt(v) = value * v_scale. NULL
 *            with a 32-bit state.
 *   len      elements; a tensor of 0 elements may have NULL pointers
 *   group    index of its hyperparameters in the step's array, in
 *            [0, ZERO_TENSOR_GROUPS)
 * A zeroed 8-bit state (bytes and scales 0) stands for m = v = 0. */
typedef struct {
  void* param;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t len;
  int32_t group;
  int32_t reserved;   /* 0 */
} zero_tensor;

/* Opaque description of a list (host memory; the device table is the caller's). */
typedef struct zero_tensors_s* zero_tensors_t;

/* ---------------------------------------------------------------------------
 * zero_tensors -- describe a list (host only; nothing is enqueued).
 * The parameters a rank owns when every tensor is cut on its own, each with
 * its slice of the optimizer state ("第 5 课：ZeRO 与 FSDP" section 2: each
 * rank keeps 1/N_d of the state; "ZeRO-3 核心流程" section 2).
 *   tensors     host array of n descriptions, copied
 *   param_type, grad_type  ZERO_BF16 or ZERO_F32, of the whole list
 *   state_bits  32 or 8
 *   out         receives a handle to free with zero_tensors_free
 * Errors: ZERO_EINVAL for n < 1 or above 2^24, a NULL argument, an unknown type
 * or state, a length below 0 or a total beyond 2^40 elements, a group out of range, a
 * NULL or misaligned pointer that the types need, a master with fp32
 * parameters, scales with a 32-bit state, or two buffers of the list that
 * overlap (the same tensor listed twice among them); ZERO_ENOMEM if the host
 * allocation fails. */
int zero_tensors(const zero_tensor* tensors, int32_t n, int32_t param_type, int32_t grad_type,
                 int32_t state_bits, zero_tensors_t* out);

/* Release a handle (NULL is ignored). The device table must outlive the work
 * enqueued with it. */
void zero_tensors_free(zero_tensors_t h);

/* ---------------------------------------------------------------------------
 * zero_tensors_upload -- write the list's table into d_table (device memory of
 * at least zero_tensors_table_bytes(h) bytes, 16-byte aligned) and bind the
 * handle to it and to the current device. The table travels in kernel
 * arguments, so the call can be captured and reads no host memory after it
 * returns. The steps read the table: order their streams after this one (after
 * a captured upload, a call outside the graph after one of its replays). The
 * table must stay as written, at that address, as long as the handle is used;
 * a second upload binds the handle to a new table.
 * Errors: ZERO_EINVAL for NULL or misaligned arguments or too few bytes;
 * ZERO_EHIP if a launch fails. zero_tensors_table_bytes returns 0 for NULL. */
size_t zero_tensors_table_bytes(zero_tensors_t h);
int zero_tensors_upload(zero_tensors_t h, void* d_table, size_t table_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * zero_tensors_sqnorm -- sum of squares of the list's gradients: *d_out = it,
 * or *d_out += it when accumulate != 0 ("ZeRO-3 核心流程", pitfall 1: the clip
 * norm covers every rank's slices; callers add the ranks' sums). Each square is
 * exact in fp64 and the sum carried in fp64, in an order that depends only on
 * the lengths, so equal inputs give bit-identical results wherever they lie.
 *   tensor_grads  HOST array of the list's n device pointers (NULL allowed)
 *   d_workspace   device scratch of at least zero_tensors_sqnorm_workspace_bytes(h)
 *                 bytes, 8-byte aligned; contents on entry do not matter. Calls
 *                 that may run at the same time need one each.
 * Errors: ZERO_EINVAL for NULL arguments, a misaligned gradient, output or
 * workspace, a workspace that is too small, or a handle without a table on the
 * current device; ZERO_EHIP if a launch fails. */
size_t zero_tensors_sqnorm_workspace_bytes(zero_tensors_t h);
int zero_tensors_sqnorm(zero_tensors_t h, const void* const* tensor_grads, double* d_out, int32_t accumulate,
                        void* d_workspace, size_t ws_bytes, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * zero_tensors_adamw_step -- clip + AdamW + parameter cast over every tensor of
 * the list that has a gradient.
 *   tensor_grads  HOST array of the list's n device pointers (NULL: the tensor
 *                 is left as it is)
 *   groups        HOST array of n_groups hyperparameter sets; tensor i takes
 *                 groups[its group]. max_norm and clip_eps must be the same in
 *                 all of them (one norm clips the whole model); lr, betas, eps,
 *                 weight_decay and step may differ.
 *   d_rank_sqnorms, n_ranks  as zero_adamw_step
 *
 * 32-bit state: the arithmetic of zero_adamw_step, the fp64 recomputation of
 * cancelled masters included; on the same values the results are bit-identical
 * to it. 28 bytes per element with bf16 gradients and parameters.
 *
 * 8-bit state, 16.06 bytes per element: per block of 256 elements,
 *   m = M * m_scale, v = (S * v_scale)^2            M, S: the stored e4m3 values
 *   g' = c*g;  m1 = beta1*m + (1-beta1)*g';  v1 = beta2*v + (1-beta2)*g'^2   in fp64
 *   master = master - lr*wd*master - (lr/(1-beta1^t)) * m1 / (sqrt(v1)/sqrt(1-beta2^t) + eps)
 *            in fp32, from m1 and v1 before they are rounded to 8 bits
 *   am = max(fp32(max |m1|), 2^-100),       m_scale = am / 448, M = e4m3(m1 * (448 / am))
 *   as = max(sqrt(fp32(max v1)), 2^-63),    v_scale = as / 448, S = e4m3(sqrt(v1) * (448 / as))
 * with the scales and quotients rounded to fp32 and each 8-bit value the
 * correct rounding (nearest, ties to even) of the fp64 value: off by at most
 * 2^-4 relative, or 2^-10 of its scale below 2^-6. The root of a second moment
 * above zero is stored as at least 2^-9 scales: it never comes back as zero
 * under the division. Where a denominator is too small for fp32 to resolve its
 * root (eps = 0 and small roots, or very different ones in a block), the update
 * is evaluated in fp64. A moment that is NaN, or infinite in fp32, is stored as
 * the e4m3 NaN and left out of the maxima, so it spoils its own element only;
 * the step of an element whose second moment is infinite in fp32 is zero.
 *
 * Over many steps: rounding to nearest returns a root to its byte unless a step
 * changes it by half a step of e4m3, 1/30 to 1/16 of itself. It changes by
 * about (1-beta2)/2 * (g'^2/v - 1) of itself: with beta2 = 0.999 a byte moves by
 * its own gradient only where g'^2 passes 68 to 131 times v, and above
 * beta2 = (31/32)^2 = 0.938 never goes down by itself. What moves then is the
 * block's scale, with the block's largest root. Up to beta2 = 0.95 the roots
 * follow AdamW's all the same (98 of 100 within 0.8 to 1.4 times it, also after
 * gradients changed); with 0.98 or more they do not: at 0.999, elements whose
 * gradients fell to a tenth have a root 7 times too large 5000 steps later, and
 * those beside elements whose gradients rose by 4 get one 3 to 11 times too
 * large, so their steps are that much too short. For such a beta2 use the 32-bit state.
 *
 * Errors: ZERO_EINVAL for NULL arguments, n_groups outside [1,
 * ZERO_TENSOR_GROUPS] or not above a group the list uses, hyperparameters that
 * zero_adamw_step refuses, different max_norm or clip_eps, n_ranks < 1 or NULL
 * sums with clipping on, a misaligned gradient or one that overlaps a buffer
 * that the step writes, or a handle without a table on the current device;
 * ZERO_EHIP if a launch fails. */
int zero_tensors_adamw_step(zero_tensors_t h, const void* const* tensor_grads, const zero_adamw_hparams* groups,
                            int32_t n_groups, const double* d_rank_sqnorms, int32_t n_ranks, hipStream_t stream);

/* ---------------------------------------------------------------------------
 * zero_tensors_state_import / zero_tensors_state_export -- fp32 moments to the
 * 8-bit state of a list (state_bits 8) and back, for a checkpoint written with
 * fp32 moments, or one to be read by an optimizer that holds them so. The
 * import rounds as the step does, from m1 = m, v1 = v (a negative v is stored
 * as NaN); the export writes m = M * m_scale and v = (S * v_scale)^2, formed in
 * fp64 and rounded to fp32. Parameters and masters are not touched.
 *   m, v   HOST arrays of the list's n device pointers to fp32 arrays of the
 *          tensors' lengths; a tensor with both entries NULL is left out
 * Errors: ZERO_EINVAL for NULL arguments, a list with a 32-bit state, one of a
 * tensor's two entries NULL, a misaligned array or one that overlaps a buffer
 * of the list, an exported array that overlaps another, or a handle without a
 * table on the current device; ZERO_EHIP if a launch fails. */
int zero_tensors_state_import(zero_tensors_t h, const float* const* m, const float* const* v, hipStream_t stream);
int zero_tensors_state_export(zero_tensors_t h, float* const* m, float* const* v, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_TENSORS_MI355X_H */
