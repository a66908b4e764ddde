/*
 * vpe_loss.h - C ABI of libvpe.so, the loss and gradient calls of a training
 * step's head: softmax cross entropy straight from a rank's LM-head shard,
 * without keeping the logits, and its gradients; the LM head's backward from a
 * given gradient of its logits; the global norm of many gradients, and clipping.
 *
 * The conventions of vpe.h hold for every call here: device pointers are the
 * caller's, nothing is allocated, kept or synchronised, arguments are checked
 * on the host before anything is enqueued on `stream`, and values in device
 * memory (targets, factors) are not checked but have defined results.  Sums are
 * taken in fp32 or more, in an order fixed by the arguments: no atomics on
 * values, so the same inputs give the same bits.  Gradients are calls of their
 * own; the Python binding builds no autograd graph either.  Tensors that a call
 * writes (workspaces among them) must not overlap each other or its inputs
 * unless it says so: that is the caller's to see to here (the Python binding
 * refuses it).  A workspace needs no initialisation, and must not be shared by
 * calls that may run at the same time.
 */
#ifndef VPE_LOSS_H
#define VPE_LOSS_H

#include "vpe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Softmax cross entropy over a vocabulary of `vocab` ids, split into shards.
 * With z[i, j] = sum_d x[i, d] W[j, d], products summed in fp32 and not rounded,
 *
 *   lse[i]  = log sum_j exp(z[i, j])               over the whole vocabulary
 *   loss[i] = lse[i] - z[i, t_i],                  t_i = targets[i]
 *   d loss[i] / d z[i, j] = exp(z[i, j] - lse[i]) - [j = t_i]
 *
 * A row whose target lies outside [0, vocab) (a padding id such as -100) has
 * loss 0, lse 0 and gradient 0, and adds nothing to the table's gradient,
 * whatever its hidden row holds.  Elsewhere infinities and NaN follow the
 * formulas, except that a row with a logit of +inf has a NaN loss.
 *
 * Over the ranks: vpe_lmhead_xent per rank, the ranks exchange two floats per
 * row, vpe_xent_loss, and vpe_lmhead_xent_grad per rank.
 */

/* Most rows of one call of these, and the widest rows. */
#define VPE_MAX_LOSS_ROWS (1 << 21)
#define VPE_MAX_LOSS_DIM (1 << 16)

/* Bytes of workspace that serve vpe_lmhead_xent for m rows and for fewer.
 * Host-only.  Errors: VPE_ERR_NULL, VPE_ERR_DTYPE, VPE_ERR_SHAPE (as
 * vpe_lmhead_xent). */
vpe_status vpe_lmhead_xent_workspace(int64_t m, int64_t dim, int64_t shard_rows, vpe_dtype dt,
                                     int64_t *bytes);

/*
 * One shard's part of the loss:
 *
 *   shard_lse[i]    = log sum_j exp(z[i, j])   over the shard's rows j
 *   target_logit[i] = z[i, t_i]                if the shard owns t_i, else 0
 *
 * both 0 for a row without a target.
 *
 * x             device, [m, dim] of `dt`: hidden rows.
 * weight        device, [shard_rows, dim] of `dt`: the shard's table, ids
 *               [vocab_start, vocab_start + shard_rows).
 * targets       device, [m] of `itype`, ids of the whole vocabulary.
 * shard_lse, target_logit  device float [m], written.
 * workspace     device, at least vpe_lmhead_xent_workspace(...) bytes, 16-byte
 *               aligned.
 * m == 0 is a no-op.
 * Errors: VPE_ERR_NULL, VPE_ERR_DTYPE, VPE_ERR_ALIGN, VPE_ERR_SHAPE (m < 0 or
 * > VPE_MAX_LOSS_ROWS, dim < 1 or > VPE_MAX_LOSS_DIM, shard_rows < 1 or >=
 * 2^31, vocab < 1, more than 2^42 logits, a tensor too large), VPE_ERR_RANGE (the
 * shard does not lie in [0, vocab)), VPE_ERR_WORKSPACE.
 */
vpe_status vpe_lmhead_xent(const void *x, int64_t m, int64_t dim, const void *weight,
                           int64_t shard_rows, vpe_dtype dt, int64_t vocab_start, int64_t vocab,
                           const void *targets, vpe_itype itype, float *shard_lse,
                           float *target_logit, void *workspace, int64_t workspace_bytes,
                           void *stream);

/*
 * The ranks' parts joined, in shard order:
 *
 *   lse[i]  = log sum_r exp(shard_lse[r][i])
 *   loss[i] = lse[i] - sum_r target_logit[r][i]
 *
 * both 0 for a row without a target.
 *
 * shard_lse, target_logit  HOST arrays of n_parts device pointers, each float
 *               [m]; n_parts in [1, VPE_MAX_PARTS].
 * loss, lse     device float [m], written; each may equal one of the inputs.
 * m == 0 is a no-op.  Errors: as vpe_lmhead_xent where they apply;
 * VPE_ERR_SHAPE also for n_parts.
 */
vpe_status vpe_xent_loss(const float *const *shard_lse, const float *const *target_logit,
                         int32_t n_parts, int64_t m, int64_t vocab, const void *targets,
                         vpe_itype itype, float *loss, float *lse, void *stream);

/* Bytes of workspace that serve vpe_lmhead_xent_grad for m rows and for fewer.
 * Host-only.  Errors: VPE_ERR_NULL, VPE_ERR_DTYPE, VPE_ERR_SHAPE. */
vpe_status vpe_lmhead_xent_grad_workspace(int64_t m, int64_t dim, int64_t shard_rows,
                                          vpe_dtype dt, int64_t *bytes);

/*
 * One shard's gradients of sum_i grad_loss[i] loss[i].  With
 * d[i, j] = grad_loss[i] (exp(z[i, j] - lse[i]) - [j = t_i]),
 *
 *   grad_x[i, :]      = rnd(sum_j d[i, j] W[j, :])     over the shard's rows j
 *   grad_weight[j, :] = rnd(s[j, :])                       accumulate == 0
 *                     = rnd(grad_weight[j, :] + s[j, :])   accumulate != 0,
 *   s[j, :]           = sum_i d[i, j] x[i, :]
 *
 * grad_x is this shard's part: the ranks' parts sum to the whole.  The logits
 * are computed again, a piece of the vocabulary at a time; a piece's d / max
 * |grad_loss| is held in `dt` and multiplied with sums in fp32.  An entry of
 * exp(z - lse) - [j = t] carries what z and lse do (lse is fp32: 2^-24 of its
 * size), a few 2^-24 (1 + |z - lse|), both times exp(z - lse), and in bf16 one
 * rounding more, up to 2^-8 of the entry; at a target of probability close to 1 the
 * first two are the larger ones.  Entries of d below 2^-126 max |grad_loss| may
 * count as 0.  A row whose grad_loss is 0 counts as one without a target.
 *
 * lse          device float [m]: over the whole vocabulary (vpe_xent_loss).
 * grad_loss    device float [m].
 * grad_x       device, [m, dim] of `gxt`, every row written; or NULL.
 * grad_weight  device, [shard_rows, dim] of `gwt`, every row written (with
 *              accumulate: added to); or NULL, not with grad_x NULL too.
 * workspace    device, at least vpe_lmhead_xent_grad_workspace(...) bytes,
 *              16-byte aligned.
 * m == 0: grad_weight is zeros (accumulate == 0) or left as it is.
 * The rest as vpe_lmhead_xent.  Errors: as vpe_lmhead_xent.
 */
vpe_status vpe_lmhead_xent_grad(const void *x, int64_t m, int64_t dim, const void *weight,
                                int64_t shard_rows, vpe_dtype dt, int64_t vocab_start,
                                int64_t vocab, const void *targets, vpe_itype itype,
                                const float *lse, const float *grad_loss, void *grad_x,
                                vpe_dtype gxt, void *grad_weight, vpe_dtype gwt,
                                int32_t accumulate, void *workspace, int64_t workspace_bytes,
                                void *stream);

/* Bytes of workspace that serve vpe_lmhead_grad for m rows and for fewer.
 * Host-only.  Errors: VPE_ERR_NULL, VPE_ERR_DTYPE, VPE_ERR_SHAPE. */
vpe_status vpe_lmhead_grad_workspace(int64_t m, int64_t dim, int64_t shard_rows, vpe_dtype dt,
                                     int64_t *bytes);

/*
 * Backward of vpe_lmhead: from the gradient d of the shard's logits (such as
 * vpe_distill_grad's),
 *
 *   grad_x[i, :]      = rnd(sum_j d[i, j] W[j, :])
 *   grad_weight[j, :] = rnd(sum_i d[i, j] x[i, :])   (accumulate != 0: added)
 *
 * with sums in fp32.
 *
 * grad_logits  device, row-major with row stride ld elements, of `dt`: row i's
 *              shard is columns [col_offset, col_offset + shard_rows).  Other
 *              columns are not used, whatever they hold.
 * The rest as vpe_lmhead_xent_grad.
 * Errors: as vpe_lmhead_xent_grad where they apply; VPE_ERR_RANGE where the
 * columns do not fit ld.
 */
vpe_status vpe_lmhead_grad(const void *grad_logits, int64_t ld, int64_t col_offset, const void *x,
                           int64_t m, int64_t dim, const void *weight, int64_t shard_rows,
                           vpe_dtype dt, void *grad_x, vpe_dtype gxt, void *grad_weight,
                           vpe_dtype gwt, int32_t accumulate, void *workspace,
                           int64_t workspace_bytes, void *stream);

/*
 * Clipping by the global norm, over any number of tensors of either type.
 * A rank sums the squares of its own tensors (a tensor that several ranks hold
 * alike belongs in one rank's sum), the ranks exchange one double, and each
 * clips its tensors:
 *
 *   sumsq = sum over the tensors' elements of g^2       (products and sums in fp64)
 *   norm  = sqrt(sum_r sumsq_r)
 *   out   = rnd(min(1, max_norm / (norm + 1e-6)) g)     (the product in fp32)
 *
 * The factor is taken in fp64 and rounded to fp32.  A NaN norm makes it NaN, an
 * infinite one 0.
 */

/* Most tensors of one call. */
#define VPE_MAX_GRAD_TENSORS (1 << 16)

/* Bytes of workspace vpe_grad_sumsq needs for n tensors of counts[0..n)
 * elements (HOST array).  Host-only.  Errors: VPE_ERR_NULL, VPE_ERR_SHAPE. */
vpe_status vpe_grad_sumsq_workspace(const int64_t *counts, int32_t n, int64_t *bytes);

/*
 * tensors    HOST array of n device pointers; counts and dtypes HOST arrays of
 *            their elements and types (all read before the call returns).  A
 *            tensor of no elements may be NULL.
 * sumsq      device double [1], 8-byte aligned, written; 0 for n == 0.
 * workspace  device, at least vpe_grad_sumsq_workspace(counts, n) bytes, 8-byte
 *            aligned.
 * Errors: VPE_ERR_NULL, VPE_ERR_DTYPE, VPE_ERR_ALIGN, VPE_ERR_SHAPE (n < 0 or >
 * VPE_MAX_GRAD_TENSORS, a count < 0 or too large), VPE_ERR_WORKSPACE.
 */
vpe_status vpe_grad_sumsq(const void *const *tensors, const int64_t *counts,
                          const int32_t *dtypes, int32_t n, double *sumsq, void *workspace,
                          int64_t workspace_bytes, void *stream);

/*
 * tensors, counts, dtypes  as vpe_grad_sumsq.
 * out        HOST array of n device pointers, each of its tensor's type: the
 *            tensor itself, or a buffer apart from all of the call's tensors.
 * sumsq      HOST array of n_parts device pointers, each double [1], summed in
 *            this order; n_parts in [1, VPE_MAX_PARTS].
 * max_norm   finite and not negative.
 * norm       device float [1], written.
 * Errors: as vpe_grad_sumsq; VPE_ERR_SHAPE also for n_parts, VPE_ERR_RANGE for
 * max_norm.
 */
vpe_status vpe_grad_clip(const void *const *tensors, const int64_t *counts, const int32_t *dtypes,
                         int32_t n, void *const *out, const double *const *sumsq, int32_t n_parts,
                         double max_norm, float *norm, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* VPE_LOSS_H */
