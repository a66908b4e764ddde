/*
 * vpe_train.h - C ABI of libvpe.so, training calls of the two
 * vocabulary-sharded layers: the scaled lookup, the gradient of the lookup
 * with respect to a rank's table shard, and distillation from a teacher's top
 * logits, forward and backward, over the ranks' shards of the logits.
 *
 * The conventions of vpe.h hold for every call here: device pointers are the
 * caller's, nothing is allocated, kept or synchronised, arguments are checked
 * on the host before anything is enqueued on `stream`, and values in device
 * memory (ids, teacher entries) are not checked but have defined results.
 * Every sum is taken in fp32 or more, in an order fixed by the arguments: no
 * atomics on values, so the same inputs give the same bits.  Gradients are calls
 * of their own; the Python binding builds no autograd graph either.
 */
#ifndef VPE_TRAIN_H
#define VPE_TRAIN_H

#include "vpe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * vpe_embed with every owned row times a factor:
 *
 *   out[i, :] = rnd(scale * weight[ids[i] - vocab_start, :])  for ids in the shard
 *             = all-zero bits (+0.0)                           otherwise
 *
 * The product is taken in fp32 and rounded once to `dt` (round to nearest,
 * ties to even).  Arguments as vpe_embed; scale must be finite.
 * Errors: as vpe_embed; VPE_ERR_RANGE also when scale is not finite.
 */
vpe_status vpe_embed_scaled(const void *ids, vpe_itype itype, int64_t n, const void *weight,
                            vpe_dtype dt, int64_t shard_rows, int64_t dim, int64_t vocab_start,
                            float scale, void *out, void *stream);

/* Bytes of workspace vpe_embed_grad needs for n ids; as much serves any smaller
 * number.  Host-only.  Errors: VPE_ERR_NULL, VPE_ERR_SHAPE (as
 * vpe_embed_grad). */
vpe_status vpe_embed_grad_workspace(int64_t n, int64_t shard_rows, int64_t dim, int64_t *bytes);

/*
 * Gradient of vpe_embed_scaled (scale = 1: of vpe_embed) with respect to the
 * shard, from the gradient of its output:
 *
 *   s[j, :]           = scale * sum_{i : ids[i] - vocab_start = j} grad_out[i, :]
 *   grad_weight[j, :] = rnd(s[j, :])                       accumulate == 0
 *                     = rnd(grad_weight[j, :] + s[j, :])   accumulate != 0
 *
 * The positions are sorted by token (stable) and each token's rows summed in
 * ascending i inside fixed pieces of the sorted order, one rounding to `gdt`: at
 * most 32 rows, and 16 such sums, in fp32, and what is longer in 64 bits, so that
 * a sum's error does not grow with the number of its rows.  Ids outside the shard add nothing, whatever their grad_out rows
 * hold (a padding id such as -1 takes no gradient).  With accumulate == 0
 * every row of grad_weight is written, +0.0 where the shard row has no id;
 * with accumulate != 0 rows without an id are left as they are.
 *
 * ids          device, [n] of `itype`, any values.
 * grad_out     device, [n, dim] of `dt`.
 * grad_weight  device, [shard_rows, dim] of `gdt` (either type, whatever `dt`
 *              is: fp32 gradients of a bf16 model).
 * workspace    device, at least vpe_embed_grad_workspace(n, shard_rows, dim)
 *              bytes, 16-byte aligned; needs no initialisation, and must not
 *              be shared by calls that may run at the same time.
 * grad_weight and workspace must overlap neither each other nor the inputs:
 * that is the caller's to see to here (the Python binding refuses it).
 * n == 0 writes zeros (accumulate == 0) or does nothing.
 * Errors: VPE_ERR_NULL, VPE_ERR_DTYPE, VPE_ERR_ALIGN, VPE_ERR_SHAPE (n < 0 or
 * >= 2^31, dim < 1 or > 2^20, shard_rows < 1 or >= 2^31, a tensor too large),
 * VPE_ERR_RANGE (vocab_start < 0 or vocab_start + shard_rows past INT64_MAX,
 * scale not finite), VPE_ERR_WORKSPACE.
 */
vpe_status vpe_embed_grad(const void *ids, vpe_itype itype, int64_t n, const void *grad_out,
                          vpe_dtype dt, int64_t dim, int64_t vocab_start, int64_t shard_rows,
                          float scale, void *grad_weight, vpe_dtype gdt, int32_t accumulate,
                          void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Distillation from a teacher's top logits.  Row i has k entries (id, t): the
 * teacher's largest logits t and their vocabulary ids.  Entries whose id lies
 * outside [0, vocab) are padding and count for nothing.  With T the
 * temperature, z the student's logits and the sums over the row's entries,
 *
 *   p_e  = exp(t_e / T - L),  L = log sum_e exp(t_e / T), or the caller's
 *          teacher_lse[i] (the teacher's log-sum-exp over its whole
 *          vocabulary: the entries then hold the mass P = sum_e p_e <= 1)
 *   lse  = log sum_j exp(z_j / T)           over the whole vocabulary
 *   loss = sum_e p_e (log p_e - z_{id_e} / T + lse)
 *   d loss / d z_j = (P exp(z_j / T - lse) - sum_{e : id_e = j} p_e) / T
 *
 * An id that occurs twice in a row counts twice.  An entry with p_e = 0 (t_e
 * = -inf) counts for nothing.  A row without entries that count has loss 0
 * and gradient 0, whatever its logits hold: that is how padded rows are
 * marked.  Elsewhere infinities and NaN follow the formulas (the log-sum-exp
 * of a row that holds +inf is +inf).  The gradient has the resolution of lse in
 * fp32: a row whose logits are all a mask's lowest value is best marked as
 * padding.
 *
 * Over vocabulary shards: vpe_distill_shard per rank (one pass over its
 * logits), the ranks exchange two floats per row, vpe_distill_loss, and
 * vpe_distill_grad per rank.  Exponentials are taken in fp32, sums and
 * logarithms in fp32 or more.
 */

/* Most entries per row, and most rows, of one distillation call. */
#define VPE_MAX_TEACHER_ENTRIES 1024
#define VPE_MAX_DISTILL_ROWS (1 << 21)

/* From this many rows on vpe_distill_shard gives each a workgroup of its own,
 * and needs no workspace. */
#define VPE_DISTILL_WHOLE_ROWS 256

/* Bytes of workspace that serve vpe_distill_shard for m rows and for fewer (so
 * not 0 from VPE_DISTILL_WHOLE_ROWS rows on).  Host-only.
 * Errors: VPE_ERR_NULL, VPE_ERR_SHAPE (m < 0 or > VPE_MAX_DISTILL_ROWS,
 * shard_rows < 1 or >= 2^31). */
vpe_status vpe_distill_workspace(int64_t m, int64_t shard_rows, int64_t *bytes);

/*
 * One shard's part of the loss:
 *
 *   shard_lse[i] = log sum_j exp(z[i, j] / T)      over the shard's columns j
 *   shard_dot[i] = sum_e p_e z[i, id_e - vocab_start] / T   over entries in the shard
 *
 * logits       device, row-major with row stride ld elements, of `dt`: row i's
 *              shard is columns [col_offset, col_offset + shard_rows), as
 *              vpe_lmhead writes them.
 * teacher_ids  device, [m, k] of `itype`, ids of the whole vocabulary.
 * teacher      device, [m, k] of `tdt`: the entries' logits.
 * teacher_lse  device float [m], or NULL.
 * shard_lse    device float [m], or NULL: not computed, and the logits are
 *              read at the entries' ids only (T = 1 after
 *              vpe_lmhead_logsumexp, whose shard_lse is this one).
 * shard_dot    device float [m].
 * workspace    device, at least vpe_distill_workspace(m, shard_rows) bytes,
 *              8-byte aligned; needs no initialisation, not shared by calls
 *              that may run at the same time; may be NULL where shard_lse is,
 *              and from VPE_DISTILL_WHOLE_ROWS rows on.
 * m == 0 is a no-op.
 * Errors: VPE_ERR_NULL, VPE_ERR_DTYPE, VPE_ERR_ALIGN, VPE_ERR_SHAPE (m < 0 or
 * > VPE_MAX_DISTILL_ROWS, shard_rows < 1 or >= 2^31, k outside [1,
 * VPE_MAX_TEACHER_ENTRIES], vocab < 1, a tensor too large), VPE_ERR_RANGE (the
 * shard does not lie in [0, vocab), the columns do not fit ld, temperature not
 * positive or past 2^100, or log2(e) / temperature infinite in fp32: below
 * 4.24e-39), VPE_ERR_WORKSPACE.
 */
vpe_status vpe_distill_shard(const void *logits, int64_t ld, int64_t col_offset, int64_t m,
                             int64_t shard_rows, vpe_dtype dt, int64_t vocab_start, int64_t vocab,
                             float temperature, const void *teacher_ids, vpe_itype itype,
                             const void *teacher, vpe_dtype tdt, int32_t k,
                             const float *teacher_lse, float *shard_lse, float *shard_dot,
                             void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The ranks' parts joined, in shard order:
 *
 *   lse[i]  = log sum_r exp(shard_lse[r][i])
 *   loss[i] = sum_e p_e log p_e - sum_r shard_dot[r][i] + P lse[i]
 *
 * shard_lse, shard_dot  HOST arrays of n_parts device pointers, each float
 *              [m]; n_parts in [1, VPE_MAX_PARTS].
 * teacher_ids, teacher, teacher_lse, vocab, temperature: as vpe_distill_shard.
 * loss, lse    device float [m], written; lse may equal one of the inputs.
 * m == 0 is a no-op.  Errors: as vpe_distill_shard where they apply;
 * VPE_ERR_SHAPE also for n_parts.
 */
vpe_status vpe_distill_loss(const float *const *shard_lse, const float *const *shard_dot,
                            int32_t n_parts, int64_t m, int64_t vocab, float temperature,
                            const void *teacher_ids, vpe_itype itype, const void *teacher,
                            vpe_dtype tdt, int32_t k, const float *teacher_lse, float *loss,
                            float *lse, void *stream);

/*
 * One shard's gradient of sum_i grad_loss[i] loss[i]:
 *
 *   grad_logits[i, j] = rnd(grad_loss[i] / T * (P exp(z[i, j] / T - lse[i])
 *                                               - sum_{e : id_e = vocab_start + j} p_e))
 *
 * computed in fp32 and rounded once to `dt`.  A row whose grad_loss is 0, and
 * a row without entries that count, is all +0.0, and its logits are not read.
 * lse          device float [m]: over the whole vocabulary (vpe_distill_loss).
 * grad_loss    device float [m].
 * grad_logits  device, row-major with row stride ld_grad elements, of `dt`:
 *              only columns [grad_col_offset, grad_col_offset + shard_rows) of
 *              rows [0, m) are written.  May be the logits themselves (the
 *              same columns of the same rows), or other columns of their
 *              buffer; any other overlap is refused.
 * The rest as vpe_distill_shard.  m == 0 is a no-op.
 * Errors: as vpe_distill_shard where they apply; VPE_ERR_RANGE also for the
 * columns of grad_logits, and where these overlap the logits' without being
 * the same.
 */
vpe_status vpe_distill_grad(const void *logits, int64_t ld, int64_t col_offset, int64_t m,
                            int64_t shard_rows, vpe_dtype dt, int64_t vocab_start, int64_t vocab,
                            float temperature, const void *teacher_ids, vpe_itype itype,
                            const void *teacher, vpe_dtype tdt, int32_t k,
                            const float *teacher_lse, const float *lse, const float *grad_loss,
                            void *grad_logits, int64_t ld_grad, int64_t grad_col_offset,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* VPE_TRAIN_H */
