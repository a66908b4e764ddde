/*
 * vpe_beam.h - C ABI of libvpe.so, beam search over the vocabulary-sharded
 * logits: the selection over beams and vocabulary from each rank's shard, the
 * merge of the ranks' picks, and the reordering of per-beam states.
 *
 * The conventions of vpe.h hold for every call here.  Rows of a sequence's
 * beams follow each other: row s * beams + b is beam b of sequence s.
 */
#ifndef VPE_BEAM_H
#define VPE_BEAM_H

#include "vpe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most beams per sequence, and most picks per sequence. */
#define VPE_MAX_BEAMS 64
#define VPE_MAX_BEAM_PICKS 64

/*
 * The candidates of a sequence are all (beam b, token j) with the score
 *
 *   c(b, j) = (z[b, j] - lse[b]) + score[b]
 *
 * each operation in fp32, rounded to nearest (-0 taken as +0): the beam's
 * accumulated log-probability plus the token's.  They are ordered by score,
 * equal scores by the lower b * vocab + j.  -inf is a score like any other
 * (masked tokens, beams that ended or do not exist yet); a NaN score comes
 * after all others.
 *
 * A pick travels as one 64-bit key,
 *
 *   key = (order(c) << 32) | (0xFFFFFFFF - (b * vocab + j))
 *
 * (order() maps binary32 bits to an unsigned integer ordered like the values,
 * NaN to 0), so larger keys are better picks and keys of different shards
 * compare directly.  Key 0 stands for no candidate.
 */

/* Bytes of workspace vpe_beam_select needs.  Host-only.  Errors: VPE_ERR_NULL,
 * VPE_ERR_SHAPE (as vpe_beam_select). */
vpe_status vpe_beam_select_workspace(int64_t n_seqs, int32_t beams, int64_t shard_rows,
                                     int32_t picks, int64_t *bytes);

/*
 * Each sequence's `picks` best candidates over one shard's tokens, as keys in
 * descending order (0 where the shard has fewer than `picks` candidates).
 *
 * logits  device, [n_seqs * beams] rows with row stride ld elements, of `dt`:
 *         the shard is columns [col_offset, col_offset + shard_rows).
 * lse     device float [n_seqs * beams]: each row's log-sum-exp over the whole
 *         vocabulary (vpe_lmhead_logsumexp, vpe_logsumexp_combine).
 * scores  device float [n_seqs * beams]: accumulated log-probabilities.
 * keys    device uint64 [n_seqs, picks], written.
 * workspace  device, at least vpe_beam_select_workspace(...) bytes, 8-byte
 *         aligned; needs no initialisation, not shared by calls that may run
 *         at the same time.
 * n_seqs == 0 is a no-op.
 * Errors: VPE_ERR_NULL, VPE_ERR_DTYPE, VPE_ERR_ALIGN, VPE_ERR_SHAPE (n_seqs <
 * 0, n_seqs * beams > 2^21, beams outside [1, VPE_MAX_BEAMS], picks outside
 * [1, VPE_MAX_BEAM_PICKS], shard_rows < 1 or >= 2^31, vocab < 1, a tensor too
 * large),
 * VPE_ERR_RANGE (the shard does not lie in [0, vocab), beams * vocab >= 2^32,
 * the columns do not fit ld), VPE_ERR_WORKSPACE.
 */
vpe_status vpe_beam_select(const void *logits, int64_t ld, int64_t col_offset, vpe_dtype dt,
                           int64_t n_seqs, int32_t beams, int64_t shard_rows, int64_t vocab_start,
                           int64_t vocab, const float *lse, const float *scores, int32_t picks,
                           uint64_t *keys, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The shards' picks merged into each sequence's `picks` best, best first:
 * score, parent beam and token of each.  Where the shards together hold fewer
 * than `picks` candidates the rest is score -inf, parent -1, token -1.
 *
 * keys    HOST array of n_parts device pointers, each uint64 [n_seqs, picks]
 *         (vpe_beam_select with the same picks and vocab); any order of the
 *         shards gives the same result.
 * score   device float [n_seqs, picks].
 * parent  device int64 [n_seqs, picks], beam of the sequence, in [0, beams).
 * token   device int64 [n_seqs, picks].
 * n_seqs == 0 is a no-op.
 * Errors: VPE_ERR_NULL, VPE_ERR_ALIGN, VPE_ERR_SHAPE (n_parts outside [1,
 * VPE_MAX_PARTS], picks outside [1, VPE_MAX_BEAM_PICKS], n_seqs < 0 or >
 * 2^21, vocab < 1 or >= 2^32).
 */
vpe_status vpe_beam_merge(const uint64_t *const *keys, int32_t n_parts, int64_t n_seqs,
                          int32_t picks, int64_t vocab, float *score, int64_t *parent,
                          int64_t *token, void *stream);

/*
 * States follow their beams:
 *
 *   dst[o, s * beams_out + b] = src[o, s * beams_in + parent[s * ld_parent + b]]
 *                               for o < outer, s < n_seqs, b < beams_out
 *
 * Rows of row_bytes bytes, copied unchanged; a parent outside [0, beams_in)
 * gives a row of zero bytes, and nothing is read for it.
 * src     device, [outer, n_seqs * beams_in, row_bytes].
 * parent  device int64, row stride ld_parent >= beams_out elements: the
 *         first beams_out parents of each sequence (ld_parent = picks takes
 *         them straight from vpe_beam_merge).
 * dst     device, [outer, n_seqs * beams_out, row_bytes]; must not overlap src
 *         or parent.
 * outer == 0 or n_seqs == 0 is a no-op.
 * Errors: VPE_ERR_NULL, VPE_ERR_ALIGN (parent), VPE_ERR_SHAPE (a size
 * negative, beams_in or beams_out < 1, row_bytes < 1, too large),
 * VPE_ERR_RANGE (ld_parent < beams_out, dst overlaps src or parent).
 */
vpe_status vpe_beam_reorder(const void *src, int64_t outer, int64_t n_seqs, int32_t beams_in,
                            int64_t row_bytes, const int64_t *parent, int64_t ld_parent,
                            int32_t beams_out, void *dst, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* VPE_BEAM_H */
