// The C ABI of the beam-search calls (include/vpe_beam.h): argument validation
// and dispatch to the kernel launchers.  Plain C++ with no HIP headers: a
// rejected call enqueues nothing.
#include "../../include/vpe_beam.h"

#include <stdint.h>

#include "vpe_train_launch.h"

namespace {

bool aligned(const void *p, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes)) == 0;
}

vpe_status launched(int rc) { return rc == 0 ? VPE_OK : VPE_ERR_LAUNCH; }

constexpr int64_t kMaxElems = int64_t(1) << 39;
constexpr int64_t kMaxRows = int64_t(1) << 21;
constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;
constexpr int64_t kMax32 = (int64_t(1) << 32) - 1;

bool beam_shape_ok(int64_t n_seqs, int32_t beams, int64_t shard_rows, int32_t picks) {
  return beams >= 1 && beams <= VPE_MAX_BEAMS && picks >= 1 && picks <= VPE_MAX_BEAM_PICKS &&
         n_seqs >= 0 && n_seqs <= kMaxRows / beams && shard_rows >= 1 && shard_rows <= kMax31;
}

}  // namespace

extern "C" {

vpe_status vpe_beam_select_workspace(int64_t n_seqs, int32_t beams, int64_t shard_rows,
                                     int32_t picks, int64_t *bytes) {
  if (!bytes) return VPE_ERR_NULL;
  if (!beam_shape_ok(n_seqs, beams, shard_rows, picks)) return VPE_ERR_SHAPE;
  // of either type of logits
  const int64_t f32 = vpe::beam_groups_per_row(beams, shard_rows, 0);
  const int64_t bf16 = vpe::beam_groups_per_row(beams, shard_rows, 1);
  *bytes = n_seqs * beams * (f32 > bf16 ? f32 : bf16) * 4;
  return VPE_OK;
}

vpe_status vpe_beam_select(const void *logits, int64_t ld, int64_t col_offset, vpe_dtype dt,
                           int64_t n_seqs, int32_t beams, int64_t shard_rows, int64_t vocab_start,
                           int64_t vocab, const float *lse, const float *scores, int32_t picks,
                           uint64_t *keys, void *workspace, int64_t workspace_bytes,
                           void *stream) {
  if (dt != VPE_F32 && dt != VPE_BF16) return VPE_ERR_DTYPE;
  if (!beam_shape_ok(n_seqs, beams, shard_rows, picks) || vocab < 1 || workspace_bytes < 0)
    return VPE_ERR_SHAPE;
  if (vocab > kMax32 / beams || vocab_start < 0 || vocab_start > vocab ||
      shard_rows > vocab - vocab_start)
    return VPE_ERR_RANGE;
  if (col_offset < 0 || ld < 1 || shard_rows > ld - col_offset) return VPE_ERR_RANGE;
  if (n_seqs * beams > kMaxElems / ld) return VPE_ERR_SHAPE;
  if (n_seqs == 0) return VPE_OK;
  if (!logits || !lse || !scores || !keys || !workspace) return VPE_ERR_NULL;
  const int64_t size = dt == VPE_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(lse, 4) || !aligned(scores, 4) || !aligned(keys, 8) ||
      !aligned(workspace, 8))
    return VPE_ERR_ALIGN;
  int64_t need = 0;
  const vpe_status rs = vpe_beam_select_workspace(n_seqs, beams, shard_rows, picks, &need);
  if (rs != VPE_OK) return rs;
  if (workspace_bytes < need) return VPE_ERR_WORKSPACE;
  return launched(vpe::launch_beam_select(
      static_cast<const char *>(logits) + col_offset * size, ld, dt == VPE_BF16 ? 1 : 0, n_seqs,
      beams, shard_rows, vocab_start, vocab, lse, scores, picks, keys,
      static_cast<float *>(workspace), stream));
}

vpe_status vpe_beam_merge(const uint64_t *const *keys, int32_t n_parts, int64_t n_seqs,
                          int32_t picks, int64_t vocab, float *score, int64_t *parent,
                          int64_t *token, void *stream) {
  if (n_parts < 1 || n_parts > VPE_MAX_PARTS || picks < 1 || picks > VPE_MAX_BEAM_PICKS ||
      n_seqs < 0 || n_seqs > kMaxRows || vocab < 1 || vocab > kMax32)
    return VPE_ERR_SHAPE;
  if (n_seqs == 0) return VPE_OK;
  if (!keys || !score || !parent || !token) return VPE_ERR_NULL;
  for (int32_t r = 0; r < n_parts; ++r) {
    if (!keys[r]) return VPE_ERR_NULL;
    if (!aligned(keys[r], 8)) return VPE_ERR_ALIGN;
  }
  if (!aligned(score, 4) || !aligned(parent, 8) || !aligned(token, 8)) return VPE_ERR_ALIGN;
  return launched(vpe::launch_beam_merge(keys, n_parts, n_seqs, picks, vocab, score, parent, token,
                                         stream));
}

vpe_status vpe_beam_reorder(const void *src, int64_t outer, int64_t n_seqs, int32_t beams_in,
                            int64_t row_bytes, const int64_t *parent, int64_t ld_parent,
                            int32_t beams_out, void *dst, void *stream) {
  if (outer < 0 || n_seqs < 0 || beams_in < 1 || beams_out < 1 || row_bytes < 1)
    return VPE_ERR_SHAPE;
  const int64_t most = beams_in > beams_out ? beams_in : beams_out;
  if (row_bytes > kMaxElems || n_seqs > kMaxElems / row_bytes / most) return VPE_ERR_SHAPE;
  if (outer > kMaxElems) return VPE_ERR_SHAPE;
  if (outer > 0 && n_seqs > 0 && outer > kMaxElems / (row_bytes * n_seqs * most))
    return VPE_ERR_SHAPE;
  if (ld_parent < beams_out) return VPE_ERR_RANGE;
  if (n_seqs > 0 && ld_parent > kMaxElems / n_seqs) return VPE_ERR_SHAPE;
  if (outer == 0 || n_seqs == 0) return VPE_OK;
  if (!src || !parent || !dst) return VPE_ERR_NULL;
  if (!aligned(parent, 8)) return VPE_ERR_ALIGN;
  const uintptr_t s0 = reinterpret_cast<uintptr_t>(src), d0 = reinterpret_cast<uintptr_t>(dst);
  const uintptr_t sb = static_cast<uintptr_t>(outer * n_seqs * beams_in * row_bytes);
  const uintptr_t db = static_cast<uintptr_t>(outer * n_seqs * beams_out * row_bytes);
  if (d0 < s0 + sb && s0 < d0 + db) return VPE_ERR_RANGE;
  // parents are read while other rows are written
  const uintptr_t p0 = reinterpret_cast<uintptr_t>(parent);
  const uintptr_t pb = static_cast<uintptr_t>(((n_seqs - 1) * ld_parent + beams_out) * 8);
  if (d0 < p0 + pb && p0 < d0 + db) return VPE_ERR_RANGE;
  return launched(vpe::launch_beam_reorder(src, outer, n_seqs, beams_in, row_bytes, parent,
                                           ld_parent, beams_out, dst, stream));
}

}  // extern "C"
