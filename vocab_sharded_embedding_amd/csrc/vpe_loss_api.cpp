// The C ABI of the loss calls (include/vpe_loss.h): argument validation and
// dispatch to the kernel launchers, as vpe_api.cpp does for vpe.h.  Plain C++
// with no HIP headers: a rejected call enqueues nothing.
#include "../../include/vpe_loss.h"

#include <math.h>
#include <stdint.h>

#include "vpe_loss_launch.h"

namespace {

bool known_dtype(vpe_dtype dt) { return dt == VPE_F32 || dt == VPE_BF16; }
bool known_itype(vpe_itype it) { return it == VPE_I32 || it == VPE_I64; }
int64_t dtype_bytes(vpe_dtype dt) { return dt == VPE_F32 ? 4 : 2; }
int64_t itype_bytes(vpe_itype it) { return it == VPE_I32 ? 4 : 8; }
int code(vpe_dtype dt) { return dt == VPE_BF16 ? 1 : 0; }

bool aligned(const void *p, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes)) == 0;
}

vpe_status launched(int rc) { return rc == 0 ? VPE_OK : VPE_ERR_LAUNCH; }

// Largest element count of any one tensor (indexes in the kernels are 64-bit).
constexpr int64_t kMaxElems = int64_t(1) << 39;
constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;
// Largest number of logits: their tiles are counted in 31 bits.
constexpr int64_t kMaxLogits = int64_t(1) << 42;

vpe_status check_sizes(int64_t m, int64_t dim, int64_t shard_rows, vpe_dtype dt) {
  if (!known_dtype(dt)) return VPE_ERR_DTYPE;
  if (m < 0 || m > VPE_MAX_LOSS_ROWS || dim < 1 || dim > VPE_MAX_LOSS_DIM || shard_rows < 1 ||
      shard_rows > kMax31 || shard_rows > kMaxElems / dim ||
      (m > 0 && shard_rows > kMaxLogits / m))
    return VPE_ERR_SHAPE;
  return VPE_OK;
}

vpe_status check_shard(int64_t m, int64_t dim, int64_t shard_rows, vpe_dtype dt,
                       int64_t vocab_start, int64_t vocab, vpe_itype itype) {
  if (!known_itype(itype)) return VPE_ERR_DTYPE;
  const vpe_status rs = check_sizes(m, dim, shard_rows, dt);
  if (rs != VPE_OK) return rs;
  if (vocab < 1) return VPE_ERR_SHAPE;
  if (vocab_start < 0 || vocab_start > vocab || shard_rows > vocab - vocab_start)
    return VPE_ERR_RANGE;
  return VPE_OK;
}

vpe_status workspace_bytes_of(vpe::LossCall call, int64_t m, int64_t dim, int64_t shard_rows,
                              vpe_dtype dt, int64_t *bytes) {
  if (!bytes) return VPE_ERR_NULL;
  const vpe_status rs = check_sizes(m, dim, shard_rows, dt);
  if (rs != VPE_OK) return rs;
  *bytes = vpe::loss_layout(call, m, dim, shard_rows, code(dt)).bytes;
  return VPE_OK;
}

vpe_status check_workspace(vpe::LossCall call, int64_t m, int64_t dim, int64_t shard_rows,
                           vpe_dtype dt, const void *workspace, int64_t bytes) {
  if (!workspace) return VPE_ERR_NULL;
  if (!aligned(workspace, 16)) return VPE_ERR_ALIGN;
  if (bytes < vpe::loss_layout(call, m, dim, shard_rows, code(dt)).bytes)
    return VPE_ERR_WORKSPACE;
  return VPE_OK;
}

vpe_status check_gradients(vpe_dtype dt, const void *x, const void *weight, int64_t m,
                           const void *grad_x, vpe_dtype gxt, const void *grad_weight,
                           vpe_dtype gwt) {
  if ((!grad_x && !grad_weight) || !weight || (m > 0 && !x)) return VPE_ERR_NULL;
  if (!aligned(x, dtype_bytes(dt)) || !aligned(weight, dtype_bytes(dt)) ||
      !aligned(grad_x, dtype_bytes(gxt)) || !aligned(grad_weight, dtype_bytes(gwt)))
    return VPE_ERR_ALIGN;
  return VPE_OK;
}

// Sums the tensors' elements; VPE_ERR_SHAPE for a count that is no size.
vpe_status check_tensors(const int64_t *counts, int32_t n, int64_t *total) {
  if (n < 0 || n > VPE_MAX_GRAD_TENSORS) return VPE_ERR_SHAPE;
  if (n > 0 && !counts) return VPE_ERR_NULL;
  *total = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (counts[i] < 0 || counts[i] > kMaxElems - *total) return VPE_ERR_SHAPE;
    *total += counts[i];
  }
  return VPE_OK;
}

vpe_status check_tensor_pointers(const void *const *tensors, const int64_t *counts,
                                 const int32_t *dtypes, int32_t n) {
  if (n > 0 && (!tensors || !dtypes)) return VPE_ERR_NULL;
  for (int32_t i = 0; i < n; ++i) {
    const vpe_dtype dt = static_cast<vpe_dtype>(dtypes[i]);
    if (dtypes[i] != VPE_F32 && dtypes[i] != VPE_BF16) return VPE_ERR_DTYPE;
    if (counts[i] > 0 && !tensors[i]) return VPE_ERR_NULL;
    if (!aligned(tensors[i], dtype_bytes(dt))) return VPE_ERR_ALIGN;
  }
  return VPE_OK;
}

}  // namespace

extern "C" {

vpe_status vpe_lmhead_xent_workspace(int64_t m, int64_t dim, int64_t shard_rows, vpe_dtype dt,
                                     int64_t *bytes) {
  return workspace_bytes_of(vpe::kLossForward, m, dim, shard_rows, dt, bytes);
}

vpe_status vpe_lmhead_xent(const void *x, int64_t m, int64_t dim, const void *weight,
                           int64_t shard_rows, vpe_dtype dt, int64_t vocab_start, int64_t vocab,
                           const void *targets, vpe_itype itype, float *shard_lse,
                           float *target_logit, void *workspace, int64_t workspace_bytes,
                           void *stream) {
  vpe_status rs = check_shard(m, dim, shard_rows, dt, vocab_start, vocab, itype);
  if (rs != VPE_OK) return rs;
  if (workspace_bytes < 0) return VPE_ERR_SHAPE;
  if (m == 0) return VPE_OK;
  if (!x || !weight || !targets || !shard_lse || !target_logit) return VPE_ERR_NULL;
  if (!aligned(x, dtype_bytes(dt)) || !aligned(weight, dtype_bytes(dt)) ||
      !aligned(targets, itype_bytes(itype)) || !aligned(shard_lse, 4) || !aligned(target_logit, 4))
    return VPE_ERR_ALIGN;
  rs = check_workspace(vpe::kLossForward, m, dim, shard_rows, dt, workspace, workspace_bytes);
  if (rs != VPE_OK) return rs;
  return launched(vpe::launch_lmhead_xent(
      vpe::LossRows{x, m, dim, weight, shard_rows, code(dt), vocab_start, vocab, targets,
                    itype == VPE_I32 ? 0 : 1},
      shard_lse, target_logit, workspace, stream));
}

vpe_status vpe_xent_loss(const float *const *shard_lse, const float *const *target_logit,
                         int32_t n_parts, int64_t m, int64_t vocab, const void *targets,
                         vpe_itype itype, float *loss, float *lse, void *stream) {
  if (!known_itype(itype)) return VPE_ERR_DTYPE;
  if (m < 0 || m > VPE_MAX_LOSS_ROWS || vocab < 1 || n_parts < 1 || n_parts > VPE_MAX_PARTS)
    return VPE_ERR_SHAPE;
  if (m == 0) return VPE_OK;
  if (!shard_lse || !target_logit || !targets || !loss || !lse) return VPE_ERR_NULL;
  for (int32_t r = 0; r < n_parts; ++r) {
    if (!shard_lse[r] || !target_logit[r]) return VPE_ERR_NULL;
    if (!aligned(shard_lse[r], 4) || !aligned(target_logit[r], 4)) return VPE_ERR_ALIGN;
  }
  if (!aligned(targets, itype_bytes(itype)) || !aligned(loss, 4) || !aligned(lse, 4))
    return VPE_ERR_ALIGN;
  return launched(vpe::launch_xent_loss(shard_lse, target_logit, n_parts, m, vocab, targets,
                                        itype == VPE_I32 ? 0 : 1, loss, lse, stream));
}

vpe_status vpe_lmhead_xent_grad_workspace(int64_t m, int64_t dim, int64_t shard_rows,
                                          vpe_dtype dt, int64_t *bytes) {
  return workspace_bytes_of(vpe::kLossGrad, m, dim, shard_rows, dt, bytes);
}

vpe_status vpe_lmhead_xent_grad(const void *x, int64_t m, int64_t dim, const void *weight,
                                int64_t shard_rows, vpe_dtype dt, int64_t vocab_start,
                                int64_t vocab, const void *targets, vpe_itype itype,
                                const float *lse, const float *grad_loss, void *grad_x,
                                vpe_dtype gxt, void *grad_weight, vpe_dtype gwt,
                                int32_t accumulate, void *workspace, int64_t workspace_bytes,
                                void *stream) {
  vpe_status rs = check_shard(m, dim, shard_rows, dt, vocab_start, vocab, itype);
  if (rs != VPE_OK) return rs;
  if (!known_dtype(gxt) || !known_dtype(gwt)) return VPE_ERR_DTYPE;
  if (workspace_bytes < 0) return VPE_ERR_SHAPE;
  rs = check_gradients(dt, x, weight, m, grad_x, gxt, grad_weight, gwt);
  if (rs != VPE_OK) return rs;
  if (m > 0 && (!targets || !lse || !grad_loss)) return VPE_ERR_NULL;
  if (!aligned(targets, itype_bytes(itype)) || !aligned(lse, 4) || !aligned(grad_loss, 4))
    return VPE_ERR_ALIGN;
  if (m == 0 && (accumulate != 0 || !grad_weight)) return VPE_OK;
  rs = check_workspace(vpe::kLossGrad, m, dim, shard_rows, dt, workspace, workspace_bytes);
  if (rs != VPE_OK) return rs;
  return launched(vpe::launch_lmhead_xent_grad(
      vpe::LossRows{x, m, dim, weight, shard_rows, code(dt), vocab_start, vocab, targets,
                    itype == VPE_I32 ? 0 : 1},
      lse, grad_loss, vpe::LossGrads{grad_x, code(gxt), grad_weight, code(gwt), accumulate != 0},
      workspace, stream));
}

vpe_status vpe_lmhead_grad_workspace(int64_t m, int64_t dim, int64_t shard_rows, vpe_dtype dt,
                                     int64_t *bytes) {
  return workspace_bytes_of(vpe::kHeadGrad, m, dim, shard_rows, dt, bytes);
}

vpe_status vpe_lmhead_grad(const void *grad_logits, int64_t ld, int64_t col_offset, const void *x,
                           int64_t m, int64_t dim, const void *weight, int64_t shard_rows,
                           vpe_dtype dt, void *grad_x, vpe_dtype gxt, void *grad_weight,
                           vpe_dtype gwt, int32_t accumulate, void *workspace,
                           int64_t workspace_bytes, void *stream) {
  vpe_status rs = check_sizes(m, dim, shard_rows, dt);
  if (rs != VPE_OK) return rs;
  if (!known_dtype(gxt) || !known_dtype(gwt)) return VPE_ERR_DTYPE;
  if (col_offset < 0 || ld < 1 || shard_rows > ld - col_offset) return VPE_ERR_RANGE;
  if (workspace_bytes < 0 || m > kMaxElems / ld) return VPE_ERR_SHAPE;
  rs = check_gradients(dt, x, weight, m, grad_x, gxt, grad_weight, gwt);
  if (rs != VPE_OK) return rs;
  if (m > 0 && !grad_logits) return VPE_ERR_NULL;
  if (!aligned(grad_logits, dtype_bytes(dt))) return VPE_ERR_ALIGN;
  if (m == 0 && (accumulate != 0 || !grad_weight)) return VPE_OK;
  rs = check_workspace(vpe::kHeadGrad, m, dim, shard_rows, dt, workspace, workspace_bytes);
  if (rs != VPE_OK) return rs;
  return launched(vpe::launch_lmhead_grad(
      m > 0 ? static_cast<const char *>(grad_logits) + col_offset * dtype_bytes(dt) : nullptr, ld,
      vpe::LossRows{x, m, dim, weight, shard_rows, code(dt), 0, shard_rows, nullptr, 0},
      vpe::LossGrads{grad_x, code(gxt), grad_weight, code(gwt), accumulate != 0}, workspace,
      stream));
}

vpe_status vpe_grad_sumsq_workspace(const int64_t *counts, int32_t n, int64_t *bytes) {
  if (!bytes) return VPE_ERR_NULL;
  int64_t total = 0;
  const vpe_status rs = check_tensors(counts, n, &total);
  if (rs != VPE_OK) return rs;
  *bytes = 8 * vpe::loss_max(1, vpe::clip_chunks(counts, n, vpe::clip_chunk(total)));
  return VPE_OK;
}

vpe_status vpe_grad_sumsq(const void *const *tensors, const int64_t *counts,
                          const int32_t *dtypes, int32_t n, double *sumsq, void *workspace,
                          int64_t workspace_bytes, void *stream) {
  int64_t total = 0;
  vpe_status rs = check_tensors(counts, n, &total);
  if (rs != VPE_OK) return rs;
  if (workspace_bytes < 0) return VPE_ERR_SHAPE;
  rs = check_tensor_pointers(tensors, counts, dtypes, n);
  if (rs != VPE_OK) return rs;
  if (!sumsq || !workspace) return VPE_ERR_NULL;
  if (!aligned(sumsq, 8) || !aligned(workspace, 8)) return VPE_ERR_ALIGN;
  if (workspace_bytes < 8 * vpe::loss_max(1, vpe::clip_chunks(counts, n, vpe::clip_chunk(total))))
    return VPE_ERR_WORKSPACE;
  return launched(vpe::launch_grad_sumsq(tensors, counts, dtypes, n, total, sumsq,
                                         static_cast<double *>(workspace), stream));
}

vpe_status vpe_grad_clip(const void *const *tensors, const int64_t *counts, const int32_t *dtypes,
                         int32_t n, void *const *out, const double *const *sumsq, int32_t n_parts,
                         double max_norm, float *norm, void *stream) {
  int64_t total = 0;
  vpe_status rs = check_tensors(counts, n, &total);
  if (rs != VPE_OK) return rs;
  if (n_parts < 1 || n_parts > VPE_MAX_PARTS) return VPE_ERR_SHAPE;
  if (!(max_norm >= 0) || !isfinite(max_norm)) return VPE_ERR_RANGE;
  rs = check_tensor_pointers(tensors, counts, dtypes, n);
  if (rs != VPE_OK) return rs;
  if ((n > 0 && !out) || !sumsq || !norm) return VPE_ERR_NULL;
  for (int32_t i = 0; i < n; ++i) {
    if (counts[i] > 0 && !out[i]) return VPE_ERR_NULL;
    if (!aligned(out[i], dtype_bytes(static_cast<vpe_dtype>(dtypes[i])))) return VPE_ERR_ALIGN;
  }
  for (int32_t r = 0; r < n_parts; ++r) {
    if (!sumsq[r]) return VPE_ERR_NULL;
    if (!aligned(sumsq[r], 8)) return VPE_ERR_ALIGN;
  }
  if (!aligned(norm, 4)) return VPE_ERR_ALIGN;
  return launched(vpe::launch_grad_clip(tensors, counts, dtypes, n, total, out, sumsq, n_parts,
                                        max_norm, norm, stream));
}

}  // extern "C"
