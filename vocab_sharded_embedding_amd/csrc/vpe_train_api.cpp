// The C ABI of the training calls (include/vpe_train.h): argument validation
// and dispatch to the kernel launchers, as vpe_api.cpp does for vpe.h.  Plain
// C++ with no HIP headers: a rejected call enqueues nothing.
#include "../../include/vpe_train.h"

#include <float.h>
#include <math.h>
#include <stdint.h>

#include "vpe_train_launch.h"

namespace {

bool known_dtype(vpe_dtype dt) { return dt == VPE_F32 || dt == VPE_BF16; }
bool known_itype(vpe_itype it) { return it == VPE_I32 || it == VPE_I64; }
int64_t dtype_bytes(vpe_dtype dt) { return dt == VPE_F32 ? 4 : 2; }
int64_t itype_bytes(vpe_itype it) { return it == VPE_I32 ? 4 : 8; }

bool aligned(const void *p, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes)) == 0;
}

vpe_status launched(int rc) { return rc == 0 ? VPE_OK : VPE_ERR_LAUNCH; }

// Largest element count of any one tensor (indexes in the kernels are 64-bit).
constexpr int64_t kMaxElems = int64_t(1) << 39;

// Largest number of ids, and of shard rows, whose sort keys are 32-bit.
constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;

bool embed_grad_shape_ok(int64_t n, int64_t shard_rows, int64_t dim) {
  return n >= 0 && n <= kMax31 && dim >= 1 && dim <= (int64_t(1) << 20) && shard_rows >= 1 &&
         shard_rows <= kMax31 && n <= kMaxElems / dim && shard_rows <= kMaxElems / dim;
}

// What vpe_distill_shard, _loss and _grad check alike.
vpe_status check_teacher(int64_t m, int64_t vocab, float temperature, vpe_itype itype,
                         vpe_dtype tdt, int32_t k) {
  if (!known_dtype(tdt) || !known_itype(itype)) return VPE_ERR_DTYPE;
  if (m < 0 || m > VPE_MAX_DISTILL_ROWS || k < 1 || k > VPE_MAX_TEACHER_ENTRIES || vocab < 1)
    return VPE_ERR_SHAPE;
  // log2(e) / temperature, the factor of the powers of two, has to be finite in
  // fp32 as well (so 1 / temperature is), and any log-sum-exp times temperature
  if (!(temperature > 0.f) || temperature > 0x1p100f ||
      1.4426950408889634 / static_cast<double>(temperature) > static_cast<double>(FLT_MAX))
    return VPE_ERR_RANGE;
  return VPE_OK;
}

vpe_status check_shard(int64_t ld, int64_t col_offset, int64_t m, int64_t shard_rows,
                       vpe_dtype dt, int64_t vocab_start, int64_t vocab) {
  if (!known_dtype(dt)) return VPE_ERR_DTYPE;
  if (shard_rows < 1 || shard_rows > kMax31) return VPE_ERR_SHAPE;
  if (vocab_start < 0 || vocab_start > vocab || shard_rows > vocab - vocab_start)
    return VPE_ERR_RANGE;
  if (col_offset < 0 || ld < 1 || shard_rows > ld - col_offset) return VPE_ERR_RANGE;
  if (m > kMaxElems / ld) return VPE_ERR_SHAPE;
  return VPE_OK;
}

// Whether rows of `cols` elements at a (stride ld_a) and at b (stride ld_b) share
// bytes, unless they are the same rows.
bool partly_overlap(const char *a, int64_t ld_a, const char *b, int64_t ld_b, int64_t m,
                    int64_t cols, int64_t size) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + static_cast<uintptr_t>(((m - 1) * ld_a + cols) * size);
  const uintptr_t b1 = b0 + static_cast<uintptr_t>(((m - 1) * ld_b + cols) * size);
  if (b1 <= a0 || a1 <= b0) return false;
  if (a0 == b0 && m == 1) return false;
  if (ld_a != ld_b) return true;
  // one stride: other columns of the same rows are apart
  const uintptr_t row = static_cast<uintptr_t>(ld_a * size), width = static_cast<uintptr_t>(cols * size);
  const uintptr_t off = b0 >= a0 ? (b0 - a0) % row : (row - (a0 - b0) % row) % row;
  if (a0 == b0) return false;
  return off < width || off > row - width;
}

vpe_status check_teacher_pointers(const void *ids, vpe_itype itype, const void *teacher,
                                  vpe_dtype tdt, const float *teacher_lse) {
  if (!ids || !teacher) return VPE_ERR_NULL;
  if (!aligned(ids, itype_bytes(itype)) || !aligned(teacher, dtype_bytes(tdt)) ||
      !aligned(teacher_lse, 4))
    return VPE_ERR_ALIGN;
  return VPE_OK;
}

vpe::Teacher teacher_of(const void *ids, vpe_itype itype, const void *teacher, vpe_dtype tdt,
                        int32_t k, const float *teacher_lse, int64_t vocab, float temperature) {
  return vpe::Teacher{ids, teacher, teacher_lse, itype == VPE_I32 ? 0 : 1, tdt == VPE_BF16 ? 1 : 0,
                      k, vocab, temperature};
}

vpe::LogitsShard shard_of(const void *logits, int64_t ld, int64_t col_offset, int64_t m,
                          int64_t shard_rows, vpe_dtype dt, int64_t vocab_start) {
  return vpe::LogitsShard{static_cast<const char *>(logits) + col_offset * dtype_bytes(dt), ld, m,
                          shard_rows, vocab_start, dt == VPE_BF16 ? 1 : 0};
}

}  // namespace

extern "C" {

vpe_status vpe_embed_scaled(const void *ids, vpe_itype itype, int64_t n, const void *weight,
                            vpe_dtype dt, int64_t shard_rows, int64_t dim, int64_t vocab_start,
                            float scale, void *out, void *stream) {
  if (!known_dtype(dt) || !known_itype(itype)) return VPE_ERR_DTYPE;
  if (n < 0 || dim < 1 || shard_rows < 1) return VPE_ERR_SHAPE;
  if (n > kMaxElems / dim || shard_rows > kMaxElems / dim) return VPE_ERR_SHAPE;
  if (vocab_start < 0 || vocab_start > INT64_MAX - shard_rows || !isfinite(scale))
    return VPE_ERR_RANGE;
  if (n == 0) return VPE_OK;
  if (!ids || !weight || !out) return VPE_ERR_NULL;
  if (!aligned(ids, itype_bytes(itype)) || !aligned(weight, dtype_bytes(dt)) ||
      !aligned(out, dtype_bytes(dt)))
    return VPE_ERR_ALIGN;
  return launched(vpe::launch_embed_scaled(ids, itype == VPE_I32 ? 0 : 1, n, weight,
                                           dt == VPE_BF16 ? 1 : 0, shard_rows, dim, vocab_start,
                                           scale, out, stream));
}

vpe_status vpe_embed_grad_workspace(int64_t n, int64_t shard_rows, int64_t dim, int64_t *bytes) {
  if (!bytes) return VPE_ERR_NULL;
  if (!embed_grad_shape_ok(n, shard_rows, dim)) return VPE_ERR_SHAPE;
  *bytes = vpe::embed_grad_layout(n, shard_rows, dim).bytes;
  return VPE_OK;
}

vpe_status vpe_embed_grad(const void *ids, vpe_itype itype, int64_t n, const void *grad_out,
                          vpe_dtype dt, int64_t dim, int64_t vocab_start, int64_t shard_rows,
                          float scale, void *grad_weight, vpe_dtype gdt, int32_t accumulate,
                          void *workspace, int64_t workspace_bytes, void *stream) {
  if (!known_dtype(dt) || !known_dtype(gdt) || !known_itype(itype)) return VPE_ERR_DTYPE;
  if (!embed_grad_shape_ok(n, shard_rows, dim) || workspace_bytes < 0) return VPE_ERR_SHAPE;
  if (vocab_start < 0 || vocab_start > INT64_MAX - shard_rows || !isfinite(scale))
    return VPE_ERR_RANGE;
  if (n == 0 && accumulate != 0) return VPE_OK;
  if (!grad_weight || !workspace || (n > 0 && (!ids || !grad_out))) return VPE_ERR_NULL;
  if (!aligned(ids, itype_bytes(itype)) || !aligned(grad_out, dtype_bytes(dt)) ||
      !aligned(grad_weight, dtype_bytes(gdt)) || !aligned(workspace, 16))
    return VPE_ERR_ALIGN;
  if (workspace_bytes < vpe::embed_grad_layout(n, shard_rows, dim).bytes)
    return VPE_ERR_WORKSPACE;
  return launched(vpe::launch_embed_grad(ids, itype == VPE_I32 ? 0 : 1, n, grad_out,
                                         dt == VPE_BF16 ? 1 : 0, dim, vocab_start, shard_rows,
                                         scale, grad_weight, gdt == VPE_BF16 ? 1 : 0,
                                         accumulate != 0, workspace, stream));
}

vpe_status vpe_distill_workspace(int64_t m, int64_t shard_rows, int64_t *bytes) {
  if (!bytes) return VPE_ERR_NULL;
  if (m < 0 || m > VPE_MAX_DISTILL_ROWS || shard_rows < 1 || shard_rows > kMax31)
    return VPE_ERR_SHAPE;
  const int64_t rows = m < vpe::kDistillWholeRows ? m : vpe::kDistillWholeRows - 1;
  *bytes = rows * vpe::distill_pairs_per_row(shard_rows, 0) * 8;
  return VPE_OK;
}

vpe_status vpe_distill_shard(const void *logits, int64_t ld, int64_t col_offset, int64_t m,
                             int64_t shard_rows, vpe_dtype dt, int64_t vocab_start, int64_t vocab,
                             float temperature, const void *teacher_ids, vpe_itype itype,
                             const void *teacher, vpe_dtype tdt, int32_t k,
                             const float *teacher_lse, float *shard_lse, float *shard_dot,
                             void *workspace, int64_t workspace_bytes, void *stream) {
  vpe_status rs = check_teacher(m, vocab, temperature, itype, tdt, k);
  if (rs != VPE_OK) return rs;
  rs = check_shard(ld, col_offset, m, shard_rows, dt, vocab_start, vocab);
  if (rs != VPE_OK) return rs;
  if (workspace_bytes < 0) return VPE_ERR_SHAPE;
  if (m == 0) return VPE_OK;
  if (!logits || !shard_dot) return VPE_ERR_NULL;
  rs = check_teacher_pointers(teacher_ids, itype, teacher, tdt, teacher_lse);
  if (rs != VPE_OK) return rs;
  if (!aligned(logits, dtype_bytes(dt)) || !aligned(shard_lse, 4) || !aligned(shard_dot, 4) ||
      !aligned(workspace, 8))
    return VPE_ERR_ALIGN;
  static_assert(vpe::kDistillWholeRows == VPE_DISTILL_WHOLE_ROWS, "rows without pairs in memory");
  if (shard_lse && m < VPE_DISTILL_WHOLE_ROWS) {
    int64_t need = 0;
    rs = vpe_distill_workspace(m, shard_rows, &need);
    if (rs != VPE_OK) return rs;
    if (!workspace) return VPE_ERR_NULL;
    if (workspace_bytes < need) return VPE_ERR_WORKSPACE;
  }
  return launched(vpe::launch_distill_shard(
      shard_of(logits, ld, col_offset, m, shard_rows, dt, vocab_start),
      teacher_of(teacher_ids, itype, teacher, tdt, k, teacher_lse, vocab, temperature), shard_lse,
      shard_dot, static_cast<float *>(workspace), stream));
}

vpe_status vpe_distill_loss(const float *const *shard_lse, const float *const *shard_dot,
                            int32_t n_parts, int64_t m, int64_t vocab, float temperature,
                            const void *teacher_ids, vpe_itype itype, const void *teacher,
                            vpe_dtype tdt, int32_t k, const float *teacher_lse, float *loss,
                            float *lse, void *stream) {
  vpe_status rs = check_teacher(m, vocab, temperature, itype, tdt, k);
  if (rs != VPE_OK) return rs;
  if (n_parts < 1 || n_parts > VPE_MAX_PARTS) return VPE_ERR_SHAPE;
  if (m == 0) return VPE_OK;
  if (!shard_lse || !shard_dot || !loss || !lse) return VPE_ERR_NULL;
  for (int32_t r = 0; r < n_parts; ++r) {
    if (!shard_lse[r] || !shard_dot[r]) return VPE_ERR_NULL;
    if (!aligned(shard_lse[r], 4) || !aligned(shard_dot[r], 4)) return VPE_ERR_ALIGN;
  }
  rs = check_teacher_pointers(teacher_ids, itype, teacher, tdt, teacher_lse);
  if (rs != VPE_OK) return rs;
  if (!aligned(loss, 4) || !aligned(lse, 4)) return VPE_ERR_ALIGN;
  return launched(vpe::launch_distill_loss(
      shard_lse, shard_dot, n_parts, m,
      teacher_of(teacher_ids, itype, teacher, tdt, k, teacher_lse, vocab, temperature), loss, lse,
      stream));
}

vpe_status vpe_distill_grad(const void *logits, int64_t ld, int64_t col_offset, int64_t m,
                            int64_t shard_rows, vpe_dtype dt, int64_t vocab_start, int64_t vocab,
                            float temperature, const void *teacher_ids, vpe_itype itype,
                            const void *teacher, vpe_dtype tdt, int32_t k,
                            const float *teacher_lse, const float *lse, const float *grad_loss,
                            void *grad_logits, int64_t ld_grad, int64_t grad_col_offset,
                            void *stream) {
  vpe_status rs = check_teacher(m, vocab, temperature, itype, tdt, k);
  if (rs != VPE_OK) return rs;
  rs = check_shard(ld, col_offset, m, shard_rows, dt, vocab_start, vocab);
  if (rs != VPE_OK) return rs;
  rs = check_shard(ld_grad, grad_col_offset, m, shard_rows, dt, vocab_start, vocab);
  if (rs != VPE_OK) return rs;
  if (m == 0) return VPE_OK;
  if (!logits || !lse || !grad_loss || !grad_logits) return VPE_ERR_NULL;
  rs = check_teacher_pointers(teacher_ids, itype, teacher, tdt, teacher_lse);
  if (rs != VPE_OK) return rs;
  if (!aligned(logits, dtype_bytes(dt)) || !aligned(grad_logits, dtype_bytes(dt)) ||
      !aligned(lse, 4) || !aligned(grad_loss, 4))
    return VPE_ERR_ALIGN;
  const int64_t size = dtype_bytes(dt);
  char *base = static_cast<char *>(grad_logits) + grad_col_offset * size;
  if (partly_overlap(static_cast<const char *>(logits) + col_offset * size, ld, base, ld_grad, m,
                     shard_rows, size))
    return VPE_ERR_RANGE;
  return launched(vpe::launch_distill_grad(
      shard_of(logits, ld, col_offset, m, shard_rows, dt, vocab_start),
      teacher_of(teacher_ids, itype, teacher, tdt, k, teacher_lse, vocab, temperature), lse,
      grad_loss, base, ld_grad, stream));
}

}  // extern "C"
