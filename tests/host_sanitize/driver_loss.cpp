// Accept and reject paths of the loss calls at edge and overflow-prone sizes, in a
// build with address and undefined-behaviour sanitizers, against stand-ins for the
// kernel launchers that record what they were asked for.  Prints "all expectations
// held" when they did.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <limits>
#include <vector>

#include "../../vocab_sharded_embedding_amd/csrc/vpe_loss_launch.h"
#include "vpe_loss.h"

static const char *g_what = "";
static int64_t g_m, g_rows, g_ld;
static const void *g_p;
static bool g_add;

namespace vpe {

int launch_lmhead_xent(const LossRows &r, float *, float *, void *, void *) {
  g_what = "xent", g_m = r.m, g_rows = r.rows;
  return 0;
}
int launch_xent_loss(const float *const *, const float *const *, int, int64_t m, int64_t,
                     const void *, int, float *, float *, void *) {
  g_what = "xent_loss", g_m = m;
  return 0;
}
int launch_lmhead_xent_grad(const LossRows &r, const float *, const float *, const LossGrads &g,
                            void *, void *) {
  g_what = "xent_grad", g_m = r.m, g_rows = r.rows, g_add = g.accumulate;
  return 0;
}
int launch_lmhead_grad(const void *d, int64_t ld, const LossRows &r, const LossGrads &g, void *,
                       void *) {
  g_what = "head_grad", g_p = d, g_ld = ld, g_m = r.m, g_rows = r.rows, g_add = g.accumulate;
  return 0;
}
int launch_grad_sumsq(const void *const *, const int64_t *, const int32_t *, int n, int64_t total,
                      double *, double *, void *) {
  g_what = "sumsq", g_m = n, g_rows = total;
  return 0;
}
int launch_grad_clip(const void *const *, const int64_t *, const int32_t *, int n, int64_t total,
                     void *const *, const double *const *, int, double, float *, void *) {
  g_what = "clip", g_m = n, g_rows = total;
  return 0;
}

}  // namespace vpe

static int g_bad = 0;
#define EXPECT(cond)                            \
  do {                                          \
    if (!(cond)) {                              \
      ++g_bad;                                  \
      printf("line %d: %s\n", __LINE__, #cond); \
    }                                           \
  } while (0)

int main() {
  char *base = reinterpret_cast<char *>(uintptr_t(0x10000));
  void *p = base;
  float *f = reinterpret_cast<float *>(base);
  double *d64 = reinterpret_cast<double *>(base);
  const int64_t big = INT64_MAX;
  const int64_t sizes[] = {0,          1,  7, 65536, 1 << 21, 2147483647, int64_t(1) << 31,
                           int64_t(1) << 39, big - 1, big, -1, INT64_MIN};

  // every size in every place: no overflow, and nothing but a status
  for (int64_t a : sizes)
    for (int64_t b : sizes)
      for (int64_t c : sizes) {
        int64_t bytes = 0;
        (void)vpe_lmhead_xent_workspace(a, b, c, VPE_BF16, &bytes);
        (void)vpe_lmhead_xent_grad_workspace(a, b, c, VPE_F32, &bytes);
        (void)vpe_lmhead_grad_workspace(a, b, c, VPE_BF16, &bytes);
        for (int64_t d : sizes) {
          (void)vpe_lmhead_xent(p, a, b, p, c, VPE_BF16, d, a, p, VPE_I32, f, f, p, big, nullptr);
          (void)vpe_lmhead_xent(p, 7, 8, p, a, VPE_F32, b, c, p, VPE_I64, f, f, p, d, nullptr);
          (void)vpe_lmhead_xent_grad(p, a, b, p, c, VPE_F32, d, big, p, VPE_I32, f, f, p, VPE_F32,
                                     p, VPE_BF16, 1, p, big, nullptr);
          (void)vpe_lmhead_xent_grad(p, a, 64, p, b, VPE_BF16, c, d, p, VPE_I64, f, f, nullptr,
                                     VPE_F32, p, VPE_F32, 0, p, a, nullptr);
          (void)vpe_lmhead_grad(p, a, b, p, c, 64, p, d, VPE_BF16, p, VPE_BF16, p, VPE_F32, 0, p,
                                big, nullptr);
          (void)vpe_lmhead_grad(p, a, b, p, 7, c, p, d, VPE_F32, p, VPE_F32, nullptr, VPE_F32, 0,
                                p, big, nullptr);
          const int64_t counts[4] = {a, b, c, d};
          (void)vpe_grad_sumsq_workspace(counts, 4, &bytes);
          const void *in[4] = {p, p, p, p};
          void *out[4] = {p, p, p, p};
          const int32_t types[4] = {VPE_F32, VPE_BF16, VPE_F32, VPE_BF16};
          const double *sums[1] = {d64};
          (void)vpe_grad_sumsq(in, counts, types, 4, d64, p, a, nullptr);
          (void)vpe_grad_clip(in, counts, types, 4, out, sums, 1, 1.0, f, nullptr);
        }
        const float *parts[1] = {f};
        (void)vpe_xent_loss(parts, parts, 1, a, b, p, VPE_I64, f, f, nullptr);
      }

  // a workspace for more rows serves fewer, at every width of rows and shard
  for (vpe_dtype dt : {VPE_F32, VPE_BF16})
    for (int64_t dim : {1, 63, 64, 1000, 4096, 65536})
      for (int64_t rows : {int64_t(1), int64_t(255), int64_t(257), int64_t(75968),
                           int64_t(2000000)}) {
        int64_t last[3] = {0, 0, 0};
        for (int64_t m = 0; m <= VPE_MAX_LOSS_ROWS; m = m < 300 ? m + 1 : m * 5 / 4) {
          if (rows > (int64_t(1) << 42) / (m + 1)) break;
          int64_t need[3] = {0, 0, 0};
          EXPECT(vpe_lmhead_xent_workspace(m, dim, rows, dt, &need[0]) == VPE_OK);
          EXPECT(vpe_lmhead_xent_grad_workspace(m, dim, rows, dt, &need[1]) == VPE_OK);
          EXPECT(vpe_lmhead_grad_workspace(m, dim, rows, dt, &need[2]) == VPE_OK);
          for (int k = 0; k < 3; ++k) {
            EXPECT(need[k] >= last[k] && need[k] > 0);
            last[k] = need[k];
          }
          // what the launchers lay in it: parts in order, none over another
          for (vpe::LossCall call : {vpe::kLossForward, vpe::kLossGrad, vpe::kHeadGrad}) {
            const int code = dt == VPE_BF16 ? 1 : 0;
            const int64_t e = code ? 2 : 4;
            const vpe::LossLayout l = vpe::loss_layout(call, m, dim, rows, code);
            EXPECT(l.dim_pad >= dim && l.dim_pad % 64 == 0 && l.table_rows >= 256);
            EXPECT(l.table + l.table_rows * l.dim_pad * e <= l.bytes);
            if (call == vpe::kLossForward) continue;
            const int64_t splits = vpe::loss_most_splits(m, l.dim_pad, rows);
            EXPECT(splits >= 1 && l.sums + splits * m * l.dim_pad * 4 <= l.piece[0]);
            EXPECT(l.x + m * l.dim_pad * e <= l.sums);
            EXPECT(l.piece[0] + l.piece_cap <= (l.piece[1] > l.piece[0] ? l.piece[1] : l.table));
            EXPECT(l.piece[1] + l.piece_cap <= l.table);
            EXPECT(m == 0 || l.piece_cap / (m * e) >= vpe::loss_min(rows, vpe::kLossMinPiece));
          }
        }
      }

  // what is accepted reaches its launcher with the offsets applied
  int64_t need = 0;
  EXPECT(vpe_lmhead_xent_workspace(5, 8, 100, VPE_BF16, &need) == VPE_OK);
  EXPECT(vpe_lmhead_xent(p, 5, 8, p, 100, VPE_BF16, 100, 200, p, VPE_I32, f, f, p, need,
                         nullptr) == VPE_OK);
  EXPECT(!strcmp(g_what, "xent") && g_m == 5 && g_rows == 100);
  EXPECT(vpe_lmhead_xent(p, 5, 8, p, 100, VPE_BF16, 101, 200, p, VPE_I32, f, f, p, need,
                         nullptr) == VPE_ERR_RANGE);
  EXPECT(vpe_lmhead_xent(p, 5, 8, p, 100, VPE_BF16, 100, 200, p, VPE_I32, f, f, p, need - 1,
                         nullptr) == VPE_ERR_WORKSPACE);
  EXPECT(vpe_lmhead_xent(base + 1, 5, 8, p, 100, VPE_BF16, 100, 200, p, VPE_I32, f, f, p, need,
                         nullptr) == VPE_ERR_ALIGN);
  EXPECT(vpe_lmhead_xent(p, 5, 8, p, 100, VPE_BF16, 100, 200, p, VPE_I32, nullptr, f, p, need,
                         nullptr) == VPE_ERR_NULL);
  EXPECT(vpe_lmhead_grad_workspace(5, 8, 100, VPE_BF16, &need) == VPE_OK);
  EXPECT(vpe_lmhead_grad(p, 130, 30, p, 5, 8, p, 100, VPE_BF16, p, VPE_F32, p, VPE_F32, 1, p, need,
                         nullptr) == VPE_OK);
  EXPECT(!strcmp(g_what, "head_grad") && g_p == base + 60 && g_ld == 130 && g_add);
  EXPECT(vpe_lmhead_grad(p, 130, 31, p, 5, 8, p, 100, VPE_BF16, p, VPE_F32, p, VPE_F32, 1, p, need,
                         nullptr) == VPE_ERR_RANGE);
  // no rows: nothing to add; a gradient that is not added to is cleared
  g_what = "";
  EXPECT(vpe_lmhead_grad(nullptr, 130, 30, nullptr, 0, 8, p, 100, VPE_BF16, p, VPE_F32, p, VPE_F32,
                         1, nullptr, 0, nullptr) == VPE_OK);
  EXPECT(!strcmp(g_what, ""));
  EXPECT(vpe_lmhead_grad(nullptr, 130, 30, nullptr, 0, 8, p, 100, VPE_BF16, p, VPE_F32, p, VPE_F32,
                         0, p, need, nullptr) == VPE_OK);
  EXPECT(!strcmp(g_what, "head_grad") && g_p == nullptr);

  // many tensors, the arrays read to their last entry
  const int n = VPE_MAX_GRAD_TENSORS;
  std::vector<int64_t> counts(n, 3);
  std::vector<const void *> in(n, p);
  std::vector<void *> out(n, p);
  std::vector<int32_t> types(n, VPE_BF16);
  const double *sums[1] = {d64};
  EXPECT(vpe_grad_sumsq_workspace(counts.data(), n, &need) == VPE_OK && need == 8 * int64_t(n));
  EXPECT(vpe_grad_sumsq(in.data(), counts.data(), types.data(), n, d64, p, need, nullptr) ==
         VPE_OK);
  EXPECT(!strcmp(g_what, "sumsq") && g_m == n && g_rows == 3 * int64_t(n));
  EXPECT(vpe_grad_sumsq(in.data(), counts.data(), types.data(), n, d64, p, need - 1, nullptr) ==
         VPE_ERR_WORKSPACE);
  EXPECT(vpe_grad_clip(in.data(), counts.data(), types.data(), n, out.data(), sums, 1, 1.0, f,
                       nullptr) == VPE_OK);
  EXPECT(vpe_grad_clip(in.data(), counts.data(), types.data(), n + 1, out.data(), sums, 1, 1.0, f,
                       nullptr) == VPE_ERR_SHAPE);
  for (double norm : {-1.0, std::numeric_limits<double>::infinity(),
                      std::numeric_limits<double>::quiet_NaN()})
    EXPECT(vpe_grad_clip(in.data(), counts.data(), types.data(), n, out.data(), sums, 1, norm, f,
                         nullptr) == VPE_ERR_RANGE);

  if (g_bad) return 1;
  printf("all expectations held\n");
  return 0;
}
