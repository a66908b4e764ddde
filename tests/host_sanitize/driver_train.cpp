// Accept and reject paths of the training and beam-search calls at edge and
// overflow-prone sizes, in a build with address and undefined-behaviour
// sanitizers.  Prints "all expectations held" when they did.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <limits>

#include "vpe_beam.h"
#include "vpe_train.h"
#include "stub_train_record.h"

static int g_bad = 0;
#define EXPECT(cond)                                                   \
  do {                                                                 \
    if (!(cond)) {                                                     \
      ++g_bad;                                                         \
      printf("line %d: %s\n", __LINE__, #cond);                        \
    }                                                                  \
  } while (0)

int main() {
  void *p = reinterpret_cast<void *>(uintptr_t(0x10000));
  char *far_p = reinterpret_cast<char *>(uintptr_t(0x700000000000));
  float *f = static_cast<float *>(p);
  const int64_t big = INT64_MAX, sizes[] = {0, 1, 7, 2147483647, int64_t(1) << 31,
                                            int64_t(1) << 39, big - 1, big, -1, INT64_MIN};
  const float inf = std::numeric_limits<float>::infinity();

  // every size in every place: no overflow, and nothing but a status
  for (int64_t a : sizes)
    for (int64_t b : sizes)
      for (int64_t c : sizes) {
        int64_t bytes = 0;
        (void)vpe_embed_scaled(p, VPE_I32, a, p, VPE_BF16, b, c, a, 1.f, p, nullptr);
        (void)vpe_embed_scaled(p, VPE_I64, a, p, VPE_F32, b, 8, c, -1.f, p, nullptr);
        (void)vpe_embed_grad_workspace(a, b, c, &bytes);
        (void)vpe_embed_grad(p, VPE_I32, a, p, VPE_F32, c, a, b, 1.f, p, VPE_BF16, 0, p, big,
                             nullptr);
        (void)vpe_embed_grad(p, VPE_I64, a, p, VPE_BF16, 8, c, b, 1.f, p, VPE_F32, 1, p, b,
                             nullptr);
        (void)vpe_distill_workspace(a, b, &bytes);
        (void)vpe_distill_shard(p, a, b, 3, c, VPE_F32, a, b, 1.f, p, VPE_I32, p, VPE_F32, 4, f, f,
                                f, p, c, nullptr);
        (void)vpe_distill_shard(p, a, 0, c, b, VPE_BF16, c, a, 1.f, p, VPE_I32, p, VPE_F32, 4,
                                nullptr, f, f, p, big, nullptr);
        (void)vpe_distill_grad(p, a, b, 3, c, VPE_BF16, b, a, 2.f, p, VPE_I64, p, VPE_BF16, 4, f,
                               f, f, far_p, b, a, nullptr);
        (void)vpe_distill_grad(p, a, b, c, 5, VPE_BF16, 0, a, 2.f, p, VPE_I64, p, VPE_BF16, 4, f,
                               f, f, p, b, c, nullptr);
        (void)vpe_beam_select_workspace(a, 4, b, 4, &bytes);
        (void)vpe_beam_select(p, a, b, VPE_F32, 2, 4, c, a, b, f, f, 4,
                              static_cast<uint64_t *>(p), p, big, nullptr);
        (void)vpe_beam_select(p, a, 0, VPE_BF16, b, 64, c, 0, a, f, f, 64,
                              static_cast<uint64_t *>(p), p, c, nullptr);
        (void)vpe_beam_reorder(p, a, b, 4, c, static_cast<int64_t *>(p), a, 4, far_p, nullptr);
        (void)vpe_beam_reorder(p, a, 3, 2147483647, b, static_cast<int64_t *>(p), c, 2147483647,
                               far_p, nullptr);
        const uint64_t *keys[2] = {static_cast<uint64_t *>(p), static_cast<uint64_t *>(p)};
        (void)vpe_beam_merge(keys, 2, a, 8, b, f, static_cast<int64_t *>(p),
                             static_cast<int64_t *>(p), nullptr);
      }

  // what is accepted reaches its launcher with the offsets applied
  EXPECT(vpe_embed_scaled(p, VPE_I64, 5, p, VPE_BF16, 10, 3, 7, 2.f, p, nullptr) == VPE_OK);
  EXPECT(!strcmp(g_train.what, "embed_scaled") && g_train.n0 == 5 && g_train.n1 == 10 &&
         g_train.n2 == 3 && g_train.n3 == 7 && g_train.i0 == 1 && g_train.i1 == 1);
  EXPECT(vpe_embed_scaled(p, VPE_I64, 5, p, VPE_BF16, 10, 3, 7, inf, p, nullptr) ==
         VPE_ERR_RANGE);
  int64_t need = 0;
  EXPECT(vpe_embed_grad_workspace(100, 50, 8, &need) == VPE_OK && need > 0);
  EXPECT(vpe_embed_grad(p, VPE_I32, 100, p, VPE_BF16, 8, 0, 50, 1.f, p, VPE_F32, 1, p, need,
                        nullptr) == VPE_OK);
  EXPECT(!strcmp(g_train.what, "embed_grad") && g_train.i1 == 1 + 4);
  EXPECT(vpe_embed_grad(p, VPE_I32, 100, p, VPE_BF16, 8, 0, 50, 1.f, p, VPE_F32, 1, p, need - 1,
                        nullptr) == VPE_ERR_WORKSPACE);
  // a workspace for more ids serves fewer
  int64_t last = 0;
  for (int64_t n = 0; n < 300000; n = n < 100 ? n + 1 : n * 9 / 8) {
    EXPECT(vpe_embed_grad_workspace(n, 1000, 24, &need) == VPE_OK && need >= last);
    last = need;
  }
  EXPECT(vpe_distill_workspace(3, 5000, &need) == VPE_OK && need == 3 * 5 * 8);
  EXPECT(vpe_distill_shard(p, 6000, 10, 3, 5000, VPE_BF16, 0, 5000, 1.f, p, VPE_I64, p, VPE_F32, 9,
                           nullptr, f, f, p, need, nullptr) == VPE_OK);
  EXPECT(!strcmp(g_train.what, "distill_shard") &&
         g_train.p == static_cast<void *>(static_cast<char *>(p) + 20));
  EXPECT(vpe_distill_shard(p, 6000, 10, 3, 5000, VPE_BF16, 0, 5000, 1.f, p, VPE_I64, p, VPE_F32, 9,
                           nullptr, nullptr, f, nullptr, 0, nullptr) == VPE_OK);
  // in place, beside the logits in their buffer, and half over them
  EXPECT(vpe_distill_grad(p, 20, 0, 3, 10, VPE_F32, 0, 10, 1.f, p, VPE_I64, p, VPE_F32, 2, nullptr,
                          f, f, p, 20, 0, nullptr) == VPE_OK);
  EXPECT(vpe_distill_grad(p, 20, 0, 3, 10, VPE_F32, 0, 10, 1.f, p, VPE_I64, p, VPE_F32, 2, nullptr,
                          f, f, p, 20, 10, nullptr) == VPE_OK);
  EXPECT(g_train.p == static_cast<void *>(static_cast<char *>(p) + 40));
  EXPECT(vpe_distill_grad(p, 20, 10, 3, 10, VPE_F32, 0, 10, 1.f, p, VPE_I64, p, VPE_F32, 2,
                          nullptr, f, f, p, 20, 0, nullptr) == VPE_OK);
  EXPECT(vpe_distill_grad(p, 20, 0, 3, 10, VPE_F32, 0, 10, 1.f, p, VPE_I64, p, VPE_F32, 2, nullptr,
                          f, f, p, 20, 9, nullptr) == VPE_ERR_RANGE);
  EXPECT(vpe_distill_grad(p, 20, 10, 3, 10, VPE_F32, 0, 10, 1.f, p, VPE_I64, p, VPE_F32, 2,
                          nullptr, f, f, p, 20, 1, nullptr) == VPE_ERR_RANGE);
  EXPECT(vpe_distill_grad(p, 20, 0, 3, 10, VPE_F32, 0, 10, 1.f, p, VPE_I64, p, VPE_F32, 2, nullptr,
                          f, f, p, 21, 0, nullptr) == VPE_ERR_RANGE);
  EXPECT(vpe_distill_grad(p, 20, 0, 3, 10, VPE_F32, 0, 10, 1.f, p, VPE_I64, p, VPE_F32, 2, nullptr,
                          f, f, static_cast<char *>(p) + 160, 20, 0, nullptr) == VPE_ERR_RANGE);
  EXPECT(vpe_distill_grad(p, 20, 0, 3, 10, VPE_F32, 0, 10, 1.f, p, VPE_I64, p, VPE_F32, 2, nullptr,
                          f, f, static_cast<char *>(p) + 240, 20, 0, nullptr) == VPE_OK);
  // a single row in place, whatever the strides; past the largest temperature
  EXPECT(vpe_distill_grad(p, 20, 0, 1, 10, VPE_F32, 0, 10, 1.f, p, VPE_I64, p, VPE_F32, 2, nullptr,
                          f, f, p, 10, 0, nullptr) == VPE_OK);
  EXPECT(vpe_distill_grad(p, 20, 0, 1, 10, VPE_F32, 0, 10, 0x1.8p100f, p, VPE_I64, p, VPE_F32, 2,
                          nullptr, f, f, p, 10, 0, nullptr) == VPE_ERR_RANGE);
  const float *two[2] = {f, f};
  EXPECT(vpe_distill_loss(two, two, 2, 4, 10, 1.f, p, VPE_I32, p, VPE_BF16, 3, nullptr, f, f,
                          nullptr) == VPE_OK);
  EXPECT(vpe_beam_select_workspace(2, 4, 100, 8, &need) == VPE_OK && need == 2 * 4 * 4 * 4);
  EXPECT(vpe_beam_select(p, 100, 0, VPE_F32, 2, 4, 100, 0, 100, f, f, 8,
                         static_cast<uint64_t *>(p), p, need, nullptr) == VPE_OK);
  EXPECT(vpe_beam_select(p, 100, 0, VPE_F32, 2, 4, 100, 0, int64_t(1) << 30, f, f, 8,
                         static_cast<uint64_t *>(p), p, need, nullptr) == VPE_ERR_RANGE);
  EXPECT(vpe_beam_select(p, 100, 0, VPE_F32, 2, 4, 100, 0, (int64_t(1) << 30) - 1, f, f, 8,
                         static_cast<uint64_t *>(p), p, need, nullptr) == VPE_OK);
  EXPECT(vpe_beam_reorder(p, 2, 3, 4, 5, static_cast<int64_t *>(p), 8, 6, far_p, nullptr) ==
         VPE_OK);
  EXPECT(!strcmp(g_train.what, "beam_reorder") && g_train.n3 == 8 && g_train.i1 == 6);
  if (g_bad == 0) printf("all expectations held\n");
  return g_bad == 0 ? 0 : 1;
}
