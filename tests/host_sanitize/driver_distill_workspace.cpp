// Which distillation calls ask for a workspace, against host stand-ins for the
// launchers.  Prints "all expectations held" when they did.
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "vpe_train.h"

int main() {
  void *p = reinterpret_cast<void *>(uintptr_t(0x10000));
  float *f = static_cast<float *>(p);
  int bad = 0;
  for (int64_t m : {int64_t(1), int64_t(255), int64_t(256), int64_t(1000), int64_t(1) << 21})
    for (vpe_dtype dt : {VPE_F32, VPE_BF16})
      for (int64_t bytes : {int64_t(0), int64_t(8)}) {
        // 149 (75) slices: more than a workgroup takes of a few rows
        const vpe_status rs =
            vpe_distill_shard(p, 151936, 0, m, 151936, dt, 0, 151936, 1.f, p, VPE_I64, p, VPE_F32, 4,
                              nullptr, f, f, bytes ? p : nullptr, bytes, nullptr);
        const vpe_status want =
            m >= VPE_DISTILL_WHOLE_ROWS ? VPE_OK : bytes ? VPE_ERR_WORKSPACE : VPE_ERR_NULL;
        if (rs != want) ++bad, printf("m %lld bytes %lld: %d\n", (long long)m, (long long)bytes, rs);
      }
  // a workspace for any number of rows serves fewer
  int64_t last = 0, need = 0;
  for (int64_t m = 0; m < 400; ++m) {
    if (vpe_distill_workspace(m, 151936, &need) != VPE_OK || need < last) ++bad;
    last = need;
  }
  if (bad == 0) printf("all expectations held\n");
  return bad == 0 ? 0 : 1;
}
