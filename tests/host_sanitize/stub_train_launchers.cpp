// Host-only stand-ins for the launchers of the training and beam-search calls,
// for the sanitized build of their validation layers: each records its name
// and sizes and touches no memory behind the pointers it receives.
#include <stdint.h>

#include "../../vocab_sharded_embedding_amd/csrc/vpe_train_launch.h"
#include "stub_train_record.h"

stub_train_call g_train;

namespace vpe {

int launch_embed_scaled(const void *, int itype, int64_t n, const void *, int dtype,
                        int64_t shard_rows, int64_t dim, int64_t vocab_start, float, void *,
                        void *) {
  g_train = stub_train_call{"embed_scaled", n, shard_rows, dim, vocab_start, itype, dtype};
  return 0;
}
int launch_embed_grad(const void *, int itype, int64_t n, const void *, int dtype, int64_t dim,
                      int64_t vocab_start, int64_t shard_rows, float, void *, int gdtype,
                      bool accumulate, void *, void *) {
  g_train = stub_train_call{"embed_grad", n, shard_rows, dim, vocab_start, itype,
                            dtype + 2 * gdtype + 4 * accumulate};
  return 0;
}
int64_t distill_pairs_per_row(int64_t cols, int dtype) {
  const int64_t per = dtype == 1 ? 2048 : 1024;
  return (cols + per - 1) / per;
}
int launch_distill_shard(const LogitsShard &z, const Teacher &t, float *, float *, float *,
                         void *) {
  g_train = stub_train_call{"distill_shard", z.m, z.cols, z.ld, t.vocab, t.k, z.dtype, z.base};
  return 0;
}
int launch_distill_loss(const float *const *, const float *const *, int n_parts, int64_t m,
                        const Teacher &t, float *, float *, void *) {
  g_train = stub_train_call{"distill_loss", m, n_parts, 0, t.vocab, t.k, t.dtype};
  return 0;
}
int launch_distill_grad(const LogitsShard &z, const Teacher &t, const float *, const float *,
                        void *grad, int64_t ld_grad, void *) {
  g_train = stub_train_call{"distill_grad", z.m, z.cols, ld_grad, t.vocab, t.k, z.dtype, grad};
  return 0;
}
int64_t beam_groups_per_row(int, int64_t cols, int) { return (cols + 31) / 32; }
int launch_beam_select(const void *base, int64_t ld, int dtype, int64_t n_seqs, int beams,
                       int64_t cols, int64_t, int64_t vocab, const float *, const float *,
                       int picks, uint64_t *, float *, void *) {
  g_train = stub_train_call{"beam_select", n_seqs * beams, cols, ld, vocab, picks, dtype, base};
  return 0;
}
int launch_beam_merge(const uint64_t *const *, int n_parts, int64_t n_seqs, int picks,
                      int64_t vocab, float *, int64_t *, int64_t *, void *) {
  g_train = stub_train_call{"beam_merge", n_seqs, n_parts, 0, vocab, picks, 0};
  return 0;
}
int launch_beam_reorder(const void *, int64_t outer, int64_t n_seqs, int beams_in,
                        int64_t row_bytes, const int64_t *, int64_t ld_parent, int beams_out,
                        void *, void *) {
  g_train = stub_train_call{"beam_reorder", outer, n_seqs, row_bytes, ld_parent, beams_in,
                            beams_out};
  return 0;
}

}  // namespace vpe
