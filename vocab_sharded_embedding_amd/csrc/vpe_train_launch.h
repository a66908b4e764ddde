// Internal interface between the validating C-ABI layer of the training and
// beam-search calls (vpe_train_api.cpp, vpe_beam_api.cpp: plain C++ with no HIP
// headers) and their kernel launchers (*.hip).  As in vpe_launch.h, launchers
// receive validated arguments, enqueue on `stream` and return 0 or the
// hipError_t value the runtime reported.  dtype: 0 = f32, 1 = bf16; itype:
// 0 = int32, 1 = int64.
#ifndef VPE_TRAIN_LAUNCH_H
#define VPE_TRAIN_LAUNCH_H

#include <stdint.h>

namespace vpe {

// ---------------------------------------------------------------------------
// scaled lookup and its gradient
// ---------------------------------------------------------------------------
int launch_embed_scaled(const void *ids, int itype, int64_t n, const void *weight, int dtype,
                        int64_t shard_rows, int64_t dim, int64_t vocab_start, float scale,
                        void *out, void *stream);

// Sorted positions are summed in pieces that end at multiples of this.
constexpr int64_t kGradPiece = 32;
// Up to this many ids are sorted by one workgroup.
constexpr int64_t kGradOneBlockIds = 8192;
// Workgroups and digit values of one pass of the sort of more ids.
constexpr int64_t kSortMaxBlocks = 128;
constexpr int64_t kSortTile = 2048;
constexpr int64_t kSortDigits = 512;

// Byte offsets of the gradient's workspace (all 16-byte aligned).
struct EmbedGradLayout {
  int64_t count;    // uint32: owned ids
  int64_t hist;     // uint32 [2][kSortMaxBlocks][kSortDigits]
  int64_t flags;    // uint8 [shard_rows]: the row has an id
  int64_t key[2];   // uint32 [n]
  int64_t pos[2];   // uint32 [n]
  int64_t partial;  // float [2 * pieces][dim]
  int64_t bytes;
};

constexpr int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

inline EmbedGradLayout embed_grad_layout(int64_t n, int64_t shard_rows, int64_t dim) {
  EmbedGradLayout l{};
  int64_t at = 0;
  l.count = at, at += 16;
  l.hist = at, at += n > kGradOneBlockIds ? 2 * kSortMaxBlocks * kSortDigits * 4 : 0;
  l.flags = at, at += round16(shard_rows);
  for (int b = 0; b < 2; ++b) {
    l.key[b] = at, at += round16(n * 4);
    l.pos[b] = at, at += round16(n * 4);
  }
  // at most one piece that starts and one that continues per piece boundary
  l.partial = at, at += n > kGradPiece ? 2 * ((n + kGradPiece - 1) / kGradPiece) * dim * 4 : 0;
  l.bytes = round16(at);
  return l;
}

int launch_embed_grad(const void *ids, int itype, int64_t n, const void *grad_out, int dtype,
                      int64_t dim, int64_t vocab_start, int64_t shard_rows, float scale,
                      void *grad_weight, int gdtype, bool accumulate, void *workspace,
                      void *stream);

// ---------------------------------------------------------------------------
// distillation
// ---------------------------------------------------------------------------
// A batch of teacher entries and the vocabulary they refer to.
struct Teacher {
  const void *ids;
  const void *logits;
  const float *lse;  // nullptr: normalised over the entries
  int itype;
  int dtype;
  int k;
  int64_t vocab;
  float temperature;
};

// One shard's columns of the student's logits: row i starts at base + i * ld
// (elements; base already includes the column offset).
struct LogitsShard {
  const void *base;
  int64_t ld;
  int64_t m;
  int64_t cols;
  int64_t vocab_start;
  int dtype;
};

// Column slices a row is cut into when there are few rows, for the pass that
// reduces it: (maximum, sum) pairs [m][slices] in the workspace.
int64_t distill_slices(int64_t m, int64_t cols);

int launch_distill_shard(const LogitsShard &z, const Teacher &t, float *shard_lse,
                         float *shard_dot, float *pairs, void *stream);
int launch_distill_loss(const float *const *shard_lse, const float *const *shard_dot, int n_parts,
                        int64_t m, const Teacher &t, float *loss, float *lse, void *stream);
int launch_distill_grad(const LogitsShard &z, const Teacher &t, const float *lse,
                        const float *grad_loss, void *grad_base, int64_t ld_grad, void *stream);

// ---------------------------------------------------------------------------
// beam search
// ---------------------------------------------------------------------------
// Groups of columns of a row, whose largest logits (one float each) the
// workspace holds; the most for f32.
int64_t beam_groups_per_row(int64_t cols, int dtype);

int launch_beam_select(const void *base, int64_t ld, int dtype, int64_t n_seqs, int beams,
                       int64_t cols, int64_t vocab_start, int64_t vocab, const float *lse,
                       const float *scores, int picks, uint64_t *keys, float *group_best,
                       void *stream);
int launch_beam_merge(const uint64_t *const *keys, int n_parts, int64_t n_seqs, int picks,
                      int64_t vocab, float *score, int64_t *parent, int64_t *token, void *stream);
int launch_beam_reorder(const void *src, int64_t outer, int64_t n_seqs, int beams_in,
                        int64_t row_bytes, const int64_t *parent, int64_t ld_parent,
                        int beams_out, void *dst, void *stream);

}  // namespace vpe

#endif
