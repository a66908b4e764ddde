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

// Sorted positions are summed in chunks of a power of two up to this, each by
// one wave per block of columns: fewer while there are few ids, so that the
// waves fill the chip.
constexpr int64_t kGradChunk = 32;
constexpr int64_t kGradFillChunks = 2048;
// Up to this many ids are sorted by one workgroup.
constexpr int64_t kGradOneBlockIds = 8192;
// Workgroups, ids per workgroup (at least) and digit values of one pass of the
// sort of more ids.
constexpr int64_t kSortMaxBlocks = 128;
constexpr int64_t kSortTile = 2048;
constexpr int64_t kSortDigits = 512;

// Byte offsets of the gradient's workspace (all 16-byte aligned).
struct EmbedGradLayout {
  int64_t count;    // uint32: owned ids
  int64_t hist;     // uint32 [kSortMaxBlocks][kSortDigits]
  int64_t flags;    // uint8 [shard_rows]: the row has an id
  int64_t key[2];   // uint32 [n]
  int64_t pos[2];   // uint32 [n]
  int64_t partial;  // float [2 * chunks][partial_ld]
  int64_t partial_ld;
  int64_t chunk;    // sorted positions per chunk
  int64_t bytes;
};

constexpr int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

inline EmbedGradLayout embed_grad_layout(int64_t n, int64_t shard_rows, int64_t dim) {
  EmbedGradLayout l{};
  const bool passes = n > kGradOneBlockIds;
  int64_t at = 0;
  l.count = at, at += 16;
  l.hist = at, at += passes ? kSortMaxBlocks * kSortDigits * 4 : 0;
  l.flags = at, at += passes ? round16(shard_rows) : 0;
  for (int b = 0; b < 2; ++b) {
    l.key[b] = at, at += b == 0 || passes ? round16(n * 4) : 0;
    l.pos[b] = at, at += b == 0 || passes ? round16(n * 4) : 0;
  }
  l.partial_ld = (dim + 7) / 8 * 8;
  l.chunk = kGradChunk;
  // (a single chunk needs no join)
  while (n > kGradChunk && l.chunk > 4 && (n + l.chunk - 1) / l.chunk < kGradFillChunks)
    l.chunk /= 2;
  // at most one run that enters a chunk and one that leaves it having begun in
  // it; the most chunks of any number of ids up to n, so that a workspace for
  // more ids serves fewer
  const int64_t small = (n + 3) / 4, full = (n + kGradChunk - 1) / kGradChunk;
  const int64_t most = full > 2 * kGradFillChunks ? full : 2 * kGradFillChunks;
  l.partial = at, at += n > 1 ? 2 * (small < most ? small : most) * l.partial_ld * 4 : 0;
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

// From this many rows on each has a workgroup of its own, and no pairs in memory.
constexpr int64_t kDistillWholeRows = 256;

// (maximum, sum) pairs of 8 bytes per row that the workspace holds; the most
// for f32.
int64_t distill_pairs_per_row(int64_t cols, int dtype);

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
// workspace holds.
int64_t beam_groups_per_row(int beams, int64_t cols, int dtype);

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
