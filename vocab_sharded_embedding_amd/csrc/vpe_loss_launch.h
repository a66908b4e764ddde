// Internal interface between the validating C-ABI layer of the loss calls
// (vpe_loss_api.cpp: plain C++ with no HIP headers) and their kernel launchers
// (*.hip).  As in vpe_launch.h, launchers receive validated arguments, enqueue
// on `stream` and return 0 or the hipError_t value the runtime reported.
// dtype: 0 = f32, 1 = bf16; itype: 0 = int32, 1 = int64.
#ifndef VPE_LOSS_LAUNCH_H
#define VPE_LOSS_LAUNCH_H

#include <stdint.h>

namespace vpe {

// ---------------------------------------------------------------------------
// cross entropy and the head's backward
// ---------------------------------------------------------------------------
// Narrowest tile of table rows, by type: a row of hidden states has at most one
// (maximum, sum) pair per this many table rows.
constexpr int64_t loss_tile_rows(int dtype) { return dtype == 1 ? 128 : 64; }
// Bytes of table rows copied to an aligned buffer at a time, where they are not
// aligned.
constexpr int64_t kLossCopyBytes = int64_t(1) << 27;
// Bytes of one piece of the logits' gradient, where the whole is more; at least
// kLossMinPiece columns of it.  (Steps of 8192 rows against 151936 x 1024 and of 2048
// against two of 75968: 64 MB 8.00 and 2.13 ms, 128 MB 7.58 and 2.06, 256 MB 7.60 and
// 2.03, 512 MB 7.75 and 2.09.)
constexpr int64_t kLossPieceBytes = int64_t(1) << 27;
constexpr int64_t kLossMinPiece = 512;
// Most fp32 sums for the gradient of the hidden rows where its sum over the
// vocabulary is split: at least kLossSplitRows table rows each.
constexpr int64_t kLossSums = int64_t(1) << 23;
constexpr int64_t kLossSplitRows = 128;

// Largest stride of rows, in elements, that the tiles read in place: 256 rows of bf16
// (128 of fp32) end before the offset of a masked load, kLoadMask.
constexpr int64_t kLossMaxStride = (int64_t(1) << 22) - 1024;

constexpr int64_t loss_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
constexpr int64_t loss_min(int64_t a, int64_t b) { return a < b ? a : b; }
constexpr int64_t loss_max(int64_t a, int64_t b) { return a > b ? a : b; }

// Byte offsets of the workspaces, 256-byte aligned.  Every size grows with m, so
// that a workspace for m rows serves fewer.
struct LossLayout {
  int64_t count;   // int32: live rows; float: scale of the gradients
  int64_t row_of;  // int32 [m]: row of the i-th live one
  int64_t target;  // int32 [m]: its target in the shard, or -1
  int64_t lse;     // float [m]: (gradients) its log-sum-exp
  int64_t ratio;   // float [m]: (gradients) its grad_loss over the largest one
  int64_t place;   // int32 [m]: (gradients) a row's place among the live ones, or -1
  int64_t x;       // [m][dim_pad] of the type: the live rows
  int64_t pairs;   // (loss) float2 [tiles][m]
  int64_t sums;    // (gradients) float [splits][m][dim_pad]
  int64_t piece[2];  // (gradients) [m][columns of a piece] of the type; the second
                     // where there is more than one piece of bf16
  int64_t piece_cap;
  int64_t table;   // [table_rows][dim_pad] of the type
  int64_t table_rows;
  int64_t dim_pad;
  int64_t bytes;
};

enum LossCall { kLossForward, kLossGrad, kHeadGrad };

// Times that sum may be split.
constexpr int64_t loss_most_splits(int64_t m, int64_t dim_pad, int64_t shard_rows) {
  return loss_max(1, loss_min(kLossSums / dim_pad / loss_max(m, 1),
                              (shard_rows + kLossSplitRows - 1) / kLossSplitRows));
}

inline LossLayout loss_layout(LossCall call, int64_t m, int64_t dim, int64_t shard_rows,
                              int dtype) {
  LossLayout l{};
  const int64_t e = dtype == 1 ? 2 : 4;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += loss_up(bytes, 256);
    return here;
  };
  l.dim_pad = loss_up(dim, 64);
  l.count = take(256);
  if (call != kHeadGrad) l.row_of = take(m * 4), l.target = take(m * 4);
  if (call == kLossGrad) l.lse = take(m * 4), l.ratio = take(m * 4), l.place = take(m * 4);
  l.x = take(m * l.dim_pad * e);
  l.table_rows = loss_min(loss_up(shard_rows, 256),
                          loss_max(4096, kLossCopyBytes / (e * l.dim_pad) / 256 * 256));
  if (call == kLossForward) {
    const int64_t tile = loss_tile_rows(dtype);
    l.pairs = take(m * ((shard_rows + tile - 1) / tile) * 8);
  } else {
    // (no less than loss_most_splits() times m rows, and growing with m)
    const int64_t most = (shard_rows + kLossSplitRows - 1) / kLossSplitRows;
    l.sums = take(loss_max(m, loss_min(kLossSums / l.dim_pad, m * most)) * l.dim_pad * 4);
    const int64_t rows = loss_up(shard_rows, 256);
    l.piece_cap = loss_max(loss_min(m * rows * e, kLossPieceBytes),
                           m * loss_min(rows, kLossMinPiece) * e);
    l.piece[0] = take(l.piece_cap);
    l.piece[1] = call == kLossGrad && dtype == 1 ? take(l.piece_cap) : l.piece[0];
  }
  l.table = take(l.table_rows * l.dim_pad * e);
  l.bytes = at;
  return l;
}

// Most workgroups of a launch over table rows and one other side, in tiles of 64 x 64 and
// more: a grid holds fewer than 2^32 work-items, 512 or 256 a workgroup.  And how many
// table rows that leaves one launch (of side 2^21: 8192; whole tiles of any width).
constexpr int64_t kLossMaxGroups = int64_t(1) << 22;
constexpr int64_t launch_rows(int64_t side) {
  return kLossMaxGroups / (loss_up(loss_max(side, 1), 64) / 64) * 64 / 256 * 256;
}

// Workgroups of 256 that join the sums of [m, dim], four values a thread, in rows of
// kFinishWidth: 2^27 of them are more than one dimension of a grid holds (fewer than 2^32
// work-items).  A loop over a bounded grid took 31 us for 4096 x 4096, 25 without.
constexpr int64_t kFinishWidth = int64_t(1) << 16;
constexpr int64_t finish_groups(int64_t m, int64_t dim) {
  return (m * ((dim + 3) / 4) + 255) / 256;
}

// `rows` in pieces of at most `most`, a multiple of 256, as even as whole tiles allow.
constexpr int64_t even_pieces(int64_t rows, int64_t most) {
  return loss_min(most, loss_up((rows + (rows + most - 1) / most - 1) / ((rows + most - 1) / most),
                                256));
}

// Table rows per launch of the loss (`copied`: as many as the copied table's buffer
// holds).
inline int64_t loss_piece(const LossLayout &l, int64_t m, int64_t rows, bool copied) {
  return loss_min(loss_min(rows, copied ? l.table_rows : rows), launch_rows(m));
}

// Columns of a piece of the logits' gradient: what its buffer (`copied`: and that of the
// copied table) holds.
inline int64_t grad_piece(const LossLayout &l, int64_t m, int64_t rows, int dtype, bool copied) {
  const int64_t e = dtype == 1 ? 2 : 4;
  int64_t most = loss_min(l.piece_cap / (m * e) / 256 * 256, kLossMaxStride);
  most = loss_min(most, launch_rows(l.dim_pad));
  if (copied) most = loss_min(most, l.table_rows);
  return even_pieces(rows, most);
}

// The same of a given gradient: all of it, where nothing is copied.
inline int64_t head_grad_piece(const LossLayout &l, int64_t m, int64_t rows, int dtype,
                               bool d_copied, bool w_copied) {
  const int64_t e = dtype == 1 ? 2 : 4;
  int64_t most = loss_min(loss_up(rows, 256), launch_rows(l.dim_pad));
  if (d_copied)
    most = loss_min(most, loss_min(l.piece_cap / (m * e) / 256 * 256, kLossMaxStride));
  if (w_copied) most = loss_min(most, l.table_rows);
  return even_pieces(rows, most);
}

// fp32 products of n x m (`splits` times) that take tiles of 64 x 64: with too few of
// 128 x 128 to fill the chip, or where those cover over 1/16 more.  (Forward and
// gradients of 512 x 32000 x 512: 597 us, 626 with 64 x 64; gradients of 300 x 8000 x
// 256: 69 us, 55 with 64 x 64; of 100 x 151936 x 64: 171 us, 102 with 64 x 64.)
constexpr bool small_tiles(int64_t n, int64_t m, int64_t splits = 1) {
  return loss_up(n, 128) * loss_up(m, 128) / (128 * 128) * splits < 256 ||
         loss_up(n, 128) * loss_up(m, 128) / 17 > loss_up(n, 64) * loss_up(m, 64) / 16;
}

// Whether the fp32 products take 64 x 64 tiles: both in one launch by the table's, the
// larger one.  (Gradients of 771 rows against 8308 x 1024: 338 us, 403 with the hidden
// rows' in a launch of 64 x 64 of its own.)  Not where the hidden rows' alone would be
// too many for a launch.
constexpr bool small_products(int64_t rows, int64_t dim, int64_t cols, int64_t splits, bool gw) {
  return (gw ? small_tiles(dim, cols) : small_tiles(dim, rows, splits)) &&
         loss_up(rows, 64) / 64 * (loss_up(dim, 64) / 64) * splits <= kLossMaxGroups;
}

// Whether the bf16 logits of m rows and `rows` of the table take 256 x 256 tiles: with
// two for every CU.  (Loss of 600 rows against 151936 x 1024: 201 us, 231 with 128 x
// 128; of 4000 rows against 5000 x 1024: 71 us, 65 with 128 x 128.)
constexpr bool large_logits(int64_t m, int64_t rows) {
  return m > 128 && loss_up(rows, 256) / 256 * (loss_up(m, 256) / 256) >= 512;
}

// Whether the bf16 products take 256 x 256 tiles: where at least three quarters of
// their rows and more than half of their columns exist.  (The head's backward of 256
// rows against 75968 x 1024: 114 us, 136 with 128 x 128; the gradients of 257 rows
// against 50257 x 999: 110 us, 91 with 128 x 128; of 4000 rows against 151936 x 128:
// 1330 us, 1220 with 128 x 128.)
constexpr bool large_products(int64_t rows, int64_t dim) {
  return rows > 128 && rows * 4 >= loss_up(rows, 256) * 3 && dim > 128;
}

struct LossRows {  // hidden rows and their targets
  const void *x;
  int64_t m, dim;
  const void *w;
  int64_t rows;
  int dtype;
  int64_t vocab_start, vocab;
  const void *targets;
  int itype;
};

// What the gradients are written to: `gxt`, `gwt` their types.
struct LossGrads {
  void *gx;
  int gxt;
  void *gw;
  int gwt;
  bool accumulate;
};

// Rows that the tiles can read in place.
inline bool loads_in_place(const void *p, int64_t ld, int dtype) {
  return ld % (dtype == 1 ? 8 : 4) == 0 && ld <= kLossMaxStride &&
         (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

// Whether rows that cannot be read in place pass through registers, in tiles of at
// most 128 x 128, rather than be copied first.  Against 50001 x 1001, loose and copied:
// loss of 16 rows 26 and 60 us, of 257 81 and 89, of 1000 189 and 155; gradients of 128
// rows 130 and 136 (against 50001 x 3001 306 and 417), of 257 259 and 183; the head's
// backward of 128 rows 94 and 162, of 257 175 and 194, of 500 255 and 223.  Gradients
// of 128 rows against 5001 x 3001, whose tiles leave CUs idle: 112 and 84.
constexpr bool loose_rows(LossCall call, int64_t m, int64_t rows, int64_t ld) {
  if (ld > kLossMaxStride) return false;
  if (call == kLossGrad) return m <= 128 && loss_up(rows, 128) / 128 >= 256;
  return m <= (call == kLossForward ? 512 : 256);
}

// The operands of the head's backward that are copied to aligned rows first, or (`loose`)
// all pass through registers: of those that a wanted gradient reads, which is the table
// for grad_x and the hidden rows for grad_weight.
struct HeadGradRows {
  bool d_copied, w_copied, x_copied, loose;
};
inline HeadGradRows head_grad_rows(const void *d, int64_t ld, const LossRows &r,
                                   const LossGrads &g) {
  // (d's rows have to end at whole 16 bytes too: what lies behind may be anything,
  // a NaN as well)
  const bool d_apart = !loads_in_place(d, ld, r.dtype) || r.rows % (r.dtype == 1 ? 8 : 4) != 0;
  const bool w_apart = g.gx != nullptr && !loads_in_place(r.w, r.dim, r.dtype);
  const bool x_apart = g.gw != nullptr && !loads_in_place(r.x, r.dim, r.dtype);
  // (x alone is a small copy)
  if ((d_apart || w_apart) && loose_rows(kHeadGrad, r.m, r.rows, loss_max(ld, r.dim)))
    return {false, false, false, true};
  return {d_apart, w_apart, x_apart, false};
}

int launch_lmhead_xent(const LossRows &r, float *shard_lse, float *target_logit, void *workspace,
                       void *stream);
int launch_xent_loss(const float *const *shard_lse, const float *const *target_logit, int n_parts,
                     int64_t m, int64_t vocab, const void *targets, int itype, float *loss,
                     float *lse, void *stream);
int launch_lmhead_xent_grad(const LossRows &r, const float *lse, const float *grad_loss,
                            const LossGrads &g, void *workspace, void *stream);
// `d`: the shard's columns of the logits' gradient, row stride ld.
int launch_lmhead_grad(const void *d, int64_t ld, const LossRows &r, const LossGrads &g,
                       void *workspace, void *stream);

// ---------------------------------------------------------------------------
// clipping
// ---------------------------------------------------------------------------
// Tensors per launch: their table travels in the kernel's arguments.
constexpr int kClipTable = 96;

// Elements per workgroup: a multiple of 4096, so that about 8192 workgroups at most
// share the elements.
inline int64_t clip_chunk(int64_t total) { return loss_up((total + 8191) / 8192 + 1, 4096); }
inline int64_t clip_chunks(const int64_t *counts, int n, int64_t chunk) {
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) chunks += (counts[i] + chunk - 1) / chunk;
  return chunks;
}

int launch_grad_sumsq(const void *const *tensors, const int64_t *counts, const int32_t *dtypes,
                      int n, int64_t total, double *sumsq, double *partial, void *stream);
int launch_grad_clip(const void *const *tensors, const int64_t *counts, const int32_t *dtypes,
                     int n, int64_t total, void *const *out, const double *const *sumsq,
                     int n_parts, double max_norm, float *norm, void *stream);

}  // namespace vpe

#endif
