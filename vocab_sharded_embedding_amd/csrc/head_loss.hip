// Cross entropy straight from the LM head's shard, its gradients, and the head's
// backward, for gfx950.
//
// The logits z = x W^T are products for the matrix cores and, at training sizes,
// far larger than their operands; they are never kept.  Rows without a target
// are left out first: `collect_rows` copies the live rows of x, so that what a
// padded row holds reaches no sum over rows and no tile is spent on it (the loss
// of up to 256 rows, which sums over none, reads x in place).
//  - Loss: every tile of z becomes one pair (maximum, sum of exponentials) per
//    row in the workgroup that computed it, and the one logit that is a row's
//    target; `join_pairs` merges a row's pairs.
//  - Gradients, a piece of the vocabulary at a time: the piece's
//    d = softmax - onehot goes to a buffer of 128 MB, and feeds two products,
//    grad_x += d W and grad_weight = d^T x, that read d and W (x) in place, in rows
//    or in columns.  d is rounded to the operands' type: the matrix cores take two
//    operands of one type, and their fp32 rate is a tenth of bf16's (bf16 gradients
//    are off by 2.0e-3 of their size with it, 1.7e-3 by their own rounding alone).
//    The sum over the vocabulary in grad_x is kept in fp32 between pieces, split
//    over several sums where there are few rows; `finish_grad_x` joins and rounds
//    them.
//  - The head's backward is the same two products on a given d.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "vpe_device.h"
#include "vpe_loss_launch.h"
#include "vpe_tile.h"

namespace vpe {
namespace {

using tile::f32x16;
using tile::f32x4;

[[maybe_unused]] constexpr float kLog2e = 1.4426950408889634f;

int last_error() { return static_cast<int>(hipGetLastError()); }

// ---------------------------------------------------------------------------
// live rows
// ---------------------------------------------------------------------------
struct Collect {
  const void *x;
  int64_t m, dim, dim_pad;
  const void *targets;
  int64_t vocab_start, vocab, rows;
  const float *lse, *grad_loss;  // gradients; nullptr for the loss
  int rows_per_block;
  int32_t *count;
  float *scale;
  int32_t *row_of, *target, *place;
  float *lse_of, *ratio;
  void *xl;
  float *shard_lse, *target_logit;  // loss: written 0
};

template <class I>
__device__ __forceinline__ bool row_lives(const Collect &c, int64_t i) {
  const int64_t t = static_cast<const I *>(c.targets)[i];
  return t >= 0 && t < c.vocab && (c.grad_loss == nullptr || c.grad_loss[i] != 0.f);
}

// Live rows in order, without a second pass (8192 x 1024 bf16: 23 us, latency; of 1021
// rows 7 us): every workgroup counts the live
// rows before its own (targets are small against x).  The gradients' factors are
// taken over the largest finite |grad_loss|, so that a loss averaged over its
// rows has factors of exactly 1 and d is rounded as softmax - onehot.
template <bool BF16, class I>
__global__ __launch_bounds__(256) void collect_rows(Collect c) {
  __shared__ int wave_n[4];
  __shared__ float wave_top[4];
  __shared__ int kept[1024], kept_at[1024];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * c.rows_per_block;
  const int64_t end = row0 + c.rows_per_block < c.m ? row0 + c.rows_per_block : c.m;
  int before = 0;
  float top = 0.f;
  if (c.grad_loss != nullptr) {
    for (int64_t i = threadIdx.x; i < c.m; i += 256) {
      const bool live = row_lives<I>(c, i);
      before += live && i < row0;
      const float a = fabsf(c.grad_loss[i]);
      if (live && a > top && a < __builtin_huge_valf()) top = a;
    }
  } else {
    for (int64_t i = threadIdx.x; i < row0; i += 256) before += row_lives<I>(c, i);
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) {
    before += __shfl_xor(before, d);
    top = fmaxf(top, __shfl_xor(top, d));
  }
  if (lane == 0) wave_n[wave] = before, wave_top[wave] = top;
  __syncthreads();
  before = wave_n[0] + wave_n[1] + wave_n[2] + wave_n[3];
  top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));
  if (top == 0.f) top = 1.f;
  int mine = 0;
  for (int64_t base = row0; base < end; base += 256) {
    const int64_t i = base + threadIdx.x;
    const bool live = i < end && row_lives<I>(c, i);
    const uint64_t votes = __ballot(live);
    __syncthreads();
    if (lane == 0) wave_n[wave] = __popcll(votes);
    __syncthreads();
    int at = mine + __popcll(votes & ((uint64_t(1) << lane) - 1));
    for (int w = 0; w < wave; ++w) at += wave_n[w];
    mine += wave_n[0] + wave_n[1] + wave_n[2] + wave_n[3];
    if (live) {
      const int64_t local = static_cast<const I *>(c.targets)[i] - c.vocab_start;
      const int to = before + at;
      c.row_of[to] = static_cast<int32_t>(i);
      c.target[to] = local >= 0 && local < c.rows ? static_cast<int32_t>(local) : -1;
      if (c.grad_loss != nullptr) {
        c.lse_of[to] = c.lse[i];
        c.ratio[to] = c.grad_loss[i] / top;
      }
      kept[at] = static_cast<int>(i - row0);
      kept_at[at] = to;
    }
    if (i < end) {
      if (c.place != nullptr) c.place[i] = live ? before + at : -1;
      if (c.shard_lse != nullptr) c.shard_lse[i] = 0.f, c.target_logit[i] = 0.f;
    }
  }
  __syncthreads();
  if (end == c.m && threadIdx.x == 0) {
    *c.count = before + mine;
    *c.scale = top;
  }
  // rows of x, with zeros up to dim_pad
  constexpr int kSize = BF16 ? 2 : 4, kEpv = 16 / kSize;
  const char *x = static_cast<const char *>(c.x);
  char *xl = static_cast<char *>(c.xl);
  const int vecs = static_cast<int>(c.dim_pad / kEpv);
  for (int k = wave; k < mine; k += 4) {
    const char *src = x + (row0 + kept[k]) * c.dim * kSize;
    char *dst = xl + static_cast<int64_t>(kept_at[k]) * c.dim_pad * kSize;
    for (int v = lane; v < vecs; v += 4 * 64) {
      float e[4][kEpv];  // four loads in flight
#pragma unroll
      for (int u = 0; u < 4; ++u)
        dev::load_vec<BF16, kEpv>(src, (static_cast<int64_t>(v) + u * 64) * kEpv, c.dim, e[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (v + u * 64 < vecs)
          *reinterpret_cast<dev::u32x4 *>(dst + (v + u * 64) * 16) =
              dev::Vec<BF16, kEpv>::narrow(e[u]);
    }
  }
}

// `rows` rows of `cols` values at stride ld, any alignment, copied to stride ld_to
// with zeros up to it.  Bound by HBM: 50257 x 999 bf16 33-42 us, 4.8-6.1 TB/s.
template <bool BF16>
__global__ __launch_bounds__(256) void copy_rows(const char *__restrict__ from, int64_t ld,
                                                 int64_t rows, int64_t cols,
                                                 char *__restrict__ to, int64_t ld_to) {
  constexpr int kSize = BF16 ? 2 : 4, kEpv = 16 / kSize;
  const int lane = threadIdx.x & 63;
  const int64_t vecs = ld_to / kEpv;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6); r < rows;
       r += static_cast<int64_t>(gridDim.x) * 4)
    for (int64_t v = lane; v < vecs; v += 64) {
      float e[kEpv];
      dev::load_vec<BF16, kEpv>(from + r * ld * kSize, v * kEpv, cols, e);
      *reinterpret_cast<dev::u32x4 *>(to + (r * ld_to + v * kEpv) * kSize) =
          dev::Vec<BF16, kEpv>::narrow(e);
    }
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
// Workgroup b's tile (n, m) of tiles_n x tiles_m.  Workgroups go to the 8 XCDs
// in turn; each XCD gets one contiguous run of tiles, ordered in groups of
// group_n tiles of n, so that the tiles it runs at once share both operands in
// its own L2.
[[maybe_unused]] __device__ __forceinline__ void tile_of(int b, int tiles_n, int tiles_m,
                                                         int group_n, int &tn, int &tm) {
  const int total = tiles_n * tiles_m;
  const int xcd = b & 7, idx = b >> 3, per = total >> 3, rem = total & 7;
  const int t = xcd < rem ? xcd * (per + 1) + idx : rem * (per + 1) + (xcd - rem) * per + idx;
  const int group = group_n * tiles_m;
  const int g = t / group, in = t - g * group;
  const int gn = min(group_n, tiles_n - g * group_n);
  tm = in / gn;
  tn = g * group_n + (in - tm * gn);
}

#if defined(__HIP_DEVICE_COMPILE__)
// Adds to acc the tile whose operands begin at a and b: n_left and m_left rows (or
// columns), ka and kb values of k that may be read, k to sum over.
template <class S, int E, bool NCOLS, bool MCOLS, bool LOOSE>
__device__ __forceinline__ void product(const void *a, int64_t lda, int64_t n_left, int64_t ka,
                                        const void *b, int64_t ldb, int64_t m_left, int64_t kb,
                                        int64_t k, char *const (&st)[tile::kStages],
                                        f32x16 (&acc)[S::FN][S::FM]) {
  const int wave = tile::wave_id();
  tile::Product<S, E, NCOLS, MCOLS> p;
  p.a.init(a, lda, n_left, ka, wave % S::WN * S::TN);
  p.b.init(b, ldb, m_left, kb, wave / S::WN * S::TM);
  const int steps = static_cast<int>((k + S::BK - 1) / S::BK);
  if constexpr (LOOSE) p.run_loose(steps, st, acc);
  else p.run(steps, st, acc);
}

// A wave's accumulators as rows of m: 32 rows at a time pass through the wave's
// part of the LDS (the stages: every wave is done with them), and `put(m, n, v)`
// gets 16 bytes of consecutive columns n.. of row m, neighbouring lanes
// neighbouring columns: 4 of fp32 (BF16 false; 64 columns at a time) or 8 rounded
// to bf16.  m and n count from the workgroup's tile.
template <class S>
struct RowWriter {
  static constexpr int kCols = S::TN < 64 ? S::TN : 64;
  static constexpr int kLd = kCols + 4, kLd16 = S::TN + 8;
  static constexpr int kWaveBytes = 32 * kLd * 4 > 32 * kLd16 * 2 ? 32 * kLd * 4 : 32 * kLd16 * 2;

  // (half of the waves in each of two stages; LDS pointers by type: a choice
  // between two generic ones would make every access a flat one)
  typedef __attribute__((address_space(3))) char lds_char;
  static __device__ __forceinline__ lds_char *region(char *const (&st)[tile::kStages]) {
    const int wave = tile::wave_id();
    lds_char *even = (lds_char *)st[0], *odd = (lds_char *)st[1];
    return ((wave & 1) ? odd : even) + wave / 2 * kWaveBytes;
  }
  template <class T>
  static __device__ __forceinline__ __attribute__((address_space(3))) T *lds(lds_char *p) {
    return (__attribute__((address_space(3))) T *)p;
  }
  static __device__ __forceinline__ void turn() {
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  }
  template <bool BF16, class Put>
  static __device__ __forceinline__ void run(const f32x16 (&acc)[S::FN][S::FM],
                                             char *const (&st)[tile::kStages], Put put) {
    const int lane = threadIdx.x & 63, wave = tile::wave_id();
    const int m0 = wave / S::WN * S::TM, n0 = wave % S::WN * S::TN;
    const int row = lane & 31, hi = lane >> 5;
#pragma unroll
    for (int j = 0; j < S::FM; ++j) {
      if constexpr (BF16) {
        lds_char *mine = region(st);
        constexpr int kPer = S::TN / 8, kRows = 64 / kPer;
#pragma unroll
        for (int i = 0; i < S::FN; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x16 &f = acc[i][j];
            *lds<dev::u32x2>(mine + (row * kLd16 + i * 32 + 8 * q + 4 * hi) * 2) =
                dev::u32x2{dev::pack_bf16(f[4 * q], f[4 * q + 1]),
                           dev::pack_bf16(f[4 * q + 2], f[4 * q + 3])};
          }
        turn();
#pragma unroll
        for (int t = 0; t < 32 / kRows; ++t) {
          const int r = t * kRows + lane / kPer, n = lane % kPer * 8;
          const dev::u32x4 v = *lds<dev::u32x4>(mine + (r * kLd16 + n) * 2);
          put(m0 + j * 32 + r, n0 + n, v);
        }
        turn();
      } else {
        lds_char *mine = region(st);
        constexpr int kPer = kCols / 4, kRows = 64 / kPer;
#pragma unroll
        for (int h = 0; h < S::TN / kCols; ++h) {
#pragma unroll
          for (int i = 0; i < kCols / 32; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f32x16 &f = acc[h * (kCols / 32) + i][j];
              *lds<f32x4>(mine + (row * kLd + i * 32 + 8 * q + 4 * hi) * 4) =
                  f32x4{f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]};
            }
          turn();
#pragma unroll
          for (int t = 0; t < 32 / kRows; ++t) {
            const int r = t * kRows + lane / kPer, n = lane % kPer * 4;
            const f32x4 v = *lds<f32x4>(mine + (r * kLd + n) * 4);
            put(m0 + j * 32 + r, n0 + h * kCols + n, v);
          }
          turn();
        }
      }
    }
  }
};
#endif

// The stages of a kernel's tile, `st`: LDS arrays of their own (see Product).  Each
// holds a stage of shape S of E-byte elements, and half of the waves' rows.
#define VPE_STAGES(S, E)                                                             \
  constexpr int kRowBytes = (S::NW + 1) / 2 * RowWriter<S>::kWaveBytes;              \
  constexpr int kTileBytes = (S::BN + S::BM) * S::BK * E;                            \
  constexpr int kStageBytes = kTileBytes > kRowBytes ? kTileBytes : kRowBytes;       \
  __shared__ __attribute__((aligned(16))) char stage0[kStageBytes];                  \
  __shared__ __attribute__((aligned(16))) char stage1[kStageBytes];                  \
  __shared__ __attribute__((aligned(16))) char stage2[S::NS > 2 ? kStageBytes : 16]; \
  char *st[tile::kStages];                                                           \
  st[0] = stage0, st[1] = stage1, st[2] = stage2;

// ---------------------------------------------------------------------------
// logits
// ---------------------------------------------------------------------------
// The targets of rows that were not collected.
struct Targets {
  const void *ids;
  int itype;
  int64_t vocab_start, vocab, rows;

  __device__ __forceinline__ bool local(int64_t i, int64_t &at) const {
    const int64_t t = itype == 0 ? static_cast<const int32_t *>(ids)[i]
                                 : static_cast<const int64_t *>(ids)[i];
    at = t - vocab_start;
    if (at < 0 || at >= rows || t >= vocab) at = -1;
    return t >= 0 && t < vocab;
  }
};

struct Logits {
  const void *x;  // live rows, stride ldx
  int64_t ldx, x_dim;  // x_dim, w_dim: values of a row that may be read
  const void *w;  // a piece of the shard's rows, stride ldw
  int64_t ldw, w_rows, w_dim;
  int64_t k;
  const int32_t *count;  // live rows; nullptr: all m, targets in `any`
  int64_t m;
  int tiles_n, tiles_m, group_n;
  int round;  // tiles that run at once, where the last round may be cut in two; or 0
  const int32_t *target;
  Targets any;
  int64_t row0;  // the piece's first row in the shard
  // loss
  float *pairs;  // [tile][pair_ld] (maximum, sum)
  int64_t pair_ld, tile0;
  float *target_logit;
  const int32_t *row_of;
  // gradients
  const float *lse, *ratio;
  void *d;
  int64_t ldd;  // the piece's columns, zeros after the last
};

// exp(z - lse), |z - lse| times a rounding closer than the exponential of the rounded
// product (z - lse) log2(e): what the difference and the product lose is added as a
// factor 1 + the loss.  (An infinite or NaN difference has no loss to add.)
__device__ __forceinline__ float exp_of(float z, float lse) {
  const float t = z - lse, back = t - z;
  const float lost = (z - (t - back)) - (lse + back);
  const float hi = t * kLog2e;
  const float lo = fmaf(t, 1.92596299e-8f, fmaf(t, kLog2e, -hi));  // log2(e) - kLog2e
  const float p = __builtin_amdgcn_exp2f(hi);
  const float more = fmaf(lo, 0.693147182f, lost);
  return fabsf(more) < 1.f ? fmaf(p, more, p) : p;
}

// (m, s) of two disjoint sets of logits; an empty one is (-inf, 0).
__device__ __forceinline__ void merge(float &m, float &s, float m2, float s2) {
  const float top = (m != m || m > m2) ? m : m2;
  const float a = m == -__builtin_huge_valf() ? 0.f : s * __expf(m - top);
  const float b = m2 == -__builtin_huge_valf() ? 0.f : s2 * __expf(m2 - top);
  m = top;
  s = a + b;
}

// A tile's last rows may fill half of it or less: then half a tile is computed, as
// wide and by as many waves.  (The live rows are known to the device alone.)
template <class S>
struct Half {
  typedef S type;  // none
};
template <>
struct Half<tile::Shape<256, 256, 2, 4, 64, 2>> {
  typedef tile::Shape<256, 128, 4, 2, 64, 2> type;
};
template <>
struct Half<tile::Shape<128, 128, 2, 2, 32, 2>> {
  typedef tile::Shape<128, 64, 2, 2, 32, 2> type;
};
template <class S>
constexpr bool has_half() {
  return !std::is_same<typename Half<S>::type, S>::value;
}

#if defined(__HIP_DEVICE_COMPILE__)
// The loss: column in the shard of the target of this lane's rows, or -1.
template <class S>
__device__ __forceinline__ void loss_targets(const Logits &a, int64_t m0, int64_t live,
                                             int (&target)[S::FM]) {
#pragma unroll
  for (int j = 0; j < S::FM; ++j) {
    const int64_t m = m0 + tile::wave_id() / S::WN * S::TM + j * 32 + (threadIdx.x & 31);
    target[j] = -1;
    if (m < live) {
      if (a.count != nullptr) {
        target[j] = a.target[m];
      } else {
        int64_t at;
        a.any.local(m, at);
        target[j] = static_cast<int>(at);
      }
    }
  }
}

// What becomes of the logits acc: columns n0.. (tile tn) of rows m0.. .  `out`: the
// loss's [BM][WN] pairs; `st`: free, for the gradients.
template <class S, bool BF16, bool GRAD>
__device__ __forceinline__ void logits_done(const Logits &a, int tn, int64_t n0, int64_t m0,
                                            int64_t live, const int (&target)[S::FM], float *out,
                                            char *const (&st)[tile::kStages],
                                            f32x16 (&acc)[S::FN][S::FM]) {
  constexpr int kSize = BF16 ? 2 : 4;
  // (opaque, so that what depends on the lane alone is not kept over a loop of tiles:
  // there are no registers for it)
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  const int wave = tile::wave_id();
  const int wn = wave % S::WN, wm = wave / S::WN, hi = lane >> 5;
  const int64_t nb = n0 + wn * S::TN;  // this wave's first column
  // this lane's columns nb + c, c = 32 i + 8 (r / 4) + 4 hi + r % 4, exist for
  // c < lim
  const int64_t left = a.w_rows - nb;
  const int lim = left < 0 ? 0 : (left < S::TN ? static_cast<int>(left) : S::TN);
  if constexpr (!GRAD) {
#pragma unroll
    for (int j = 0; j < S::FM; ++j) {
      const int64_t m = m0 + wm * S::TM + j * 32 + (lane & 31);
      if (lim < S::TN) {  // columns past the last: exponentials of 0
#pragma unroll
        for (int i = 0; i < S::FN; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (i * 32 + 8 * (r / 4) + 4 * hi + r % 4 >= lim)
              acc[i][j][r] = -__builtin_huge_valf();
      }
      float top = -__builtin_huge_valf();
#pragma unroll
      for (int i = 0; i < S::FN; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, acc[i][j][r]);
      const float base = top == -__builtin_huge_valf() ? 0.f : top;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < S::FN; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          // (the difference first: a rounded shift of base log2(e) would be in every term,
          // and infinite for a finite base past 2.3e38)
          s += __builtin_amdgcn_exp2f((acc[i][j][r] - base) * kLog2e);
      if (s != s) top = s;  // a NaN logit, or +inf
      merge(top, s, __shfl_xor(top, 32), __shfl_xor(s, 32));
      if (hi == 0) {
        float *e = out + ((wm * S::TM + j * 32 + lane) * S::WN + wn) * 2;
        e[0] = top, e[1] = s;
      }
      // the row's target, where this wave has its column
      const int64_t rel = target[j] < 0 ? -1 : target[j] - a.row0 - nb;
      if (__any(rel >= 0 && rel < S::TN)) {
        float z = 0.f;
        const int at = rel >= 0 && rel < lim ? static_cast<int>(rel) : -1;
#pragma unroll
        for (int i = 0; i < S::FN; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (at == i * 32 + 8 * (r / 4) + 4 * hi + r % 4) z = acc[i][j][r];
        if (at >= 0 && ((at >> 2) & 1) == hi)
          a.target_logit[a.count != nullptr ? a.row_of[m] : m] = z;
      }
    }
    __syncthreads();
    for (int r = threadIdx.x; r < S::BM; r += S::NT) {
      if (m0 + r >= live) continue;
      float top = out[r * S::WN * 2], s = out[r * S::WN * 2 + 1];
#pragma unroll
      for (int w = 1; w < S::WN; ++w)
        merge(top, s, out[(r * S::WN + w) * 2], out[(r * S::WN + w) * 2 + 1]);
      float *e = a.pairs + ((a.tile0 + tn) * a.pair_ld + m0 + r) * 2;
      e[0] = top, e[1] = s;
    }
  } else {
    // (elementwise work is as long as several steps of the product: what few
    // elements need is kept out of the common path)
#pragma unroll
    for (int j = 0; j < S::FM; ++j) {
      const int64_t m = m0 + wm * S::TM + j * 32 + (lane & 31);
      float lse = 0.f, ratio = 0.f;
      int at = -1;
      if (m < live) {
        lse = a.lse[m], ratio = a.ratio[m];
        const int32_t t = a.target[m];
        const int64_t rel = t < 0 ? -1 : t - a.row0 - nb;
        at = rel >= 0 && rel < lim ? static_cast<int>(rel) : -1;
      }
      // (the difference first: one fma with a rounded -lse log2(e) would put that rounding
      // into every entry of the row, as large as lse, and be NaN or 0 for a finite lse
      // past 2.3e38)
#pragma unroll
      for (int i = 0; i < S::FN; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          acc[i][j][r] = BF16 ? __builtin_amdgcn_exp2f((acc[i][j][r] - lse) * kLog2e)
                              : exp_of(acc[i][j][r], lse);
      if (__any(at >= 0)) {
#pragma unroll
        for (int i = 0; i < S::FN; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (at == i * 32 + 8 * (r / 4) + 4 * hi + r % 4) acc[i][j][r] -= 1.f;
      }
#pragma unroll
      for (int i = 0; i < S::FN; ++i) acc[i][j] *= ratio;
      if (lim < S::TN) {
#pragma unroll
        for (int i = 0; i < S::FN; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (i * 32 + 8 * (r / 4) + 4 * hi + r % 4 >= lim) acc[i][j][r] = 0.f;
      }
    }
    auto put = [&](int m, int n, auto v) {
      // (ldd is a multiple of 64: the columns of v are inside or past it together)
      if (m0 + m >= live || n0 + n >= a.ldd) return;
      char *to = static_cast<char *>(a.d) + ((m0 + m) * a.ldd + n0 + n) * kSize;
      *reinterpret_cast<decltype(v) *>(to) = v;
    };
    RowWriter<S>::template run<BF16>(acc, st, put);
  }
}

template <class S, bool BF16, bool GRAD, bool LOOSE>
__device__ __forceinline__ void logits_of(const Logits &a, int tn, int64_t n0, int64_t m0,
                                          int64_t live, float *out,
                                          char *const (&st)[tile::kStages]) {
  constexpr int kSize = BF16 ? 2 : 4;
  f32x16 acc[S::FN][S::FM];
#pragma unroll
  for (int i = 0; i < S::FN; ++i)
#pragma unroll
    for (int j = 0; j < S::FM; ++j) acc[i][j] = f32x16(0.f);
  int target[S::FM];
  if constexpr (!GRAD) loss_targets<S>(a, m0, live, target);
  product<S, kSize, false, false, LOOSE>(
      static_cast<const char *>(a.w) + n0 * a.ldw * kSize, a.ldw, a.w_rows - n0, a.w_dim,
      static_cast<const char *>(a.x) + m0 * a.ldx * kSize, a.ldx, live - m0, a.x_dim, a.k, st,
      acc);
  __syncthreads();  // every wave is done with the stages
  logits_done<S, BF16, GRAD>(a, tn, n0, m0, live, target, out, st, acc);
}

// The tiles of a launch, with the device's count of live rows: whole ones first;
// then, where they exist, half ones: those of the last live rows, or the whole tiles
// that would begin a round of the chip's CUs and leave most of it idle, in two.
template <class S>
struct Tiles {
  typedef typename Half<S>::type H;
  int live, whole_m, whole, split, halves;

  __device__ __forceinline__ explicit Tiles(const Logits &a) {
    live = static_cast<int>(a.count != nullptr ? *a.count : a.m);
    whole_m = (live + S::BM - 1) / S::BM, halves = split = 0;
    if (has_half<S>() && whole_m * S::BM - live >= S::BM / 2) whole_m -= 1, halves = a.tiles_n;
    whole = a.tiles_n * whole_m;
    if (has_half<S>() && halves == 0 && a.round > 0 && whole > a.round &&
        whole % a.round <= a.round / 2) {
      split = whole % a.round;
      whole -= split, halves = 2 * split;
    }
  }
  // Whole tile t < whole,
  __device__ __forceinline__ void place(const Logits &a, int t, int &tn, int64_t &m0) const {
    int tm;
    tile_of(t, a.tiles_n, whole_m, a.group_n, tn, tm);
    m0 = static_cast<int64_t>(tm) * S::BM;
  }
  // and half tile j < halves.
  __device__ __forceinline__ void place_half(const Logits &a, int j, int &tn, int64_t &m0) const {
    if (split > 0) {
      place(a, whole + j / 2, tn, m0);
      m0 += j % 2 * H::BM;
    } else {
      tn = j, m0 = static_cast<int64_t>(whole_m) * S::BM;
    }
  }
};

template <class S, bool BF16, bool GRAD, bool LOOSE>
__device__ __forceinline__ void logits_tile(const Logits &a, int block,
                                            char *const (&st)[tile::kStages]) {
  const Tiles<S> tiles(a);
  int tn;
  int64_t m0;
  float *out = reinterpret_cast<float *>(st[0]);
  if (block < tiles.whole) {
    tiles.place(a, block, tn, m0);
    logits_of<S, BF16, GRAD, LOOSE>(a, tn, static_cast<int64_t>(tn) * S::BN, m0, tiles.live, out,
                                    st);
  } else if constexpr (has_half<S>()) {
    if (block - tiles.whole >= tiles.halves) return;
    tiles.place_half(a, block - tiles.whole, tn, m0);
    logits_of<typename Half<S>::type, BF16, GRAD, LOOSE>(
        a, tn, static_cast<int64_t>(tn) * S::BN, m0, tiles.live, out, st);
  }
}
#endif

// One workgroup per tile.  Few rows: bound by reading the table (1 row against 151936 x
// 1024 bf16: 51 us, 6.05 TB/s).  Loose rows: by the latency of loads that pass through
// registers (257 rows against 50257 x 999: 60 us, 33 on aligned rows).  fp32: by the
// matrix cores (448 rows against 32000 x 512: 132-144 us, 102-111 TFLOP/s, two rounds of
// tiles; 2048 against 32000 x 1024: 0.97 ms, 138).
// (4 waves: two workgroups per CU)
template <class S, bool BF16, bool GRAD, bool LOOSE>
__global__ __launch_bounds__(S::NT, S::NT == 256 ? 2 : 1) void logits_tiles(Logits a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kSize = BF16 ? 2 : 4;
  VPE_STAGES(S, kSize)
  static_assert(kStageBytes >= S::BM * S::WN * 8, "the pairs fit a stage");
  logits_tile<S, BF16, GRAD, LOOSE>(a, blockIdx.x, st);
#endif
}

// The loss in large tiles: a workgroup per CU takes tile after tile, and the loads
// of the next one are under way while the exponentials of one are taken.
//
// Bound by the matrix cores and, between two tiles of K = 1024, by the exponentials
// (a seventh of the cycles: all eight waves take them at once).  8192 rows, 7168 of
// them live, against 151936 x 1024: 1.79-1.92 ms, 1.16-1.24 PFLOP/s, matrix cores busy
// 63% at 1.82-1.84 GHz; 3584 live rows against 37984 x 4096: 0.92
// ms, 1.21 PFLOP/s; 896 against 75968 x 1024: 142-147 us, 0.95-0.98 PFLOP/s, four and a half
// rounds of tiles for the work of four.  A workgroup per tile: 1% slower.  Four stages
// of 32 values of k: 5% slower.
template <class S>
__global__ __launch_bounds__(S::NT) void loss_tiles(Logits a) {
#if defined(__HIP_DEVICE_COMPILE__)
  VPE_STAGES(S, 2)
  __shared__ float out[S::BM * S::WN * 2];
  static_assert(Half<S>::type::BM * Half<S>::type::WN <= S::BM * S::WN, "its pairs fit too");
  const Tiles<S> tiles(a);
  const int nk = static_cast<int>((a.k + S::BK - 1) / S::BK);
  tile::Product<S, 2, false, false> p;
  int t = blockIdx.x, tn = 0;
  int64_t m0 = 0;
  auto start = [&]() {
    tiles.place(a, t, tn, m0);
    const int64_t n0 = static_cast<int64_t>(tn) * S::BN;
    p.a.init(static_cast<const char *>(a.w) + n0 * a.ldw * 2, a.ldw, a.w_rows - n0, a.w_dim,
             tile::wave_id() % S::WN * S::TN);
    p.b.init(static_cast<const char *>(a.x) + m0 * a.ldx * 2, a.ldx, tiles.live - m0, a.x_dim,
             tile::wave_id() / S::WN * S::TM);
    p.start(nk, st);
  };
  if (t < tiles.whole) start();
  while (t < tiles.whole) {
    int target[S::FM];
    loss_targets<S>(a, m0, tiles.live, target);
    f32x16 acc[S::FN][S::FM];
#pragma unroll
    for (int i = 0; i < S::FN; ++i)
#pragma unroll
      for (int j = 0; j < S::FM; ++j) acc[i][j] = f32x16(0.f);
    p.go_on(nk, st, acc);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // (all done with the stages)
    const int tn_now = tn;
    const int64_t m0_now = m0;
    t += gridDim.x;
    if (t < tiles.whole) start();
    logits_done<S, true, false>(a, tn_now, static_cast<int64_t>(tn_now) * S::BN, m0_now,
                                tiles.live, target, out, st, acc);
  }
  for (int j = t - tiles.whole; j < tiles.halves; j += gridDim.x) {
    tiles.place_half(a, j, tn, m0);
    __syncthreads();
    logits_of<typename Half<S>::type, true, false, false>(
        a, tn, static_cast<int64_t>(tn) * S::BN, m0, tiles.live, out, st);
  }
#endif
}

// A row's pairs joined: shard_lse[row] = log sum exp.  ROWS rows per workgroup of
// 1024: neighbouring lanes have neighbouring rows, and 1024 / ROWS threads share a
// row's tiles (297 tiles of 896 rows: 5.8 us; 10.4 with 64 rows per workgroup; 594 of
// 7168: 11.7 and 23.3).  Rows that were not collected (count nullptr) get their zeros here.
template <int ROWS>
__global__ __launch_bounds__(1024) void join_pairs(const float *__restrict__ pairs, int64_t ld,
                                                   int tiles, const int32_t *__restrict__ count,
                                                   int64_t m_all, Targets any,
                                                   const int32_t *__restrict__ row_of,
                                                   float *__restrict__ shard_lse,
                                                   float *__restrict__ target_logit) {
  constexpr int kShare = 1024 / ROWS;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __shared__ float part[16][ROWS][2];
  const int64_t live = count != nullptr ? *count : m_all;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + lane % ROWS;
  if (static_cast<int64_t>(blockIdx.x) * ROWS >= live) return;
  float m = -__builtin_huge_valf(), s = 0.f;
  if (row < live)
    for (int t = threadIdx.x / ROWS; t < tiles; t += 4 * kShare) {
      dev::f32x2 e[4];  // four loads in flight
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        e[u] = dev::f32x2{-__builtin_huge_valf(), 0.f};
        if (t + u * kShare < tiles)
          e[u] = *reinterpret_cast<const dev::f32x2 *>(pairs + ((t + u * kShare) * ld + row) * 2);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) merge(m, s, e[u][0], e[u][1]);
    }
#pragma unroll
  for (int d = ROWS; d < 64; d *= 2) merge(m, s, __shfl_xor(m, d), __shfl_xor(s, d));
  if (lane < ROWS) part[wave][lane][0] = m, part[wave][lane][1] = s;
  __syncthreads();
  if (wave == 0 && lane < ROWS && row < live) {
    for (int w = 1; w < 16; ++w) merge(m, s, part[w][lane][0], part[w][lane][1]);
    float v = m == -__builtin_huge_valf() ? m : m + logf(s);
    if (count == nullptr) {
      int64_t at;
      if (!any.local(row, at)) v = 0.f;
      if (at < 0) target_logit[row] = 0.f;
    }
    shard_lse[count != nullptr ? row_of[row] : row] = v;
  }
}

struct Parts {
  const float *lse[64];
  const float *target[64];
};

template <class I>
__global__ __launch_bounds__(256) void xent_loss(Parts p, int n, int64_t m, int64_t vocab,
                                                 const I *targets, float *loss, float *lse) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= m) return;
  const int64_t t = targets[i];
  float whole = 0.f, value = 0.f;
  if (t >= 0 && t < vocab) {
    float top = p.lse[0][i], s = 1.f, z = p.target[0][i];
    if (top == -__builtin_huge_valf()) s = 0.f;
    for (int r = 1; r < n; ++r) {
      merge(top, s, p.lse[r][i], 1.f);
      z += p.target[r][i];
    }
    whole = n == 1 || top == -__builtin_huge_valf() ? top : top + logf(s);
    value = whole - z;
  }
  loss[i] = value;
  lse[i] = whole;
}

// ---------------------------------------------------------------------------
// products with the logits' gradient
// ---------------------------------------------------------------------------
struct Products {
  const void *d;  // [rows][cols] at stride ldd
  int64_t ldd, cols;
  const void *w;  // the same piece of the table, stride ldw
  int64_t ldw;
  const void *x;  // rows of x, stride ldx
  int64_t ldx;
  int64_t rows;          // rows of d and x,
  const int32_t *count;  // or (not nullptr) how many of them
  int64_t dim;
  // gradient of x
  float *sums;  // [splits][rows][ld_sums]
  int64_t ld_sums, per_split;  // columns of d per split, a multiple of the k step
  bool first;
  int x_tiles_n, x_tiles_m, splits;
  // gradient of the table
  void *gw;  // the piece's first row
  bool gw_bf16, accumulate;
  const float *scale;
  int w_tiles_n, w_tiles_m;
};

#if defined(__HIP_DEVICE_COMPILE__)
// sums (+)= columns k0.. (k of them) of d, rows m0.., times the table's columns n0.. .
template <class S, bool BF16, bool LOOSE>
__device__ __forceinline__ void grad_x_of(const Products &a, int split, int64_t n0, int64_t m0,
                                          int64_t live, char *const (&st)[tile::kStages]) {
  constexpr int kSize = BF16 ? 2 : 4;
  const int64_t k0 = split * a.per_split;
  int64_t k = a.cols - k0 < a.per_split ? a.cols - k0 : a.per_split;
  if (k < 0) k = 0;
  if (k == 0 && !a.first) return;
  f32x16 acc[S::FN][S::FM];
#pragma unroll
  for (int i = 0; i < S::FN; ++i)
#pragma unroll
    for (int j = 0; j < S::FM; ++j) acc[i][j] = f32x16(0.f);
  // (columns of d up to whole 16 bytes: the table's rows end before)
  constexpr int kEpp = LOOSE ? 1 : 16 / kSize;
  product<S, kSize, true, false, LOOSE>(
      static_cast<const char *>(a.w) + (k0 * a.ldw + n0) * kSize, a.ldw, a.dim - n0, k,
      static_cast<const char *>(a.d) + (m0 * a.ldd + k0) * kSize, a.ldd, live - m0,
      (k + kEpp - 1) / kEpp * kEpp, k, st, acc);
  __syncthreads();
  float *sums = a.sums + split * a.rows * a.ld_sums;
  RowWriter<S>::template run<false>(acc, st, [&](int m, int n, f32x4 v) {
    if (m0 + m >= live || n0 + n >= a.ld_sums) return;
    f32x4 *to = reinterpret_cast<f32x4 *>(sums + (m0 + m) * a.ld_sums + n0 + n);
    *to = a.first ? v : *to + v;
  });
}

// Parts of the launch: 1 the gradient of x, 2 that of the table, 3 both, the
// first's workgroups before the second's.
//
// With many rows bound by the matrix cores: 4096 rows against 37984 x 4096, fp32
// gradients, both products 2.15-2.45 ms, 1.04-1.18 PFLOP/s; fp32, 448 rows against
// 32000 x 512, 265-277 us, 106-111 TFLOP/s.  With few by HBM: 256 against 75968 x 1024 bf16, 92-98
// us, 3.6-3.8 TB/s, the workgroups of either product reading d for themselves.
template <class S, bool BF16, int PARTS, bool LOOSE>
__device__ __forceinline__ void products_tile(const Products &a, int b,
                                              char *const (&st)[tile::kStages]) {
  constexpr int kSize = BF16 ? 2 : 4;
  const int64_t live = a.count != nullptr ? *a.count : a.rows;
  const int x_blocks = (PARTS & 1) ? a.x_tiles_n * a.x_tiles_m * a.splits : 0;
  if constexpr ((PARTS & 1) != 0) {
    if (b < x_blocks) {
      int tn, t2;  // (tiles of m and splits together)
      tile_of(b, a.x_tiles_n, a.x_tiles_m * a.splits, a.x_tiles_n, tn, t2);
      const int split = t2 / a.x_tiles_m, tm = t2 - split * a.x_tiles_m;
      const int64_t n0 = static_cast<int64_t>(tn) * S::BN, m0 = static_cast<int64_t>(tm) * S::BM;
      if (m0 >= live) return;
      if (has_half<S>() && live - m0 <= S::BM / 2)
        grad_x_of<typename Half<S>::type, BF16, LOOSE>(a, split, n0, m0, live, st);
      else
        grad_x_of<S, BF16, LOOSE>(a, split, n0, m0, live, st);
      return;
    }
  }
  if constexpr ((PARTS & 2) != 0) {
    int tn, tm;
    tile_of(b - x_blocks, a.w_tiles_n, a.w_tiles_m, a.w_tiles_n, tn, tm);
    const int64_t n0 = static_cast<int64_t>(tn) * S::BN, m0 = static_cast<int64_t>(tm) * S::BM;
    f32x16 acc[S::FN][S::FM];
#pragma unroll
    for (int i = 0; i < S::FN; ++i)
#pragma unroll
      for (int j = 0; j < S::FM; ++j) acc[i][j] = f32x16(0.f);
    product<S, kSize, true, true, LOOSE>(
        static_cast<const char *>(a.x) + n0 * kSize, a.ldx, a.dim - n0, live,
        static_cast<const char *>(a.d) + m0 * kSize, a.ldd, a.cols - m0, live, live, st, acc);
    __syncthreads();
    const float scale = a.scale != nullptr ? *a.scale : 1.f;
#pragma unroll
    for (int i = 0; i < S::FN; ++i)
#pragma unroll
      for (int j = 0; j < S::FM; ++j) acc[i][j] *= scale;
    // (rows may begin at any element: the vector types ask for no more)
    if (a.gw_bf16 && !a.accumulate) {
      RowWriter<S>::template run<true>(acc, st, [&](int m, int n, dev::u32x4 v) {
        const int64_t left = a.dim - (n0 + n);
        if (m0 + m >= a.cols || left <= 0) return;
        uint16_t *to = static_cast<uint16_t *>(a.gw) + (m0 + m) * a.dim + n0 + n;
        if (left >= 8)
          __builtin_nontemporal_store(v, reinterpret_cast<dev::Vec<true, 8>::loose *>(to));
        else
          for (int e = 0; e < left; ++e)
            to[e] = static_cast<uint16_t>(v[e / 2] >> (e % 2 * 16));
      });
      return;
    }
    RowWriter<S>::template run<false>(acc, st, [&](int m, int n, f32x4 v) {
      if (m0 + m >= a.cols || n0 + n >= a.dim) return;
      const int64_t row = (m0 + m) * a.dim;
      float e[4] = {v[0], v[1], v[2], v[3]}, old[4];
      if (a.gw_bf16) {
        uint16_t *to = static_cast<uint16_t *>(a.gw) + row;
        dev::load_vec<true, 4>(to, n0 + n, a.dim, old);  // (only to accumulate)
#pragma unroll
        for (int k = 0; k < 4; ++k) e[k] += old[k];
        dev::store_vec_nt<true, 4>(to, n0 + n, a.dim, e);
      } else {
        float *to = static_cast<float *>(a.gw) + row;
        if (a.accumulate) {
          dev::load_vec<false, 4>(to, n0 + n, a.dim, old);
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] += old[k];
        }
        dev::store_vec_nt<false, 4>(to, n0 + n, a.dim, e);
      }
    });
  }
}
#endif

template <class S, bool BF16, int PARTS, bool LOOSE>
__global__ __launch_bounds__(S::NT) void grad_tiles(Products a) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kSize = BF16 ? 2 : 4;
  VPE_STAGES(S, kSize)
  products_tile<S, BF16, PARTS, LOOSE>(a, blockIdx.x, st);
#endif
}

// Both products of one piece, and the logits' gradient of the next: the second
// fills the CUs that the first, with few and long tiles, leaves idle.  Bound by the
// matrix cores (7168 live rows, 8192 columns, K = 1024 and 7168: 300-310 us, 1.16-1.20
// PFLOP/s, busy 61%; 355 MB read and 160 written past the L2, 1.7 TB/s).
template <class S>
__global__ __launch_bounds__(S::NT) void grad_and_logits_tiles(Products p, int n, Logits a) {
#if defined(__HIP_DEVICE_COMPILE__)
  VPE_STAGES(S, 2)
  if (static_cast<int>(blockIdx.x) < n) products_tile<S, true, 3, false>(p, blockIdx.x, st);
  else logits_tile<S, true, true, false>(a, blockIdx.x - n, st);
#endif
}

// grad_x from its sums: row i's is at place[i] (nullptr: i), 0 where that is -1.
// (4096 x 4096 fp32 of 1 sum: 25 us, 5.3 TB/s.)
template <bool BF16>
__global__ __launch_bounds__(256) void finish_grad_x(const float *__restrict__ sums,
                                                     int64_t ld_sums, int64_t split_stride,
                                                     int splits, const int32_t *place,
                                                     const float *scale, int64_t m, int64_t dim,
                                                     void *gx) {
  const int64_t vecs = (dim + 3) / 4;
  const int64_t group = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t at = group * 256 + threadIdx.x;
  const int64_t i = at / vecs, n = (at - i * vecs) * 4;
  if (i >= m) return;
  const int64_t from = place != nullptr ? place[i] : i;
  f32x4 v = f32x4(0.f);
  if (from >= 0) {
    const float *p = sums + from * ld_sums + n;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4 *>(p + s * split_stride);
    if (scale != nullptr) v *= *scale;
  }
  float e[4] = {v[0], v[1], v[2], v[3]};
  char *row = static_cast<char *>(gx) + i * dim * (BF16 ? 2 : 4);
  dev::store_vec_nt<BF16, 4>(row, n, dim, e);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// bf16 tiles: 8 waves of 128 x 64 each on 256 x 256, one workgroup per CU; 4
// waves on 128 x 128, two per CU; narrow ones for few hidden rows.
typedef tile::Shape<256, 256, 2, 4, 64, 2> Large;
typedef tile::Shape<128, 128, 2, 2, 64, 2> Medium;
typedef tile::Shape<128, 64, 2, 2, 64, 3> Low64;
typedef tile::Shape<128, 32, 4, 1, 64, 3> Low32;
// fp32 tiles
typedef tile::Shape<128, 128, 2, 2, 32, 2> MediumF;
typedef tile::Shape<64, 64, 2, 2, 32, 2> SmallF;
typedef tile::Shape<128, 32, 4, 1, 32, 3> LowF;

int blocks(int64_t n, int64_t per) { return static_cast<int>((n + per - 1) / per); }

char *at(void *workspace, int64_t offset) { return static_cast<char *>(workspace) + offset; }

int run_collect(const LossRows &r, const LossLayout &l, const float *lse, const float *grad_loss,
                float *shard_lse, float *target_logit, void *ws, hipStream_t st) {
  Collect c{};
  c.x = r.x, c.m = r.m, c.dim = r.dim, c.dim_pad = l.dim_pad;
  c.targets = r.targets, c.vocab_start = r.vocab_start, c.vocab = r.vocab, c.rows = r.rows;
  c.lse = lse, c.grad_loss = grad_loss;
  // about 1024 workgroups, so that the counting of earlier rows stays small against
  // the copying; a row per wave at least
  const int64_t per = loss_max(4, loss_min(1024, loss_up(r.m / 1024, 4)));
  c.rows_per_block = static_cast<int>(per);
  c.count = reinterpret_cast<int32_t *>(at(ws, l.count));
  c.scale = reinterpret_cast<float *>(at(ws, l.count)) + 1;
  c.row_of = reinterpret_cast<int32_t *>(at(ws, l.row_of));
  c.target = reinterpret_cast<int32_t *>(at(ws, l.target));
  if (grad_loss != nullptr) {
    c.place = reinterpret_cast<int32_t *>(at(ws, l.place));
    c.lse_of = reinterpret_cast<float *>(at(ws, l.lse));
    c.ratio = reinterpret_cast<float *>(at(ws, l.ratio));
  }
  c.xl = at(ws, l.x);
  c.shard_lse = shard_lse, c.target_logit = target_logit;
  const dim3 grid(blocks(r.m, per));
  if (r.dtype == 1) {
    if (r.itype == 0) hipLaunchKernelGGL((collect_rows<true, int32_t>), grid, dim3(256), 0, st, c);
    else hipLaunchKernelGGL((collect_rows<true, int64_t>), grid, dim3(256), 0, st, c);
  } else {
    if (r.itype == 0) hipLaunchKernelGGL((collect_rows<false, int32_t>), grid, dim3(256), 0, st, c);
    else hipLaunchKernelGGL((collect_rows<false, int64_t>), grid, dim3(256), 0, st, c);
  }
  return last_error();
}

// Up to this many rows (one tile of them in bf16) the loss reads x in place:
// leaving rows out saves no tile, and collecting them costs a launch (of 1 row
// against 151936 x 1024: 66 -> 62 us).  A row only reaches its own results there,
// whatever it holds.
constexpr int64_t kWholeRows = 256;

void run_copy(const void *from, int64_t ld, int64_t rows, int64_t cols, void *to, int64_t ld_to,
              int dtype, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(loss_min((rows + 3) / 4, 4096)));
  if (dtype == 1)
    hipLaunchKernelGGL(copy_rows<true>, grid, dim3(256), 0, st, static_cast<const char *>(from),
                       ld, rows, cols, static_cast<char *>(to), ld_to);
  else
    hipLaunchKernelGGL(copy_rows<false>, grid, dim3(256), 0, st, static_cast<const char *>(from),
                       ld, rows, cols, static_cast<char *>(to), ld_to);
}

// Sets a's tiles of shape S; returns how many.
template <class S, bool GRAD>
int set_tiles(Logits &a, int64_t m) {
  a.tiles_n = blocks(GRAD ? a.ldd : a.w_rows, S::BN);
  a.tiles_m = blocks(m, S::BM);
  a.group_n = 8;
  return a.tiles_n * a.tiles_m;
}

template <class S, bool BF16, bool GRAD, bool LOOSE>
void run_logits(Logits a, int64_t m, hipStream_t st) {
  int n = set_tiles<S, GRAD>(a, m);
  a.round = std::is_same<S, Large>::value ? 256 : 0;
  if (a.round > 0) n += a.round / 2;
  hipLaunchKernelGGL((logits_tiles<S, BF16, GRAD, LOOSE>), dim3(n), dim3(S::NT), 0, st, a);
}

static_assert(256 * kLossMaxStride * 2 <= kLoadMask && 128 * kLossMaxStride * 4 <= kLoadMask,
              "a tile's rows lie before the masked loads");
static_assert(SmallF::BN == loss_tile_rows(0) && Medium::BN == loss_tile_rows(1),
              "the workspace holds a pair per tile");

// Width of the tiles that `pick_logits` takes, as the loss counts its pairs.
int64_t logits_tile_rows(int64_t m, int64_t rows, int dtype, bool loose) {
  if (dtype == 1) return !loose && large_logits(m, rows) ? Large::BN : Medium::BN;
  return m > 32 && small_tiles(rows, m) ? SmallF::BN : MediumF::BN;
}

// `rows`: the table's rows by which the tiles are chosen, the same for all pieces of
// a loss.
template <bool GRAD, bool LOOSE>
void pick_logits(const Logits &a, int64_t m, int64_t rows, int dtype, hipStream_t st) {
  if (dtype == 0) {
    if (m <= 32) run_logits<LowF, false, GRAD, LOOSE>(a, m, st);
    else if (small_tiles(rows, m)) run_logits<SmallF, false, GRAD, LOOSE>(a, m, st);
    else run_logits<MediumF, false, GRAD, LOOSE>(a, m, st);
  } else if (m <= 32) {
    run_logits<Low32, true, GRAD, LOOSE>(a, m, st);
  } else if (m <= 64) {
    run_logits<Low64, true, GRAD, LOOSE>(a, m, st);
  } else if (LOOSE || !large_logits(m, rows)) {
    run_logits<Medium, true, GRAD, LOOSE>(a, m, st);
  } else if constexpr (GRAD && !LOOSE) {
    run_logits<Large, true, true, false>(a, m, st);
  } else if constexpr (!LOOSE) {
    Logits b = a;
    const int n = set_tiles<Large, false>(b, m);
    b.round = 256;
    hipLaunchKernelGGL(loss_tiles<Large>, dim3(n < b.round ? n : b.round), dim3(Large::NT), 0, st,
                       b);
  }
}

// Sets a's tiles of shape S; returns how many.
template <class S, int PARTS>
int set_tiles(Products &a) {
  a.x_tiles_n = blocks(a.dim, S::BN);
  a.x_tiles_m = blocks(a.rows, S::BM);
  a.w_tiles_n = blocks(a.dim, S::BN);
  a.w_tiles_m = blocks(a.cols, S::BM);
  return ((PARTS & 1) ? a.x_tiles_n * a.x_tiles_m * a.splits : 0) +
         ((PARTS & 2) ? a.w_tiles_n * a.w_tiles_m : 0);
}

template <class S, bool BF16, int PARTS, bool LOOSE>
void run_products(Products a, hipStream_t st) {
  const int n = set_tiles<S, PARTS>(a);
  if (n > 0)
    hipLaunchKernelGGL((grad_tiles<S, BF16, PARTS, LOOSE>), dim3(n), dim3(S::NT), 0, st, a);
}

// Splits of the sum over the vocabulary so that about `want` workgroups of
// tiles of n x m share it.
int64_t splits_for(int64_t rows, int64_t dim, int64_t cols, int64_t bn, int64_t bm, int64_t want,
                   int64_t most) {
  const int64_t tiles = blocks(dim, bn) * static_cast<int64_t>(blocks(rows, bm));
  int64_t s = want / tiles;
  s = loss_min(s, (cols + kLossSplitRows - 1) / kLossSplitRows);
  return loss_max(1, loss_min(s, most));
}

// The two products of a piece.  `splits` is fixed for all pieces of a call.
template <bool LOOSE>
void pick_products(const Products &a, int dtype, bool gx, bool gw, hipStream_t st) {
  if (dtype == 0) {
    const bool small = small_products(a.rows, a.dim, a.cols, a.splits, gw);
    if (gx && gw && a.rows > 32) {
      if (small) run_products<SmallF, false, 3, LOOSE>(a, st);
      else run_products<MediumF, false, 3, LOOSE>(a, st);
      return;
    }
    if (gx) {
      if (a.rows <= 32) run_products<LowF, false, 1, LOOSE>(a, st);
      else if (small) run_products<SmallF, false, 1, LOOSE>(a, st);
      else run_products<MediumF, false, 1, LOOSE>(a, st);
    }
    if (gw) {
      if (small) run_products<SmallF, false, 2, LOOSE>(a, st);
      else run_products<MediumF, false, 2, LOOSE>(a, st);
    }
    return;
  }
  if constexpr (!LOOSE) {
    if (large_products(a.rows, a.dim)) {
      if (gx && gw) run_products<Large, true, 3, false>(a, st);
      else if (gx) run_products<Large, true, 1, false>(a, st);
      else run_products<Large, true, 2, false>(a, st);
      return;
    }
  }
  if (gx && gw && a.rows > 64) {
    run_products<Medium, true, 3, LOOSE>(a, st);
    return;
  }
  if (gx && a.rows <= 32) run_products<Low32, true, 1, LOOSE>(a, st);
  else if (gx && a.rows <= 64) run_products<Low64, true, 1, LOOSE>(a, st);
  else if (gx) run_products<Medium, true, 1, LOOSE>(a, st);
  if (gw) run_products<Medium, true, 2, LOOSE>(a, st);
}

int64_t pick_splits(int64_t rows, int64_t dim, int64_t cols, int dtype, bool loose, bool gw,
                    int64_t most) {
  const int64_t side = rows <= 32 ? 32 : (rows <= 64 && dtype == 1) ? 64 : 128;
  if (dtype == 1 && !loose && large_products(rows, dim))
    return splits_for(rows, dim, cols, 256, 256, 256, most);
  const int64_t s = splits_for(rows, dim, cols, 128, side, 512, most);
  if (dtype == 1 || rows <= 32 || !small_products(rows, dim, cols, s, gw)) return s;
  return splits_for(rows, dim, cols, 64, 64, 512, most);
}

void run_finish(const Products &a, const LossRows &r, const LossGrads &g, const int32_t *place,
                hipStream_t st) {
  const int64_t groups = finish_groups(r.m, r.dim), wide = loss_min(groups, kFinishWidth);
  const dim3 grid(static_cast<unsigned>(wide), static_cast<unsigned>((groups + wide - 1) / wide));
  const int64_t stride = a.rows * a.ld_sums;
  if (g.gxt == 1)
    hipLaunchKernelGGL(finish_grad_x<true>, grid, dim3(256), 0, st, a.sums, a.ld_sums, stride,
                       a.splits, place, a.scale, r.m, r.dim, g.gx);
  else
    hipLaunchKernelGGL(finish_grad_x<false>, grid, dim3(256), 0, st, a.sums, a.ld_sums, stride,
                       a.splits, place, a.scale, r.m, r.dim, g.gx);
}

// The gradients of an empty batch: zeros.
int zero_table(const LossRows &r, const LossGrads &g, hipStream_t st) {
  if (g.gw == nullptr || g.accumulate) return 0;
  const int64_t step = launch_rows(r.dim);
  for (int64_t row = 0; row < r.rows; row += step) {
    Products a{};
    a.dim = r.dim, a.cols = loss_min(step, r.rows - row), a.gw_bf16 = g.gwt == 1;
    a.gw = static_cast<char *>(g.gw) + row * r.dim * (a.gw_bf16 ? 2 : 4);
    // (no rows: no operand is read)
    if (r.dtype == 1) run_products<Medium, true, 2, false>(a, st);
    else run_products<MediumF, false, 2, false>(a, st);
    const int rc = last_error();
    if (rc != 0) return rc;
  }
  return 0;
}

}  // namespace

int launch_lmhead_xent(const LossRows &r, float *shard_lse, float *target_logit, void *workspace,
                       void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // clear a stale error so the status below is this launch's
  const LossLayout l = loss_layout(kLossForward, r.m, r.dim, r.rows, r.dtype);
  const int64_t e = r.dtype == 1 ? 2 : 4;
  int rc = 0;
  Logits a{};
  a.m = r.m;
  a.any = Targets{r.targets, r.itype, r.vocab_start, r.vocab, r.rows};
  const bool w_in_place = loads_in_place(r.w, r.dim, r.dtype);
  const bool loose = !w_in_place && loose_rows(kLossForward, r.m, r.rows, r.dim);
  if (r.m <= kWholeRows && (loose || loads_in_place(r.x, r.dim, r.dtype))) {
    a.x = r.x, a.ldx = r.dim, a.x_dim = r.dim;
  } else {
    rc = run_collect(r, l, nullptr, nullptr, shard_lse, target_logit, workspace, st);
    if (rc != 0) return rc;
    a.x = at(workspace, l.x), a.ldx = l.dim_pad, a.x_dim = l.dim_pad;
    a.count = reinterpret_cast<const int32_t *>(at(workspace, l.count));
  }
  a.row_of = reinterpret_cast<const int32_t *>(at(workspace, l.row_of));
  a.target = reinterpret_cast<const int32_t *>(at(workspace, l.target));
  a.pairs = reinterpret_cast<float *>(at(workspace, l.pairs)), a.pair_ld = r.m;
  a.target_logit = target_logit;
  const int64_t tile_rows = logits_tile_rows(r.m, r.rows, r.dtype, loose);
  const int64_t step = loss_piece(l, r.m, r.rows, !w_in_place && !loose);  // (whole tiles)
  for (int64_t row = 0; row < r.rows; row += step) {
    const char *w = static_cast<const char *>(r.w) + row * r.dim * e;
    a.w_rows = loss_min(step, r.rows - row), a.row0 = row, a.tile0 = row / tile_rows;
    a.w = w, a.ldw = a.w_dim = a.k = r.dim;
    if (!w_in_place && !loose) {
      run_copy(w, r.dim, a.w_rows, r.dim, at(workspace, l.table), l.dim_pad, r.dtype, st);
      a.w = at(workspace, l.table), a.ldw = a.w_dim = l.dim_pad;
    }
    if (loose) pick_logits<false, true>(a, r.m, r.rows, r.dtype, st);
    else pick_logits<false, false>(a, r.m, r.rows, r.dtype, st);
    rc = last_error();
    if (rc != 0) return rc;
  }
  const int tiles = blocks(r.rows, tile_rows);
  if (r.m <= 256)
    hipLaunchKernelGGL(join_pairs<1>, dim3(static_cast<unsigned>(r.m)), dim3(1024), 0, st,
                       a.pairs, a.pair_ld, tiles, a.count, a.m, a.any, a.row_of, shard_lse,
                       target_logit);
  else
    hipLaunchKernelGGL(join_pairs<16>, dim3(blocks(r.m, 16)), dim3(1024), 0, st, a.pairs,
                       a.pair_ld, tiles, a.count, a.m, a.any, a.row_of, shard_lse, target_logit);
  return last_error();
}

int launch_xent_loss(const float *const *shard_lse, const float *const *target_logit, int n_parts,
                     int64_t m, int64_t vocab, const void *targets, int itype, float *loss,
                     float *lse, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  Parts p{};
  for (int i = 0; i < n_parts; ++i) p.lse[i] = shard_lse[i], p.target[i] = target_logit[i];
  const dim3 grid(blocks(m, 256));
  if (itype == 0)
    hipLaunchKernelGGL(xent_loss<int32_t>, grid, dim3(256), 0, st, p, n_parts, m, vocab,
                       static_cast<const int32_t *>(targets), loss, lse);
  else
    hipLaunchKernelGGL(xent_loss<int64_t>, grid, dim3(256), 0, st, p, n_parts, m, vocab,
                       static_cast<const int64_t *>(targets), loss, lse);
  return last_error();
}

int launch_lmhead_xent_grad(const LossRows &r, const float *lse, const float *grad_loss,
                            const LossGrads &g, void *workspace, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (r.m == 0) return zero_table(r, g, st);
  const LossLayout l = loss_layout(kLossGrad, r.m, r.dim, r.rows, r.dtype);
  const int64_t e = r.dtype == 1 ? 2 : 4;
  int rc = run_collect(r, l, lse, grad_loss, nullptr, nullptr, workspace, st);
  if (rc != 0) return rc;
  const bool w_in_place = loads_in_place(r.w, r.dim, r.dtype);
  const bool loose = !w_in_place && loose_rows(kLossGrad, r.m, r.rows, r.dim);
  const bool copied = !w_in_place && !loose;
  const int64_t step = grad_piece(l, r.m, r.rows, r.dtype, copied);
  Logits a{};
  a.x = at(workspace, l.x), a.ldx = a.x_dim = l.dim_pad, a.k = r.dim;
  a.count = reinterpret_cast<const int32_t *>(at(workspace, l.count));
  a.target = reinterpret_cast<const int32_t *>(at(workspace, l.target));
  a.lse = reinterpret_cast<const float *>(at(workspace, l.lse));
  a.ratio = reinterpret_cast<const float *>(at(workspace, l.ratio));
  Products p{};
  p.x = a.x, p.ldx = a.ldx, p.rows = r.m, p.count = a.count, p.dim = r.dim;
  p.sums = reinterpret_cast<float *>(at(workspace, l.sums)), p.ld_sums = l.dim_pad;
  p.scale = reinterpret_cast<const float *>(at(workspace, l.count)) + 1;
  p.gw_bf16 = g.gwt == 1, p.accumulate = g.accumulate;
  p.splits = static_cast<int>(pick_splits(r.m, r.dim, loss_min(step, r.rows), r.dtype, loose,
                                          g.gw != nullptr,
                                          loss_most_splits(r.m, l.dim_pad, r.rows)));
  p.per_split = loss_up((loss_min(step, r.rows) + p.splits - 1) / p.splits, 64);
  // the piece of d that begins at `row`
  auto piece_logits = [&](int64_t row) {
    const char *w = static_cast<const char *>(r.w) + row * r.dim * e;
    a.w_rows = loss_min(step, r.rows - row), a.row0 = row, a.ldd = loss_up(a.w_rows, 64);
    a.d = at(workspace, l.piece[row / step % 2]);
    a.w = w, a.ldw = a.w_dim = r.dim;
    if (copied) {
      run_copy(w, r.dim, a.w_rows, r.dim, at(workspace, l.table), l.dim_pad, r.dtype, st);
      a.w = at(workspace, l.table), a.ldw = a.w_dim = l.dim_pad;
    }
  };
  // its products, once `a` is it
  auto piece_products = [&]() {
    p.d = a.d, p.ldd = a.ldd, p.cols = a.w_rows, p.w = a.w, p.ldw = a.ldw, p.first = a.row0 == 0;
    p.gw = g.gw == nullptr ? nullptr
                           : static_cast<char *>(g.gw) + a.row0 * r.dim * (g.gwt == 1 ? 2 : 4);
  };
  // (a copied table leaves no second copy to read beside the products of the first)
  const bool together =
      r.dtype == 1 && w_in_place && large_products(r.m, r.dim) && g.gx && g.gw;
  for (int64_t row = 0; row < r.rows; row += step) {
    if (!together || row == 0) {
      piece_logits(row);
      if (loose) pick_logits<true, true>(a, r.m, a.w_rows, r.dtype, st);
      else pick_logits<true, false>(a, r.m, a.w_rows, r.dtype, st);
    }
    piece_products();
    if (together && row + step < r.rows) {
      piece_logits(row + step);
      const int n = set_tiles<Large, 3>(p), more = set_tiles<Large, true>(a, r.m);
      hipLaunchKernelGGL(grad_and_logits_tiles<Large>, dim3(n + more), dim3(Large::NT), 0, st, p,
                         n, a);
    } else {
      if (loose) pick_products<true>(p, r.dtype, g.gx != nullptr, g.gw != nullptr, st);
      else pick_products<false>(p, r.dtype, g.gx != nullptr, g.gw != nullptr, st);
    }
    rc = last_error();
    if (rc != 0) return rc;
  }
  if (g.gx != nullptr)
    run_finish(p, r, g, reinterpret_cast<const int32_t *>(at(workspace, l.place)), st);
  return last_error();
}

int launch_lmhead_grad(const void *d, int64_t ld, const LossRows &r, const LossGrads &g,
                       void *workspace, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (r.m == 0) return zero_table(r, g, st);
  const LossLayout l = loss_layout(kHeadGrad, r.m, r.dim, r.rows, r.dtype);
  const int64_t e = r.dtype == 1 ? 2 : 4;
  const auto [d_copied, w_copied, x_copied, loose] = head_grad_rows(d, ld, r, g);
  const int64_t step = head_grad_piece(l, r.m, r.rows, r.dtype, d_copied, w_copied);
  Products p{};
  p.rows = r.m, p.dim = r.dim;
  p.sums = reinterpret_cast<float *>(at(workspace, l.sums)), p.ld_sums = l.dim_pad;
  p.gw_bf16 = g.gwt == 1, p.accumulate = g.accumulate;
  p.splits = static_cast<int>(pick_splits(r.m, r.dim, loss_min(step, r.rows), r.dtype, loose,
                                          g.gw != nullptr,
                                          loss_most_splits(r.m, l.dim_pad, r.rows)));
  p.per_split = loss_up((loss_min(step, r.rows) + p.splits - 1) / p.splits, 64);
  p.x = r.x, p.ldx = r.dim;
  if (x_copied) {
    run_copy(r.x, r.dim, r.m, r.dim, at(workspace, l.x), l.dim_pad, r.dtype, st);
    p.x = at(workspace, l.x), p.ldx = l.dim_pad;
  }
  for (int64_t row = 0; row < r.rows; row += step) {
    const int64_t cols = loss_min(step, r.rows - row);
    p.cols = cols;
    p.d = static_cast<const char *>(d) + row * e, p.ldd = ld;
    if (d_copied) {
      run_copy(p.d, ld, r.m, cols, at(workspace, l.piece[0]), loss_up(cols, 64), r.dtype, st);
      p.d = at(workspace, l.piece[0]), p.ldd = loss_up(cols, 64);
    }
    p.w = static_cast<const char *>(r.w) + row * r.dim * e, p.ldw = r.dim;
    if (w_copied) {
      run_copy(p.w, r.dim, cols, r.dim, at(workspace, l.table), l.dim_pad, r.dtype,
               st);
      p.w = at(workspace, l.table), p.ldw = l.dim_pad;
    }
    p.gw = g.gw == nullptr ? nullptr
                           : static_cast<char *>(g.gw) + row * r.dim * (g.gwt == 1 ? 2 : 4);
    p.first = row == 0;
    if (loose) pick_products<true>(p, r.dtype, g.gx != nullptr, g.gw != nullptr, st);
    else pick_products<false>(p, r.dtype, g.gx != nullptr, g.gw != nullptr, st);
    const int rc = last_error();
    if (rc != 0) return rc;
  }
  if (g.gx != nullptr) run_finish(p, r, g, nullptr, st);
  return last_error();
}

}  // namespace vpe
