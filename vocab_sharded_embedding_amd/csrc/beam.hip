// Beam search over the vocabulary-sharded logits for gfx950: the selection
// over beams and vocabulary, the merge of the shards' picks, and the
// reordering of per-beam states.
//
// Selection reads every logit once; its picks are a few keys.  A candidate is
// a 64-bit key (order of the score, then the lower place), and all keys of a
// sequence are distinct, so "the k best" is one definite set.
//  - A workgroup holds a chunk of a row in registers, kItems scores per
//    thread.  The k-th largest of the threads' best keys is a bound that at
//    least k keys reach, and only the k threads at or above it hold any that
//    do: at most k * kItems candidates, usually little more than k.  Those go
//    to LDS, where each finds its rank by counting.
//  - A row is cut into slices, one workgroup each; a second kernel joins the
//    slices' sorted lists of all beams of a sequence.  With L lists the k-th
//    largest of the lists' heads is such a bound again: at most k lists reach
//    it, so at most k * k candidates.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "vpe_device.h"
#include "vpe_train_launch.h"

namespace vpe {
namespace {

using namespace dev;

constexpr int kBlock = 256;
constexpr int kMaxPicks = 64;
constexpr int kItems = 32;                  // scores per thread and chunk
constexpr int kChunk = kBlock * kItems;     // columns per chunk
constexpr int kMaxSlices = 32;              // lists per row

// Unsigned integers ordered like the scores, NaN below all.
__device__ __forceinline__ uint32_t order_of(float c) {
  const uint32_t u = __float_as_uint(c);
  const uint32_t o = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return c != c ? 0u : o;
}
__device__ __forceinline__ float score_of(uint32_t o) {
  if (o == 0) return __uint_as_float(0x7fc00000u);
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}

template <bool BF16> struct Row;
template <> struct Row<true> {
  static constexpr int kEpv = 8;
  typedef u32x4 __attribute__((aligned(2))) loose;
  static __device__ __forceinline__ float one(const void *base, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(base)[i]) << 16);
  }
};
template <> struct Row<false> {
  static constexpr int kEpv = 4;
  typedef u32x4 __attribute__((aligned(4))) loose;
  static __device__ __forceinline__ float one(const void *base, int64_t i) {
    return static_cast<const float *>(base)[i];
  }
};

// The rank of `mine` among keys[0, n): how many are larger, or equal with a
// lower index (keys of different candidates differ; key 0 may repeat).
__device__ __forceinline__ int rank_among(const uint64_t *keys, int n, uint64_t mine, int index) {
  int rank = 0;
  for (int j = 0; j < n; ++j) rank += keys[j] > mine || (keys[j] == mine && j < index);
  return rank;
}

struct BeamArgs {
  const char *base;
  int64_t ld_bytes;
  int64_t cols, vocab_start, vocab;
  const float *lse, *scores;
  int beams, picks, slices;
  int64_t slice;  // columns per slice, a multiple of the vector length
};

// blockIdx.x = row * slices + s: the slice's best keys, descending, 0 beyond.
template <bool BF16>
__global__ __launch_bounds__(kBlock) void beam_slice(BeamArgs a, uint64_t *__restrict__ out) {
  typedef Row<BF16> R;
  constexpr int kEpv = R::kEpv, kVecs = kItems / kEpv;
  __shared__ __attribute__((aligned(16))) uint64_t top[kBlock];
  __shared__ __attribute__((aligned(16))) uint64_t cand[kMaxPicks * kItems + kMaxPicks];
  __shared__ uint64_t best[kMaxPicks];
  __shared__ uint64_t bound;
  __shared__ int n_cand;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / static_cast<unsigned>(a.slices);
  const int s = static_cast<int>(blockIdx.x - row * a.slices);
  const int64_t c0 = s * a.slice;
  const int64_t n = c0 + a.slice < a.cols ? a.slice : a.cols - c0;
  const char *p = a.base + row * a.ld_bytes + c0 * (BF16 ? 2 : 4);
  const float lse = a.lse[row], score = a.scores[row];
  // places count down from the beam's first token, as the low key half does
  const uint32_t low0 = 0xFFFFFFFFu - static_cast<uint32_t>((row % a.beams) * a.vocab +
                                                            a.vocab_start + c0);
  const int k = a.picks;

  if (tid < k) best[tid] = 0;
  __syncthreads();
  for (int64_t at = 0; at < n; at += kChunk) {
    uint32_t ord[kItems];
    uint32_t low[kVecs];
    uint64_t mine = 0;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int64_t j = at + static_cast<int64_t>(u * kBlock + tid) * kEpv;
      low[u] = low0 - static_cast<uint32_t>(j);
      float v[kEpv];
      const int left = n - j < kEpv ? static_cast<int>(n - j) : kEpv;
      if (left == kEpv) {
        Vec<BF16, kEpv>::widen(*reinterpret_cast<const typename R::loose *>(p + j * (BF16 ? 2 : 4)), v);
      } else {
#pragma unroll
        for (int e = 0; e < kEpv; ++e) v[e] = e < left ? R::one(p, j + e) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < kEpv; ++e) {
        const float c = ((v[e] - lse) + score) + 0.f;  // -0 becomes +0
        ord[u * kEpv + e] = order_of(c);
        const uint64_t key = (static_cast<uint64_t>(ord[u * kEpv + e]) << 32) | (low[u] - e);
        if (e < left && key > mine) mine = key;
      }
    }
    const uint64_t floor_key = best[k - 1];
    top[tid] = mine;
    if (tid == 0) bound = 0, n_cand = 0;
    __syncthreads();
    if (rank_among(top, kBlock, mine, tid) == k - 1) bound = mine;
    __syncthreads();
    const uint64_t least = bound > floor_key ? bound : floor_key;
    if (mine != 0 && mine >= least) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int64_t j = at + static_cast<int64_t>(u * kBlock + tid) * kEpv;
#pragma unroll
        for (int e = 0; e < kEpv; ++e) {
          const uint64_t key = (static_cast<uint64_t>(ord[u * kEpv + e]) << 32) | (low[u] - e);
          if (j + e < n && key >= least) cand[atomicAdd(&n_cand, 1)] = key;
        }
      }
    }
    if (tid < k && best[tid] != 0) cand[atomicAdd(&n_cand, 1)] = best[tid];
    __syncthreads();
    const int nc = n_cand;
    if (tid < k) best[tid] = 0;
    __syncthreads();
    for (int i = tid; i < nc; i += kBlock) {
      const uint64_t key = cand[i];
      const int r = rank_among(cand, nc, key, i);
      if (r < k) best[r] = key;
    }
    __syncthreads();
  }
  if (tid < k) out[static_cast<int64_t>(blockIdx.x) * k + tid] = best[tid];
}

// ---------------------------------------------------------------------------
// sorted lists of k keys joined: lists l < n_lists of block `seq`
// ---------------------------------------------------------------------------
struct Adjacent {  // the slices of a sequence's beams follow each other
  const uint64_t *keys;
  int64_t n_lists;
  int k;
  __device__ __forceinline__ const uint64_t *list(int64_t seq, int l) const {
    return keys + (seq * n_lists + l) * k;
  }
};
struct PerPart {  // one array per shard
  const uint64_t *part[64];
  int k;
  __device__ __forceinline__ const uint64_t *list(int64_t seq, int l) const {
    return part[l] + seq * k;
  }
};

// best[0, k) (LDS) = the k largest keys of the lists, descending, 0 beyond.
template <class Lists>
__device__ __forceinline__ void join_lists(const Lists &lists, int64_t seq, int n_lists, int k,
                                           uint64_t *top, uint64_t *cand, int cap, uint64_t *best,
                                           uint64_t *bound, int *n_cand) {
  const int tid = threadIdx.x;
  // a bound that k heads reach: the k-th largest of the threads' best heads,
  uint64_t mine = 0;
  for (int l = tid; l < n_lists; l += kBlock) {
    const uint64_t h = lists.list(seq, l)[0];
    if (h > mine) mine = h;
  }
  top[tid] = mine;
  if (tid == 0) *bound = 0, *n_cand = 0;
  if (tid < k) best[tid] = 0;
  __syncthreads();
  if (rank_among(top, kBlock, mine, tid) == k - 1) *bound = mine;
  __syncthreads();
  uint64_t least = *bound;
  if (n_lists > kBlock) {
    // then exactly the k-th largest head, among the heads that reach it
    for (int l = tid; l < n_lists; l += kBlock) {
      const uint64_t h = lists.list(seq, l)[0];
      if (h != 0 && h >= least) {
        const int i = atomicAdd(n_cand, 1);
        if (i < cap) cand[i] = h;
      }
    }
    __syncthreads();
    const int nh = *n_cand < cap ? *n_cand : cap;
    for (int i = tid; i < nh; i += kBlock)
      if (rank_among(cand, nh, cand[i], i) == k - 1) *bound = cand[i];
    __syncthreads();
    least = *bound;
    if (tid == 0) *n_cand = 0;
    __syncthreads();
  }
  for (int l = tid; l < n_lists; l += kBlock) {
    const uint64_t *list = lists.list(seq, l);
    for (int i = 0; i < k; ++i) {
      const uint64_t key = list[i];
      if (key == 0 || key < least) break;
      const int at = atomicAdd(n_cand, 1);
      if (at < cap) cand[at] = key;
    }
  }
  __syncthreads();
  const int nc = *n_cand < cap ? *n_cand : cap;
  for (int i = tid; i < nc; i += kBlock) {
    const uint64_t key = cand[i];
    const int r = rank_among(cand, nc, key, i);
    if (r < k) best[r] = key;
  }
  __syncthreads();
}

// k lists of k keys reach the bound at most; at most kMaxSlices * 64 / kBlock
// heads per thread do (fewer).
constexpr int kListCap = kMaxPicks * kMaxPicks;

#define VPE_JOIN_LDS                                                    \
  __shared__ __attribute__((aligned(16))) uint64_t top[kBlock];         \
  __shared__ __attribute__((aligned(16))) uint64_t cand[kListCap];      \
  __shared__ uint64_t best[kMaxPicks];                                  \
  __shared__ uint64_t bound;                                            \
  __shared__ int n_cand

__global__ __launch_bounds__(kBlock) void beam_join(Adjacent lists, uint64_t *__restrict__ keys) {
  VPE_JOIN_LDS;
  const int64_t seq = blockIdx.x;
  join_lists(lists, seq, static_cast<int>(lists.n_lists), lists.k, top, cand, kListCap, best,
             &bound, &n_cand);
  if (static_cast<int>(threadIdx.x) < lists.k) keys[seq * lists.k + threadIdx.x] = best[threadIdx.x];
}

__global__ __launch_bounds__(kBlock) void beam_merge_rows(PerPart lists, int n_parts, int64_t vocab,
                                                         float *__restrict__ score,
                                                         int64_t *__restrict__ parent,
                                                         int64_t *__restrict__ token) {
  VPE_JOIN_LDS;
  const int64_t seq = blockIdx.x;
  const int k = lists.k, tid = threadIdx.x;
  uint64_t key = 0;
  if (n_parts == 1) {
    if (tid < k) key = lists.part[0][seq * k + tid];
  } else {
    join_lists(lists, seq, n_parts, k, top, cand, kListCap, best, &bound, &n_cand);
    if (tid < k) key = best[tid];
  }
  if (tid < k) {
    const int64_t i = seq * k + tid;
    const uint64_t place = 0xFFFFFFFFull - (key & 0xFFFFFFFFull);
    const uint64_t b = place / static_cast<uint64_t>(vocab);
    score[i] = key == 0 ? -__builtin_huge_valf() : score_of(static_cast<uint32_t>(key >> 32));
    parent[i] = key == 0 ? -1 : static_cast<int64_t>(b);
    token[i] = key == 0 ? -1 : static_cast<int64_t>(place - b * static_cast<uint64_t>(vocab));
  }
}

// ---------------------------------------------------------------------------
// reordering of states
// ---------------------------------------------------------------------------
// 2^log2g lanes serve a unit: `span` vectors (of V) of one destination row.
template <typename V>
__global__ __launch_bounds__(kBlock) void reorder_rows(const V *__restrict__ src, int64_t row0,
                                                      int64_t n_rows, int64_t rows_per_outer,
                                                      int beams_in, int beams_out, int64_t n_seqs,
                                                      int64_t vr, int64_t units_per_row,
                                                      int64_t span, int log2g,
                                                      const int64_t *__restrict__ parent,
                                                      int64_t ld_parent, V *__restrict__ dst) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  const int64_t unit = t >> log2g;
  const int64_t rel = unit / units_per_row;
  if (rel >= n_rows) return;
  const int group = 1 << log2g;
  const int64_t v0 = (unit - rel * units_per_row) * span + (t & (group - 1));
  const int64_t v1 = (unit - rel * units_per_row + 1) * span < vr
                         ? (unit - rel * units_per_row + 1) * span
                         : vr;
  const int64_t row = row0 + rel;
  const int64_t o = row / rows_per_outer;
  const int64_t in = row - o * rows_per_outer;  // s * beams_out + b
  const int64_t s = in / beams_out;
  const int64_t from = parent[s * ld_parent + (in - s * beams_out)];
  const bool valid = static_cast<uint64_t>(from) < static_cast<uint64_t>(beams_in);
  const V *from_row = src + ((o * n_seqs + s) * beams_in + (valid ? from : 0)) * vr;
  V *to_row = dst + row * vr;
  constexpr int kDeep = 4;
  for (int64_t v = v0; v < v1; v += kDeep * group) {
    V r[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      r[u] = V(0);
      if (valid && v + u * group < v1) r[u] = from_row[v + u * group];
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
      if (v + u * group < v1) __builtin_nontemporal_store(r[u], to_row + v + u * group);
  }
}

template <typename V>
int launch_reorder(const void *src, int64_t outer, int64_t n_seqs, int beams_in, int64_t vr,
                   const int64_t *parent, int64_t ld_parent, int beams_out, void *dst,
                   hipStream_t st) {
  int log2g = 0;
  while (log2g < 6 && (int64_t(1) << log2g) < vr) ++log2g;
  // a wave moves 4 vectors per lane, more where a row has over 2^20 such units
  const int64_t span = vr < 64 * 4 ? vr : 64 * 4 * ((vr >> 28) + 1);
  const int64_t units = (vr + span - 1) / span;
  const int64_t rows = outer * n_seqs * beams_out;
  const int64_t step = std::max<int64_t>(1, ((int64_t(1) << 30) >> log2g) / units);
  for (int64_t r = 0; r < rows; r += step) {
    const int64_t nr = std::min(step, rows - r);
    const int64_t threads = (nr * units) << log2g;
    hipLaunchKernelGGL((reorder_rows<V>), dim3(static_cast<unsigned>((threads + kBlock - 1) / kBlock)),
                       dim3(kBlock), 0, st, static_cast<const V *>(src), r, nr,
                       n_seqs * beams_out, beams_in, beams_out, n_seqs, vr, units, span, log2g,
                       parent, ld_parent, static_cast<V *>(dst));
  }
  return static_cast<int>(hipGetLastError());
}

}  // namespace

int64_t beam_slices(int64_t rows, int64_t cols) {
  (void)rows;
  const int64_t slices = (cols + kChunk - 1) / kChunk;
  return std::min<int64_t>(slices, kMaxSlices);
}

int launch_beam_select(const void *base, int64_t ld, int dtype, int64_t n_seqs, int beams,
                       int64_t cols, int64_t vocab_start, int64_t vocab, const float *lse,
                       const float *scores, int picks, uint64_t *keys, uint64_t *slice_keys,
                       void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // clear a stale error so the status returned is this launch's
  const int64_t want = beam_slices(n_seqs * beams, cols);
  const int64_t slice = ((cols + want - 1) / want + 7) / 8 * 8;
  const int slices = static_cast<int>((cols + slice - 1) / slice);
  const BeamArgs a{static_cast<const char *>(base), ld * (dtype == 1 ? 2 : 4), cols, vocab_start,
                   vocab, lse, scores, beams, picks, slices, slice};
  const dim3 grid(static_cast<unsigned>(n_seqs * beams * slices));
  if (dtype == 1)
    hipLaunchKernelGGL((beam_slice<true>), grid, dim3(kBlock), 0, st, a, slice_keys);
  else
    hipLaunchKernelGGL((beam_slice<false>), grid, dim3(kBlock), 0, st, a, slice_keys);
  const Adjacent lists{slice_keys, static_cast<int64_t>(beams) * slices, picks};
  hipLaunchKernelGGL(beam_join, dim3(static_cast<unsigned>(n_seqs)), dim3(kBlock), 0, st, lists,
                     keys);
  return static_cast<int>(hipGetLastError());
}

int launch_beam_merge(const uint64_t *const *keys, int n_parts, int64_t n_seqs, int picks,
                      int64_t vocab, float *score, int64_t *parent, int64_t *token, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  PerPart lists{};
  for (int r = 0; r < n_parts; ++r) lists.part[r] = keys[r];
  lists.k = picks;
  hipLaunchKernelGGL(beam_merge_rows, dim3(static_cast<unsigned>(n_seqs)), dim3(kBlock), 0, st,
                     lists, n_parts, vocab, score, parent, token);
  return static_cast<int>(hipGetLastError());
}

int launch_beam_reorder(const void *src, int64_t outer, int64_t n_seqs, int beams_in,
                        int64_t row_bytes, const int64_t *parent, int64_t ld_parent,
                        int beams_out, void *dst, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const uint64_t low = reinterpret_cast<uint64_t>(src) | reinterpret_cast<uint64_t>(dst) |
                       static_cast<uint64_t>(row_bytes);
#define VPE_REORDER(V, B) \
  launch_reorder<V>(src, outer, n_seqs, beams_in, row_bytes / B, parent, ld_parent, beams_out, dst, st)
  if ((low & 15) == 0) return VPE_REORDER(u32x4, 16);
  if ((low & 7) == 0) return VPE_REORDER(u32x2, 8);
  if ((low & 3) == 0) return VPE_REORDER(uint32_t, 4);
  if ((low & 1) == 0) return VPE_REORDER(uint16_t, 2);
  return VPE_REORDER(uint8_t, 1);
#undef VPE_REORDER
}

}  // namespace vpe
