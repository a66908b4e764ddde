// Beam search over the vocabulary-sharded logits for gfx950: the selection
// over beams and vocabulary, the merge of the shards' picks, and the
// reordering of per-beam states.
//
// Selection reads every logit once; its picks are a few keys.  A candidate is
// a 64-bit key (order of the score, then the lower place), and all keys of a
// sequence are distinct, so "the k best" is one definite set.
//  - A first kernel leaves the largest logit of every group of 64 vectors of a
//    row (of 8 where a sequence has few): a widening and half a maximum per
//    logit, no branches, bound by HBM.  The score rises with the logit, so the
//    group's best score follows from it.
//  - A second kernel, one workgroup per sequence, orders the groups of all
//    beams by (best score, lower place).  A candidate outside the k best groups
//    is beaten by k candidates, one in each, so only about k groups are read
//    again, and of those only the scores at the k-th group's best and above are
//    looked at: usually little more than k.
//  - The k-th largest of many keys is found by digits of 11 bits, counted in
//    LDS, of their distance from a score that 64 of them reach: one round for
//    scores that differ.  (Digits from the top of the key put most scores into
//    a few counters, whose atomics then follow each other: 18000 cycles for
//    6304 keys.  A selection by single bits, ballots in one wave, took 150 to
//    400 cycles a bit, and one per row slice 32 us for [256, 75968] logits.)
//  - Few candidates (kDirect) are ordered by the second kernel alone.
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
constexpr int kVecsAhead = 4;            // vectors in flight per lane
constexpr int64_t kRowsPerGrid = 32768;
constexpr int64_t kDirect = 16384;       // candidates a workgroup orders by itself
constexpr int kThreads = 1024;           // of that workgroup
constexpr int kDigitBits = 11;
constexpr int kBins = 1 << kDigitBits;
constexpr int kLoose = 48;               // 16 of them bits of the score's order
constexpr int kCap = 2048;               // keys collected
constexpr int kFew = 256;                // keys ordered by counting
constexpr int kHeld = 8192;              // groups whose best scores are held in LDS

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

template <bool BF16>
struct Row : Vec<BF16, BF16 ? 8 : 4> {
  static constexpr int kEpv = BF16 ? 8 : 4;
};

struct BeamArgs {
  const char *base;
  int64_t ld_bytes;
  int64_t cols, vocab_start, vocab;
  const float *lse, *scores;
  int beams, picks;
  int64_t groups;  // per row
  int group_log2;  // vectors per group: 2^6, or 2^3
};

// best[row * groups + g] = the largest logit of group g of the row, NaN if
// there is none (grid: vectors of the row / 1024, rows).  256 bf16 rows of 75968
// (39 MB) 8.8 us, 160 fp32 rows of 50257 (32 MB) 7.8 us: 4.4 and 4.1 TB/s, the
// first and last 2 us of it latency.
template <bool BF16>
__global__ __launch_bounds__(kBlock) void beam_groups(BeamArgs a, int64_t row0,
                                                     float *__restrict__ best) {
  typedef Row<BF16> R;
  constexpr int kEpv = R::kEpv, kSize = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63;
  const int64_t row = row0 + blockIdx.y;
  // waves take kVecsAhead times 64 vectors, from vector 64 * g0 on
  const int64_t g0 =
      (static_cast<int64_t>(blockIdx.x) * (kBlock / 64) + wave_in_block()) * kVecsAhead;
  if (g0 * 64 * kEpv >= a.cols) return;
  const char *p = a.base + row * a.ld_bytes;
  const uint32_t none = BF16 ? 0x7fc07fc0u : 0x7fc00000u;
  u32x4 raw[kVecsAhead];
#pragma unroll
  for (int u = 0; u < kVecsAhead; ++u) {
    const int64_t j = ((g0 + u) * 64 + lane) * kEpv;
    raw[u] = u32x4(none);
    if (j + kEpv <= a.cols) raw[u] = *reinterpret_cast<const typename R::loose *>(p + j * kSize);
  }
  // where +inf has a NaN score (a row whose log-sum-exp is +inf, a beam at
  // -inf) the others of its group come before it
  const float inf = __builtin_huge_valf();
  const float top = (inf - a.lse[row]) + a.scores[row];
  const bool no_inf = top != top;
  float mx[kVecsAhead];
#pragma unroll
  for (int u = 0; u < kVecsAhead; ++u) {
    float v[kEpv];
    Vec<BF16, kEpv>::widen(raw[u], v);
    if (no_inf) {
#pragma unroll
      for (int e = 0; e < kEpv; ++e) v[e] = v[e] == inf ? __uint_as_float(0x7fc00000u) : v[e];
    }
    mx[u] = v[0];
#pragma unroll
    for (int e = 1; e < kEpv; ++e) mx[u] = fmaxf(mx[u], v[e]);
    // the row's last columns where they do not fill a vector
    const int64_t j = ((g0 + u) * 64 + lane) * kEpv;
    if (j < a.cols && j + kEpv > a.cols) {
#pragma nounroll
      for (int64_t i = j; i < a.cols; ++i) {
        const float x = load_one<BF16>(p, i);
        if (!(no_inf && x == inf)) mx[u] = fmaxf(mx[u], x);
      }
    }
  }
  float *out = best + row * a.groups;
  if (a.group_log2 == 6) {
    float mine = 0.f;
#pragma unroll
    for (int u = 0; u < kVecsAhead; ++u) {
      const float m = wave_max(mx[u]);
      if (lane == u) mine = m;
    }
    if (lane < kVecsAhead && g0 + lane < a.groups) out[g0 + lane] = mine;
  } else {
    // lanes 7, 15, ... end with the maximum of their eight
#pragma unroll
    for (int u = 0; u < kVecsAhead; ++u) {
      float m = mx[u];
      m = fmaxf(m, dpp<0x111, 0xf>(m, m));
      m = fmaxf(m, dpp<0x112, 0xf>(m, m));
      m = fmaxf(m, dpp<0x114, 0xf>(m, m));
      const int64_t g = (g0 + u) * 8 + lane / 8;
      if ((lane & 7) == 7 && g < a.groups) out[g] = m;
    }
  }
}

// ---------------------------------------------------------------------------
// selection by one workgroup of kThreads
// ---------------------------------------------------------------------------
struct SelectLds {
  uint32_t bins[kBins];
  uint32_t sums[kThreads / 64], least[kThreads / 64];
  uint64_t cand[kCap];
  uint64_t few[kFew];
  float lse[kMaxPicks], score[kMaxPicks];  // of the sequence's beams
  uint32_t group[kFew];                    // groups read again
  uint32_t held[kHeld];                    // order of the groups' best scores
  int n;                                   // keys collected
  uint32_t rank[kFew];
  uint32_t digit, above, reach;
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
      static_cast<int>(v), static_cast<int>(v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp_u32<0x111>(v)), v = max(v, dpp_u32<0x112>(v));
  v = max(v, dpp_u32<0x114>(v)), v = max(v, dpp_u32<0x118>(v));
  v = max(v, dpp_u32<0x142>(v)), v = max(v, dpp_u32<0x143>(v));
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// A bound that at least k <= 64 of the keys (key 0 stands for none) reach, and
// at most k + slack unless they are copies of one key; 1 where there are fewer.
// At most kLoose low bits are left open below it: the score of the bound is
// within 2^-7 of the k-th largest, also where fewer keys than k + slack exist.
template <class Keys>
__device__ __forceinline__ uint64_t bound_of(const Keys &keys, int n, int k, int slack,
                                             SelectLds &s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_in_block();
  // the largest order; and the best, over the waves, of the least of the lanes'
  // largest, which 64 keys reach
  uint32_t most = 0;
#pragma unroll 2
  for (int i = tid; i < n; i += kThreads) most = max(most, static_cast<uint32_t>(keys(i) >> 32));
  const uint32_t wave_most = wave_max_u32(most), wave_least = ~wave_max_u32(~most);
  for (int i = tid; i < kBins; i += kThreads) s.bins[i] = 0;
  if (lane == 0) s.sums[wave] = wave_most, s.least[wave] = wave_least;
  __syncthreads();
  uint32_t top = 0, low = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) top = max(top, s.sums[w]), low = max(low, s.least[w]);
  const uint64_t base = static_cast<uint64_t>(low) << 32;
  const int span = 64 - __builtin_clz((top - low) | 1u);  // bits of a distance from base, >= 33

  uint64_t prefix = 0;
  int need = k;  // keys still to be found among those of the prefix
#pragma nounroll
  for (int open = span; open > 0;) {  // low bits not decided yet
    const int bits = open < kDigitBits ? open : kDigitBits;
    const int shift = open - bits;
    if (open != span) {
      for (int i = tid; i < kBins; i += kThreads) s.bins[i] = 0;
    }
    if (tid == 0) s.reach = 0;
    __syncthreads();
#pragma unroll 2
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = keys(i), far = key - base;
      if (key != 0 && key >= base && (open >= 64 || far >> open == prefix))
        atomicAdd(&s.bins[(far >> shift) & ((1 << bits) - 1)], 1u);
    }
    __syncthreads();
    // thread t: digits kBins - 1 - 2t and the one below; `above`: keys of larger ones
    static_assert(kBins == 2 * kThreads, "two digits per thread");
    const uint32_t hi = s.bins[kBins - 1 - 2 * tid], lo = s.bins[kBins - 2 - 2 * tid];
    uint32_t above = hi + lo;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const uint32_t up = __shfl_up(above, d);
      if (lane >= d) above += up;
    }
    if (lane == 63) s.sums[wave] = above;
    __syncthreads();
    above -= hi + lo;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) above += w < wave ? s.sums[w] : 0;
    const uint32_t want = static_cast<uint32_t>(need);
    if (above < want && above + hi + lo >= want) {
      const bool upper = above + hi >= want;
      s.digit = upper ? kBins - 1 - 2 * tid : kBins - 2 - 2 * tid;
      s.above = upper ? above : above + hi;
      s.reach = upper ? above + hi : above + hi + lo;
    }
    __syncthreads();
    const int reach = static_cast<int>(s.reach);  // keys of the digit and larger ones
    if (reach == 0) return 1;
    prefix = (prefix << bits) | s.digit;
    const int total = k - need + reach;
    need -= static_cast<int>(s.above);
    open = shift;
    __syncthreads();  // read before the next round (or call) clears it
    if ((total <= k + slack && open <= kLoose) || open == 0) return base + (prefix << open);
  }
  return 1;  // not reached
}

// out[0 .. s.n) = value(i) of the keys that reach the bound, in any order;
// s.n counts those past cap too.
template <class Keys, class Value, typename T>
__device__ __forceinline__ void collect(const Keys &keys, const Value &value, int n, uint64_t bound,
                                        T *out, int cap, SelectLds &s) {
  if (threadIdx.x == 0) s.n = 0;
  __syncthreads();
#pragma nounroll
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = keys(i);
    if (key != 0 && key >= bound) {
      const int at = atomicAdd(&s.n, 1);
      if (at < cap) out[at] = value(i, key);
    }
  }
  __syncthreads();
}

// The k best of s.few[0, n), best first, to thread t < k (0 beyond them).
__device__ __forceinline__ uint64_t best_of_few(int n, int k, SelectLds &s) {
  const int tid = threadIdx.x;
  if (n > kFew) n = kFew;  // copies of one key
  if (tid < k) s.cand[tid] = 0;
  if (tid < kFew) s.rank[tid] = 0;
  __syncthreads();
  // thread (i, part): how many of a quarter of the keys come before key i
  constexpr int kParts = kThreads / kFew;
  const int i = tid % kFew, share = (n + kParts - 1) / kParts;
  const int j0 = tid / kFew * share, j1 = j0 + share < n ? j0 + share : n;
  const uint64_t mine = i < n ? s.few[i] : 0;
  if (i < n) {
    uint32_t rank = 0;
#pragma unroll 8
    for (int j = j0; j < j1; ++j) rank += s.few[j] > mine || (s.few[j] == mine && j < i);
    atomicAdd(&s.rank[i], rank);
  }
  __syncthreads();
  if (tid < n && s.rank[tid] < static_cast<uint32_t>(k)) s.cand[s.rank[tid]] = mine;
  __syncthreads();
  return tid < k ? s.cand[tid] : 0;
}

struct TheKey {
  __device__ __forceinline__ uint64_t operator()(int, uint64_t key) const { return key; }
};
struct TheIndex {
  __device__ __forceinline__ uint32_t operator()(int i, uint64_t) const {
    return static_cast<uint32_t>(i);
  }
};
struct LdsKeys {
  const uint64_t *keys;
  __device__ __forceinline__ uint64_t operator()(int i) const { return keys[i]; }
};

// A sequence's candidates.
template <bool BF16>
struct Candidates {
  const BeamArgs &a;
  const SelectLds &s;
  const char *base;  // the sequence's first row
  const float *best; // its groups' largest logits
  static constexpr int kEpv = Row<BF16>::kEpv;

  __device__ __forceinline__ uint32_t group_cols() const { return kEpv << a.group_log2; }
  __device__ __forceinline__ uint64_t key(int beam, uint32_t col, float z) const {
    const float c = ((z - s.lse[beam]) + s.score[beam]) + 0.f;  // -0 becomes +0
    const uint32_t place = static_cast<uint32_t>(beam * a.vocab + a.vocab_start) + col;
    return (static_cast<uint64_t>(order_of(c)) << 32) | (0xFFFFFFFFu - place);
  }
  __device__ __forceinline__ uint64_t at(int beam, uint32_t col) const {
    return key(beam, col, load_one<BF16>(base + beam * a.ld_bytes, col));
  }
};
// all of them, one by one
template <bool BF16>
struct AllKeys {
  const Candidates<BF16> &c;
  __device__ __forceinline__ uint64_t operator()(int i) const {
    const uint32_t cols = static_cast<uint32_t>(c.a.cols), beam = static_cast<uint32_t>(i) / cols;
    return c.at(static_cast<int>(beam), static_cast<uint32_t>(i) - beam * cols);
  }
};
// group i's best, as if it were the group's first column
template <bool BF16>
struct GroupKeys {
  const Candidates<BF16> &c;
  __device__ __forceinline__ uint64_t operator()(int i) const {
    const uint32_t groups = static_cast<uint32_t>(c.a.groups);
    const uint32_t beam = static_cast<uint32_t>(i) / groups;
    return c.key(static_cast<int>(beam), (static_cast<uint32_t>(i) - beam * groups) * c.group_cols(),
                 c.best[i]);
  }
};
// the same with the order of the score held in LDS, and group numbers for
// places (they are ordered alike)
struct HeldKeys {
  const uint32_t *held;
  __device__ __forceinline__ uint64_t operator()(int i) const {
    return (static_cast<uint64_t>(held[i]) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(i));
  }
};
// those of the groups listed in s.group
template <bool BF16>
struct ListedKeys {
  const Candidates<BF16> &c;
  __device__ __forceinline__ uint64_t operator()(int i) const {
    const uint32_t cols = c.group_cols();
    const uint32_t group = c.s.group[static_cast<uint32_t>(i) / cols];
    const uint32_t groups = static_cast<uint32_t>(c.a.groups), beam = group / groups;
    const uint32_t col = (group - beam * groups) * cols + static_cast<uint32_t>(i) % cols;
    return col < c.a.cols ? c.at(static_cast<int>(beam), col) : 0;
  }
};

// One workgroup per sequence: its `picks` best keys, descending, 0 beyond.
// best == nullptr: few candidates, ordered one by one.  Bound by the latency of
// its steps, each waiting for the one before: 16 picks of 8 x 75968 in 8.4 us, 8
// of 4 x 151936 in 6.6, 64 of 32 x 50257 (6304 groups) in 12.2.
template <bool BF16>
__global__ __launch_bounds__(kThreads) void beam_pick(BeamArgs a, const float *__restrict__ best,
                                                     uint64_t *__restrict__ keys) {
  __shared__ SelectLds s;
  const int64_t seq = blockIdx.x;
  const int tid = threadIdx.x, k = a.picks;
  if (tid < a.beams) {
    s.lse[tid] = a.lse[seq * a.beams + tid];
    s.score[tid] = a.scores[seq * a.beams + tid];
  }
  __syncthreads();
  const Candidates<BF16> c{a, s, a.base + seq * a.beams * a.ld_bytes,
                           best ? best + seq * a.beams * a.groups : nullptr};
  if (best == nullptr) {
    const int n = static_cast<int>(a.beams * a.cols);
    const AllKeys<BF16> all{c};
    collect(all, TheKey{}, n, n <= kFew ? 1 : bound_of(all, n, k, kFew - k, s), s.few, kFew, s);
  } else {
    // the k best groups (up to as many again where that saves a round)
    const GroupKeys<BF16> groups{c};
    const int n = static_cast<int>(a.beams * a.groups);
    uint64_t bound;
    if (n <= kHeld) {
#pragma unroll 4
      for (int i = tid; i < n; i += kThreads)
        s.held[i] = static_cast<uint32_t>(groups(i) >> 32);
      __syncthreads();
      const HeldKeys held{s.held};
      bound = bound_of(held, n, k, k, s);
      collect(held, TheIndex{}, n, bound, s.group, kFew, s);
    } else {
      bound = bound_of(groups, n, k, k, s);
      collect(groups, TheIndex{}, n, bound, s.group, kFew, s);
    }
    const int listed = s.n;
    __syncthreads();
    // their scores at the bound and above
    typedef Row<BF16> R;
    constexpr int kEpv = R::kEpv;
    if (tid == 0) s.n = 0;
    __syncthreads();
    const uint32_t least = static_cast<uint32_t>(bound >> 32);
    constexpr int kDeep = 4;  // vectors in flight per thread
    const uint32_t ng = static_cast<uint32_t>(a.groups);
    const int vecs = listed << a.group_log2;
    for (int i0 = tid; i0 < vecs; i0 += kDeep * kThreads) {
      u32x4 raw[kDeep];
      uint32_t beam[kDeep], col[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) {
        const int i = i0 + u * kThreads;
        raw[u] = u32x4(0), beam[u] = 0, col[u] = 0xFFFFFFFFu - kEpv;  // past every row
        if (i < vecs) {
          const uint32_t group = s.group[i >> a.group_log2];
          beam[u] = group / ng;
          col[u] = (((group - beam[u] * ng) << a.group_log2) + (i & ((1 << a.group_log2) - 1))) * kEpv;
          if (col[u] + kEpv <= a.cols)
            raw[u] = *reinterpret_cast<const typename R::loose *>(
                c.base + beam[u] * a.ld_bytes + static_cast<int64_t>(col[u]) * R::kSize);
        }
      }
      // rolled, the vectors moving down: cold instructions cost more than moves
#pragma nounroll
      for (int u = 0; u < kDeep; ++u) {
        if (__ballot(col[0] < a.cols) == 0) break;
        float v[kEpv];
        Vec<BF16, kEpv>::widen(raw[0], v);
        if (col[0] < a.cols && col[0] + kEpv > a.cols)
          load_vec<BF16, kEpv>(c.base + beam[0] * a.ld_bytes, col[0], a.cols, v);
#pragma unroll
        for (int e = 0; e < kEpv; ++e) {
          const uint64_t key = c.key(static_cast<int>(beam[0]), col[0] + e, v[e]);
          if (col[0] + e < a.cols && static_cast<uint32_t>(key >> 32) >= least) {
            const int at = atomicAdd(&s.n, 1);
            if (at < kCap) s.cand[at] = key;
          }
        }
#pragma unroll
        for (int q = 0; q + 1 < kDeep; ++q)
          raw[q] = raw[q + 1], beam[q] = beam[q + 1], col[q] = col[q + 1];
      }
    }
    __syncthreads();
    const int n_cand = s.n;
    __syncthreads();
    if (n_cand <= kCap) {
      const LdsKeys some{s.cand};
      collect(some, TheKey{}, n_cand, n_cand <= kFew ? 1 : bound_of(some, n_cand, k, kFew - k, s),
              s.few, kFew, s);
    } else {  // many equal scores
      const ListedKeys<BF16> some{c};
      const int n_some = listed * static_cast<int>(c.group_cols());
      collect(some, TheKey{}, n_some, bound_of(some, n_some, k, kFew - k, s), s.few, kFew, s);
    }
  }
  const uint64_t key = best_of_few(s.n, k, s);
  if (tid < k) keys[seq * k + tid] = key;
}

struct PartKeys {  // one array per shard
  const uint64_t *part[64];
};
struct SeqParts {
  const PartKeys &parts;
  int64_t at;
  int k;
  __device__ __forceinline__ uint64_t operator()(int i) const {
    const int part = static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(k));
    return parts.part[part][at + i - part * k];
  }
};

// One workgroup per sequence: 2.5 us for one, 4.1 us for 32, latency.
__global__ __launch_bounds__(kThreads) void beam_merge_rows(PartKeys parts, int n_parts, int k,
                                                           int64_t vocab,
                                                           float *__restrict__ score,
                                                           int64_t *__restrict__ parent,
                                                           int64_t *__restrict__ token) {
  __shared__ SelectLds s;
  const int64_t seq = blockIdx.x;
  const int tid = threadIdx.x, n = n_parts * k;
  const SeqParts all{parts, seq * k, k};
  collect(all, TheKey{}, n, n <= kFew ? 1 : bound_of(all, n, k, kFew - k, s), s.few, kFew, s);
  const uint64_t key = best_of_few(s.n, k, s);
  if (tid >= k) return;
  const int64_t i = seq * k + tid;
  const uint64_t place = 0xFFFFFFFFull - (key & 0xFFFFFFFFull);
  const uint64_t b = place / static_cast<uint64_t>(vocab);
  score[i] = key == 0 ? -__builtin_huge_valf() : score_of(static_cast<uint32_t>(key >> 32));
  parent[i] = key == 0 ? -1 : static_cast<int64_t>(b);
  token[i] = key == 0 ? -1 : static_cast<int64_t>(place - b * static_cast<uint64_t>(vocab));
}

// ---------------------------------------------------------------------------
// reordering of states
// ---------------------------------------------------------------------------
// 2^log2g lanes serve a unit: `span` vectors (of V) of one destination row,
// rows row0 .. row0 + n_rows - 1 in units_per_row units each.  A copy: 28 x 256
// rows of 4 KB (29 MB, read from the caches for the most part) in 8.4 us.
template <typename V>
__global__ __launch_bounds__(kBlock) void reorder_rows(const V *__restrict__ src, int64_t row0,
                                                      uint32_t n_rows, int64_t rows_per_outer,
                                                      int beams_in, int beams_out, int64_t n_seqs,
                                                      int64_t vr, uint32_t units_per_row,
                                                      int64_t span, int log2g,
                                                      const int64_t *__restrict__ parent,
                                                      int64_t ld_parent, V *__restrict__ dst) {
  const uint32_t t = blockIdx.x * kBlock + threadIdx.x;
  const uint32_t unit = t >> log2g, rel = unit / units_per_row;
  if (rel >= n_rows) return;
  const int group = 1 << log2g;
  const int64_t begin = (unit - rel * units_per_row) * span;
  const int64_t v1 = begin + span < vr ? begin + span : vr;
  const int64_t row = row0 + rel;
  // 64-bit divisions cost more than the rest of a short row's work
  int64_t o, s;
  int b;
  if (row < 0x7fffffff && rows_per_outer < 0x7fffffff) {
    const uint32_t r = static_cast<uint32_t>(row), per = static_cast<uint32_t>(rows_per_outer);
    const uint32_t q = r / per, in = r - q * per, sq = in / static_cast<uint32_t>(beams_out);
    o = q, s = sq, b = static_cast<int>(in - sq * beams_out);
  } else {
    o = row / rows_per_outer;
    const int64_t in = row - o * rows_per_outer;
    s = in / beams_out;
    b = static_cast<int>(in - s * beams_out);
  }
  const int64_t from = parent[s * ld_parent + b];
  const bool valid = static_cast<uint64_t>(from) < static_cast<uint64_t>(beams_in);
  const V *from_row = src + ((o * n_seqs + s) * beams_in + (valid ? from : 0)) * vr;
  V *to_row = dst + row * vr;
  constexpr int kDeep = 4;
  for (int64_t v = begin + (t & (group - 1)); v < v1; v += kDeep * group) {
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
    const dim3 grid(static_cast<unsigned>((threads + kBlock - 1) / kBlock));
    hipLaunchKernelGGL((reorder_rows<V>), grid, dim3(kBlock), 0, st, static_cast<const V *>(src), r,
                       static_cast<uint32_t>(nr), n_seqs * beams_out, beams_in, beams_out, n_seqs,
                       vr, static_cast<uint32_t>(units), span, log2g, parent, ld_parent,
                       static_cast<V *>(dst));
  }
  return static_cast<int>(hipGetLastError());
}

// Vectors per group, as a power of two: 8 where all of a sequence's groups
// still fit LDS.  Groups of 64 are too few there: 30 picks of 15 x 1619 logits
// need half of the 60 groups, in which 2000 scores reach the bound (28 us).
int group_log2(int beams, int64_t cols, int dtype) {
  const int64_t small = 8 * (dtype == 1 ? Row<true>::kEpv : Row<false>::kEpv);
  return beams * ((cols + small - 1) / small) <= kHeld ? 3 : 6;
}

}  // namespace

int64_t beam_groups_per_row(int beams, int64_t cols, int dtype) {
  const int64_t group = int64_t(dtype == 1 ? Row<true>::kEpv : Row<false>::kEpv)
                        << group_log2(beams, cols, dtype);
  return (cols + group - 1) / group;
}

int launch_beam_select(const void *base, int64_t ld, int dtype, int64_t n_seqs, int beams,
                       int64_t cols, int64_t vocab_start, int64_t vocab, const float *lse,
                       const float *scores, int picks, uint64_t *keys, float *group_best,
                       void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // clear a stale error so the status returned is this launch's
  const int64_t groups = beam_groups_per_row(beams, cols, dtype);
  const BeamArgs a{static_cast<const char *>(base), ld * (dtype == 1 ? 2 : 4), cols, vocab_start,
                   vocab, lse, scores, beams, picks, groups, group_log2(beams, cols, dtype)};
  const bool direct = beams * cols <= kDirect;
  if (!direct) {
    const int64_t per_block = kVecsAhead * kBlock * (dtype == 1 ? Row<true>::kEpv : Row<false>::kEpv);
    const unsigned gx = static_cast<unsigned>((cols + per_block - 1) / per_block);
    const int64_t rows = n_seqs * beams;
    for (int64_t r = 0; r < rows; r += kRowsPerGrid) {
      const dim3 grid(gx, static_cast<unsigned>(std::min(kRowsPerGrid, rows - r)));
      if (dtype == 1)
        hipLaunchKernelGGL((beam_groups<true>), grid, dim3(kBlock), 0, st, a, r, group_best);
      else
        hipLaunchKernelGGL((beam_groups<false>), grid, dim3(kBlock), 0, st, a, r, group_best);
    }
  }
  const float *best = direct ? nullptr : group_best;
  const dim3 seqs(static_cast<unsigned>(n_seqs));
  if (dtype == 1)
    hipLaunchKernelGGL((beam_pick<true>), seqs, dim3(kThreads), 0, st, a, best, keys);
  else
    hipLaunchKernelGGL((beam_pick<false>), seqs, dim3(kThreads), 0, st, a, best, keys);
  return static_cast<int>(hipGetLastError());
}

int launch_beam_merge(const uint64_t *const *keys, int n_parts, int64_t n_seqs, int picks,
                      int64_t vocab, float *score, int64_t *parent, int64_t *token, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  PartKeys parts{};
  for (int r = 0; r < n_parts; ++r) parts.part[r] = keys[r];
  hipLaunchKernelGGL(beam_merge_rows, dim3(static_cast<unsigned>(n_seqs)), dim3(kThreads), 0, st,
                     parts, n_parts, picks, vocab, score, parent, token);
  return static_cast<int>(hipGetLastError());
}

int launch_beam_reorder(const void *src, int64_t outer, int64_t n_seqs, int beams_in,
                        int64_t row_bytes, const int64_t *parent, int64_t ld_parent,
                        int beams_out, void *dst, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  const uint64_t low = reinterpret_cast<uint64_t>(src) | reinterpret_cast<uint64_t>(dst) |
                       static_cast<uint64_t>(row_bytes);
#define VPE_REORDER(V, B)                                                                  \
  launch_reorder<V>(src, outer, n_seqs, beams_in, row_bytes / B, parent, ld_parent, beams_out, \
                    dst, st)
  if ((low & 15) == 0) return VPE_REORDER(u32x4, 16);
  if ((low & 7) == 0) return VPE_REORDER(u32x2, 8);
  if ((low & 3) == 0) return VPE_REORDER(uint32_t, 4);
  if ((low & 1) == 0) return VPE_REORDER(uint16_t, 2);
  return VPE_REORDER(uint8_t, 1);
#undef VPE_REORDER
}

}  // namespace vpe
