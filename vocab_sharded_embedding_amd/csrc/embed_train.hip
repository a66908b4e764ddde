// The scaled lookup and its gradient for gfx950.
//
// Scaled lookup: out[i] = rnd(scale * W[ids[i] - start]), zero rows for ids
// outside the shard: the gather of gather.hip with one fp32 product and one
// rounding per element on the way, bound by HBM like it.
//
// Gradient: dW[j] = scale * sum over the positions i of token j of dY[i].  The
// positions are sorted by token first (a stable radix sort), so that every sum
// has one owner, a fixed order and no atomics; then one wave sums each run of
// equal tokens, reading every owned row of dY once and writing every row of dW
// once.
//  - Sort: digits of up to 9 bits, so a vocabulary shard (2^11 to 2^18 rows)
//    takes two passes.  Up to kGradOneBlockIds ids are sorted by one workgroup
//    in LDS in a single launch; more ids take two launches per pass (digit
//    counts per workgroup, then ranks and scatter).  Ids outside the shard
//    are dropped in the first pass.
//  - Sum: the sorted positions are cut into chunks of up to 32, one wave each
//    (and per block of columns), so that a token with thousands of positions
//    (natural text) is spread over the chip; the parts of a run that crosses
//    chunks leave fp32 partial sums, which a second kernel joins in order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "vpe_device.h"
#include "vpe_train_launch.h"

namespace vpe {
namespace {

using namespace dev;

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / 64;

// ---------------------------------------------------------------------------
// scaled lookup
// ---------------------------------------------------------------------------
// Local row of an id, or -1: one unsigned compare covers both ends of the shard
// (a wrapped difference is >= rows).
template <typename IdT>
__device__ __forceinline__ int64_t local_row(IdT id, uint64_t start, uint64_t rows) {
  const uint64_t local = static_cast<uint64_t>(static_cast<int64_t>(id)) - start;
  return local < rows ? static_cast<int64_t>(local) : -1;
}

// One row by `group` lanes, VPL vectors per lane loaded before any is stored.
template <bool BF16, int VPL>
__device__ __forceinline__ void scale_row(const char *src, char *dst, int64_t dim, float scale,
                                          int lane, int group) {
  constexpr int kEpv = BF16 ? 8 : 4;
  typedef Vec<BF16, kEpv> V;
  const typename V::loose *src_v = reinterpret_cast<const typename V::loose *>(src);
  typename V::loose *dst_v = reinterpret_cast<typename V::loose *>(dst);
  const int64_t whole = dim / kEpv;
  for (int64_t c0 = lane; c0 < whole; c0 += VPL * group) {
    typename V::raw r[VPL];
#pragma unroll
    for (int c = 0; c < VPL; ++c) {
      r[c] = typename V::raw(0);
      if (src != nullptr && c0 + c * group < whole) r[c] = src_v[c0 + c * group];
    }
#pragma unroll
    for (int c = 0; c < VPL; ++c) {
      float v[kEpv];
      V::widen(r[c], v);
#pragma unroll
      for (int e = 0; e < kEpv; ++e) v[e] *= scale;
      typename V::raw o = V::narrow(v);
      if (src == nullptr) o = typename V::raw(0);  // +0, also for a negative factor
      if (c0 + c * group < whole) __builtin_nontemporal_store(o, dst_v + c0 + c * group);
    }
  }
  for (int64_t i = whole * kEpv + lane; i < dim; i += group)
    store_one<BF16>(dst, i, src != nullptr ? load_one<BF16>(src, i) * scale : 0.f);
}

// 2^log2g lanes (at most 64) serve one row.  131072 rows of 8 KB, a quarter of
// them owned: 220 us, 5.7 TB/s; 8 rows in turn per wave, for longer spans of
// stores, took 246 us (less in flight).
template <bool BF16, int VPL, typename IdT>
__global__ __launch_bounds__(kBlock) void scaled_rows(const IdT *__restrict__ ids, int64_t n,
                                                     const char *__restrict__ weight,
                                                     uint64_t start, uint64_t rows, int64_t dim,
                                                     float scale, int log2g,
                                                     char *__restrict__ out) {
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  const int64_t row = t >> log2g;
  if (row >= n) return;
  const int group = 1 << log2g;
  const int64_t row_bytes = dim * (BF16 ? 2 : 4);
  const int64_t local = local_row(ids[row], start, rows);
  scale_row<BF16, VPL>(local >= 0 ? weight + local * row_bytes : nullptr, out + row * row_bytes,
                       dim, scale, static_cast<int>(t) & (group - 1), group);
}

int ceil_log2(int64_t v) {
  int l = 0;
  while ((int64_t(1) << l) < v) ++l;
  return l;
}

// Rows per launch: keeps every grid inside the 32-bit work-item range.
constexpr int64_t kRowsPerLaunch = int64_t(1) << 24;

template <bool BF16, typename IdT>
int scaled_any(const IdT *ids, int64_t n, const void *weight, int64_t rows, int64_t dim,
               int64_t start, float scale, void *out, hipStream_t st) {
  const int64_t vr = (dim + (BF16 ? 7 : 3)) / (BF16 ? 8 : 4);  // vectors per row
  const int log2g = std::min(6, ceil_log2(vr));
  for (int64_t r0 = 0; r0 < n; r0 += kRowsPerLaunch) {
    const int64_t nr = std::min(n - r0, kRowsPerLaunch);
    const unsigned blocks = static_cast<unsigned>(((nr << log2g) + kBlock - 1) / kBlock);
    char *o = static_cast<char *>(out) + r0 * dim * (BF16 ? 2 : 4);
#define VPE_SCALED(VPL)                                                                     \
  hipLaunchKernelGGL((scaled_rows<BF16, VPL, IdT>), dim3(blocks), dim3(kBlock), 0, st,      \
                     ids + r0, nr, static_cast<const char *>(weight),                       \
                     static_cast<uint64_t>(start), static_cast<uint64_t>(rows), dim, scale, \
                     log2g, o)
    if (vr <= 64) VPE_SCALED(1);
    else if (vr <= 128) VPE_SCALED(2);
    else if (vr <= 256) VPE_SCALED(4);
    else VPE_SCALED(8);
#undef VPE_SCALED
  }
  return static_cast<int>(hipGetLastError());
}

// ---------------------------------------------------------------------------
// stable sort of the owned positions by token
// ---------------------------------------------------------------------------
constexpr int kDigitBits = 9;
constexpr int kDigits = static_cast<int>(kSortDigits);
static_assert(kDigits == 1 << kDigitBits, "digit values");

// Lanes of the wave whose digit equals this lane's, among lanes with `valid`.
// All kDigitBits bits, unrolled: a rolled loop pays more for its branch than
// for a bit.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, bool valid) {
  const uint64_t mask = __ballot(valid);
  uint32_t lo = static_cast<uint32_t>(mask), hi = static_cast<uint32_t>(mask >> 32);
#pragma unroll
  for (int b = 0; b < kDigitBits; ++b) {
    const uint32_t bit = (digit >> b) & 1u, set = 0u - bit;
    const uint64_t one = __ballot(bit != 0);
    lo &= ~(static_cast<uint32_t>(one) ^ set);
    hi &= ~(static_cast<uint32_t>(one >> 32) ^ set);
  }
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

__device__ __forceinline__ int below(uint64_t mask) {  // set lanes below this one
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t up = __shfl_up(v, d);
    if (lane >= d) v += up;
  }
  return v;
}

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

// Workgroups of zeros that ride along with the sort, which leaves most of the
// chip idle: rows [row0, row1) of the gradient, `blocks` workgroups after the
// sort's own.  flags == nullptr: all of them; else those without an id.
struct ZeroRows {
  char *dw;
  int64_t row_bytes;
  int64_t row0, row1;
  const uint8_t *flags;
  unsigned blocks;
  int log2g;  // lanes that clear a row with flags
};

// `block` of z.blocks workgroups of `threads` threads, all of their rows.  Plain
// stores where the whole shard is cleared beside one sorting workgroup (8192 ids,
// 156 MB: 30 us against 39 with non-temporal ones), non-temporal ones (NT) where
// many sorted rows are read meanwhile and after, which plain ones push out of the
// caches (65536 ids, 622 MB: 166 us against 186).
template <bool NT>
__device__ __forceinline__ void zero_all_rows(const ZeroRows &z, unsigned block, int threads) {
  const int64_t share = (z.row1 - z.row0 + z.blocks - 1) / z.blocks;
  const int64_t r0 = z.row0 + block * share, r1 = r0 + share < z.row1 ? r0 + share : z.row1;
  if (r0 < r1)
    zero_bytes<NT>(z.dw + r0 * z.row_bytes, (r1 - r0) * z.row_bytes, threadIdx.x, threads);
}

// The same beside the passes, and of rows with flags those without an id.
__device__ __forceinline__ void zero_rows(const ZeroRows &z, unsigned block, int threads) {
  if (z.flags == nullptr) return zero_all_rows<true>(z, block, threads);
  const int64_t share = (z.row1 - z.row0 + z.blocks - 1) / z.blocks;
  const int64_t r0 = z.row0 + block * share, r1 = r0 + share < z.row1 ? r0 + share : z.row1;
  if (r0 >= r1) return;
  // a contiguous part per wave
  const int lane = threadIdx.x & 63, waves = threads / 64;
  const int64_t part = (r1 - r0 + waves - 1) / waves, w0 = r0 + wave_in_block() * part;
  const int64_t w1 = w0 + part < r1 ? w0 + part : r1;
  if (z.log2g < 6) {
    // several rows at a time, 2^log2g lanes each
    constexpr int kDeep = 4;
    const int in = lane & ((1 << z.log2g) - 1), step = 64 >> z.log2g;
    for (int64_t r = w0 + (lane >> z.log2g); r < w1; r += kDeep * step) {
      uint8_t has_id[kDeep];
#pragma unroll
      for (int u = 0; u < kDeep; ++u) has_id[u] = r + u * step < w1 ? z.flags[r + u * step] : 1;
#pragma unroll
      for (int u = 0; u < kDeep; ++u)
        if (has_id[u] == 0)
          zero_bytes<true>(z.dw + (r + u * step) * z.row_bytes, z.row_bytes, in, 1 << z.log2g);
    }
    return;
  }
  for (int64_t r = w0; r < w1; r += 64) {
    uint64_t empty = __ballot(r + lane < w1 && z.flags[r + lane < w1 ? r + lane : w0] == 0);
    while (empty) {
      const int64_t row = r + __builtin_ctzll(empty);
      empty &= empty - 1;
      zero_bytes<true>(z.dw + row * z.row_bytes, z.row_bytes, lane, 64);
    }
  }
}

// Every owned id of at most kGradOneBlockIds, sorted in LDS by workgroup 0.
// Wave w takes the w-th run of items in every pass; an item's place is behind
// the smaller digits, behind its digit's items of the waves and rounds before
// and of the lanes before, so the sort is stable.  Bound by the latency of its
// rounds, one after the other: 257 ids in two passes 5.2 us; 8192 ids end within
// the 21 us in which the workgroups beside them clear 156 MB.
template <typename IdT>
__global__ __launch_bounds__(kSortThreads) void sort_one_block(
    const IdT *__restrict__ ids, int n, uint64_t start, uint64_t rows, int bits, int passes,
    uint32_t *__restrict__ key_out, uint32_t *__restrict__ pos_out,
    uint32_t *__restrict__ count_out, ZeroRows zero) {
  constexpr uint32_t kNone = 0xffffffffu;  // an id of another shard (rows < 2^31)
  __shared__ uint32_t skey[2][kGradOneBlockIds];
  __shared__ uint16_t spos[2][kGradOneBlockIds];
  __shared__ uint32_t at_[kSortWaves][kDigits];
  __shared__ uint32_t sums[kDigits / 64];
  if (blockIdx.x > 0) return zero_all_rows<false>(zero, blockIdx.x - 1, kSortThreads);
  // a wave reads and updates its own counters in program order
  volatile uint32_t(*at)[kDigits] = at_;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_in_block();
#pragma unroll 4
  for (int i = tid; i < n; i += kSortThreads) {
    const uint64_t local = static_cast<uint64_t>(static_cast<int64_t>(ids[i])) - start;
    skey[0][i] = local < rows ? static_cast<uint32_t>(local) : kNone;
    spos[0][i] = static_cast<uint16_t>(i);
  }
  const uint32_t low = (1u << bits) - 1;
  int m = n;
  for (int pass = 0; pass < passes; ++pass) {
    const uint32_t *from = skey[pass & 1];
    const uint16_t *from_pos = spos[pass & 1];
    uint32_t *to_key = skey[1 - (pass & 1)];
    uint16_t *to_pos = spos[1 - (pass & 1)];
    const int shift = pass * bits;
    const int share = (m + kSortThreads - 1) / kSortThreads * 64;
    const int i0 = wave * share, i1 = i0 + share < m ? i0 + share : m;
#pragma unroll
    for (int d = 0; d < kSortWaves * kDigits; d += kSortThreads)
      reinterpret_cast<uint32_t *>(at_)[d + tid] = 0;
    __syncthreads();
    for (int i = i0 + lane; i < i1; i += 64)
      if (from[i] != kNone) atomicAdd(&at_[wave][(from[i] >> shift) & low], 1u);
    __syncthreads();
    // exclusive sums over (digit, wave)
    uint32_t c[kSortWaves], total = 0, incl = 0;
    if (tid < kDigits) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) c[w] = at_[w][tid], total += c[w];
      incl = wave_scan(total);
      if (lane == 63) sums[wave] = incl;
    }
    __syncthreads();
    uint32_t all = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kDigits / 64; ++w) {
      before += w < wave ? sums[w] : 0;
      all += sums[w];
    }
    if (tid < kDigits) {
      uint32_t to = before + incl - total;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) at_[w][tid] = to, to += c[w];
    }
    __syncthreads();
    for (int r = i0; r < i1; r += 64) {
      const int i = r + lane;
      const uint32_t key = i < i1 ? from[i] : kNone;
      const uint32_t d = (key >> shift) & low;
      const uint64_t same = same_digit(d, key != kNone);
      if (key != kNone) {
        const uint32_t seen = at[wave][d];
        const int ahead = below(same);
        if (ahead == 0) at[wave][d] = seen + __popcll(same);
        to_key[seen + ahead] = key;
        to_pos[seen + ahead] = from_pos[i];
      }
    }
    m = static_cast<int>(all);
    __syncthreads();
  }
  for (int i = tid; i < m; i += kSortThreads) {
    key_out[i] = skey[passes & 1][i];
    pos_out[i] = spos[passes & 1][i];
  }
  if (tid == 0) *count_out = static_cast<uint32_t>(m);
}

// One pass over more ids: item i of the pass is ids[i] (FIRST) or
// key_in[i] / pos_in[i].  Workgroup b takes items [b * tile, (b + 1) * tile).
template <bool FIRST, typename IdT>
struct SortItems {
  const IdT *ids;
  const uint32_t *key_in, *pos_in;
  uint64_t start, rows;
  uint8_t *flags;  // FIRST: of the rows, or nullptr
  __device__ __forceinline__ bool get(int64_t i, uint32_t &key) const {
    if constexpr (FIRST) {
      const uint64_t local = static_cast<uint64_t>(static_cast<int64_t>(ids[i])) - start;
      key = static_cast<uint32_t>(local);
      return local < rows;
    } else {
      key = key_in[i];
      return true;
    }
  }
};
struct SortPass {
  int64_t n;       // ids
  int64_t tile;    // items per workgroup, a multiple of kSortThreads
  unsigned blocks;
  int shift, bits;
};

// hist[b][d] = items of digit d in workgroup b's tile.  The first pass also
// clears the rows' flags.  Latency again: 65536 ids of 18 bits, counts 6.4 and
// scatter 8.7 us in the first pass; the second pass's 28 us each are the time of
// the 142 MB that the workgroups beside them clear (5.1 TB/s).
template <bool FIRST, typename IdT>
__global__ __launch_bounds__(kSortThreads) void sort_counts(SortItems<FIRST, IdT> items,
                                                           SortPass pass, const uint32_t *count,
                                                           uint32_t *hist, ZeroRows zero) {
  __shared__ uint32_t h[kDigits];
  if (blockIdx.x >= pass.blocks) return zero_rows(zero, blockIdx.x - pass.blocks, kSortThreads);
  const int tid = threadIdx.x;
  if (FIRST && items.flags != nullptr) {
    u32x4 *f = reinterpret_cast<u32x4 *>(items.flags);
    const int64_t nf = static_cast<int64_t>((items.rows + 15) / 16);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kSortThreads + tid; i < nf;
         i += static_cast<int64_t>(pass.blocks) * kSortThreads)
      f[i] = u32x4(0);
  }
  if (tid < kDigits) h[tid] = 0;
  __syncthreads();
  const int64_t m = FIRST ? pass.n : static_cast<int64_t>(*count);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * pass.tile;
  const int64_t i1 = i0 + pass.tile < pass.n ? i0 + pass.tile : pass.n;
  const uint32_t low = (1u << pass.bits) - 1;
  // keys past m are read and dropped: they lie inside the buffer, and waiting
  // for m first costs a latency
#pragma unroll 2
  for (int64_t i = i0 + tid; i < i1; i += kSortThreads) {
    uint32_t key;
    if (items.get(i, key) && i < m) atomicAdd(&h[(key >> pass.shift) & low], 1u);
  }
  __syncthreads();
  if (tid < kDigits) hist[static_cast<int64_t>(blockIdx.x) * kDigits + tid] = h[tid];
}

// Every item to its place: behind the smaller digits, behind its digit's items
// in the workgroups, waves and rounds before, behind the lanes before.
template <bool FIRST, typename IdT>
__global__ __launch_bounds__(kSortThreads) void sort_scatter(
    SortItems<FIRST, IdT> items, SortPass pass, uint32_t *count, const uint32_t *__restrict__ hist,
    uint32_t *__restrict__ key_out, uint32_t *__restrict__ pos_out, ZeroRows zero) {
  constexpr int kParts = kSortThreads / (kDigits / 2);  // threads that share a pair of digits
  __shared__ uint32_t at_[kSortWaves][kDigits];
  __shared__ u32x2 part_before[kParts][kDigits / 2], part_total[kParts][kDigits / 2];
  __shared__ uint32_t base[kDigits];
  __shared__ uint32_t sums[kDigits / 128];
  if (blockIdx.x >= pass.blocks) return zero_rows(zero, blockIdx.x - pass.blocks, kSortThreads);
  // a wave reads and updates its own counters in program order
  volatile uint32_t(*at)[kDigits] = at_;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_in_block();
  const int64_t m = FIRST ? pass.n : static_cast<int64_t>(*count);
  const uint32_t low = (1u << pass.bits) - 1;

  // A wave's items, kAhead rounds of 64 at a time: the first are on their way
  // while the workgroups' counts are summed, and stay in registers where they
  // are all there is (a tile of kSortTile).
  constexpr int kAhead = static_cast<int>(kSortTile) / kSortThreads;
  const int64_t per_wave = pass.tile / kSortWaves;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * pass.tile + wave * per_wave;
  const int64_t i1 = i0 + per_wave < pass.n ? i0 + per_wave : pass.n;
  uint32_t key[kAhead], from[kAhead];
  bool have[kAhead];
  auto take = [&](int64_t r) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t i = r + u * 64 + lane;
      key[u] = 0, from[u] = static_cast<uint32_t>(i);
      have[u] = i < i1 && items.get(i, key[u]);
      if (!FIRST && i < i1) from[u] = items.pos_in[i];
      have[u] = have[u] && i < m;
    }
  };
  take(i0);

  // the workgroups' counts: pair of digits `pair`, every kParts-th workgroup
  const int pair = tid % (kDigits / 2), part = tid / (kDigits / 2);
  u32x2 before = u32x2(0), total = u32x2(0);
  const u32x2 *h2 = reinterpret_cast<const u32x2 *>(hist);
#pragma unroll 8
  for (unsigned b = part; b < pass.blocks; b += kParts) {
    const u32x2 c = h2[b * (kDigits / 2) + pair];
    if (b < blockIdx.x) before += c;
    total += c;
  }
  // counts of every wave's part of the tile
  for (int d = tid; d < kSortWaves * kDigits; d += kSortThreads)
    reinterpret_cast<uint32_t *>(at_)[d] = 0;
  __syncthreads();
  const bool again = per_wave > kAhead * 64;  // items do not stay in registers
  for (int64_t r = i0; r < i1; r += kAhead * 64) {
    if (r != i0) take(r);
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (have[u]) atomicAdd(&at_[wave][(key[u] >> pass.shift) & low], 1u);
  }
  part_before[part][pair] = before;
  part_total[part][pair] = total;
  __syncthreads();
  uint32_t incl = 0;
  if (part == 0) {
#pragma unroll
    for (int q = 1; q < kParts; ++q) before += part_before[q][pair], total += part_total[q][pair];
    incl = wave_scan(total[0] + total[1]);
    if (lane == 63) sums[wave] = incl;
  }
  __syncthreads();
  if (part == 0) {
    uint32_t first = incl - total[0] - total[1];
#pragma unroll
    for (int w = 0; w < kDigits / 128; ++w) first += w < wave ? sums[w] : 0;
    base[2 * pair] = first + before[0];
    base[2 * pair + 1] = first + total[0] + before[1];
    if (FIRST && blockIdx.x == 0 && pair == kDigits / 2 - 1) *count = first + total[0] + total[1];
  }
  __syncthreads();
  if (tid < kDigits) {
    uint32_t c[kSortWaves], to = base[tid];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) c[w] = at_[w][tid];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) at_[w][tid] = to, to += c[w];
  }
  __syncthreads();
  for (int64_t r = i0; r < i1; r += kAhead * 64) {
    if (again) take(r);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t d = (key[u] >> pass.shift) & low;
      const uint64_t same = same_digit(d, have[u]);
      if (have[u]) {
        const uint32_t seen = at[wave][d];
        const uint32_t to = seen + below(same);
        if (below(same) == 0) at[wave][d] = seen + __popcll(same);
        key_out[to] = key[u];
        pos_out[to] = from[u];
        if (FIRST && items.flags != nullptr) items.flags[key[u]] = 1;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// sums of the sorted rows
// ---------------------------------------------------------------------------
struct GradArgs {
  const uint32_t *key, *pos, *count;
  const char *dy;
  int64_t dim;
  float scale;
  char *dw;
  bool accumulate;
  float *partial;      // [2 * chunks][partial_ld]
  int64_t partial_ld;
  int chunk;           // sorted positions per wave, a power of two up to 32
  int col_blocks;      // waves per chunk
};

template <bool OUT16, int EPV>
__device__ __forceinline__ void write_row(const GradArgs &a, uint32_t row, int64_t col,
                                          const float (&sum)[EPV]) {
  char *dw = a.dw + static_cast<int64_t>(row) * a.dim * (OUT16 ? 2 : 4);
  float v[EPV];
  if (a.accumulate) {
    load_vec<OUT16, EPV>(dw, col, a.dim, v);
#pragma unroll
    for (int e = 0; e < EPV; ++e) v[e] = v[e] + a.scale * sum[e];
  } else {
#pragma unroll
    for (int e = 0; e < EPV; ++e) v[e] = a.scale * sum[e];
  }
  store_vec_nt<OUT16, EPV>(dw, col, a.dim, v);
}

// One wave per chunk of sorted positions and block of 64 vectors of columns: it
// walks the chunk's rows, kDeep of them in flight, and leaves each run of equal
// tokens when it ends.  A run that began before the chunk or goes on behind it
// leaves a partial sum: slot 2c if it holds the chunk's first position, slot
// 2c + 1 if it begins inside.  Workgroups after them write zero rows.  Bound by
// HBM: 65536 Zipf ids x 1024 bf16 with an fp32 gradient read 136 MB and write 239
// MB, most of it zero rows, in 64 us, 5.9 TB/s.
template <bool IN16, bool OUT16, int EPV>
__global__ __launch_bounds__(kBlock) void grad_chunks(GradArgs a, int64_t chunk0, int64_t n_chunks,
                                                     unsigned chunk_blocks, ZeroRows zero) {
  if (blockIdx.x >= chunk_blocks) return zero_rows(zero, blockIdx.x - chunk_blocks, kBlock);
  typedef Vec<IN16, EPV> V;
  constexpr int kDeep = 8;
  const int lane = threadIdx.x & 63;
  const uint32_t wave = blockIdx.x * kWaves + wave_in_block();
  const uint32_t rel = wave / static_cast<uint32_t>(a.col_blocks);
  if (rel >= n_chunks) return;
  const int64_t c = chunk0 + rel;
  const int64_t n = *a.count, p0 = c * a.chunk;
  if (p0 >= n) return;
  const int len = n - p0 < a.chunk ? static_cast<int>(n - p0) : a.chunk;
  // lane l < len: position p0 + l; lane len: the position behind the chunk
  const uint32_t key = p0 + lane < n ? a.key[p0 + lane] : 0;
  const uint32_t before = p0 > 0 ? a.key[p0 - 1] : 0;
  const uint32_t pos = lane < len ? a.pos[p0 + lane] : 0;
  // ends: bit l is set where the run of position l ends with it
  const uint32_t next = __shfl_down(key, 1);
  const uint64_t ends = __ballot(lane < len && (p0 + lane + 1 >= n || next != key));
  const bool begun = p0 > 0 && before == static_cast<uint32_t>(
                                             __builtin_amdgcn_readfirstlane(static_cast<int>(key)));

  const int64_t col = (static_cast<int64_t>(wave - rel * a.col_blocks) * 64 + lane) * EPV;
  const bool whole = col + EPV <= a.dim;
  const bool ragged = __ballot(!whole && col < a.dim) != 0;  // a row's end inside a vector
  const int64_t in_bytes = a.dim * V::kSize;
  float sum[EPV];
#pragma unroll
  for (int e = 0; e < EPV; ++e) sum[e] = 0.f;
  bool inside = !begun;  // the run began in this chunk, at its first position or later
  int first = 0;         // the run's first position in the chunk
  for (int i0 = 0; i0 < len; i0 += kDeep) {
    typename V::raw r[kDeep];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int64_t s = static_cast<uint32_t>(
          __builtin_amdgcn_readlane(static_cast<int>(pos), i0 + u < len ? i0 + u : i0));
      r[u] = typename V::raw(0);
      if (whole && i0 + u < len)
        r[u] = *reinterpret_cast<const typename V::loose *>(a.dy + s * in_bytes + col * V::kSize);
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int i = i0 + u;
      if (i >= len) break;
      float v[EPV];
      V::widen(r[u], v);
      if (ragged) {
        const int64_t s = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(pos), i));
        if (!whole) load_vec<IN16, EPV>(a.dy + s * in_bytes, col, a.dim, v);
      }
#pragma unroll
      for (int e = 0; e < EPV; ++e) sum[e] += v[e];
      const bool end = (ends >> i) & 1;
      if (end || i == len - 1) {
        if (col < a.dim) {
          if (inside && end) {
            const uint32_t token =
                static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(key), i));
            write_row<OUT16, EPV>(a, token, col, sum);
          } else {
            f32x4 *o = reinterpret_cast<f32x4 *>(a.partial + (2 * c + (first > 0)) * a.partial_ld +
                                                 col);
#pragma unroll
            for (int e = 0; e < EPV; e += 4)
              o[e / 4] = f32x4{sum[e], sum[e + 1], sum[e + 2], sum[e + 3]};
          }
        }
#pragma unroll
        for (int e = 0; e < EPV; ++e) sum[e] = 0.f;
        inside = true;
        first = i + 1;
      }
    }
  }
}

// One wave per chunk and block of 256 columns: the run that leaves the chunk
// having begun in it is joined from its partial sums, in order: 16 in fp32, and
// those sums in 64 bits, as a run has up to 2^26 pieces (added one by one in fp32,
// pieces of one sign lost 1.6e-4 of the sum of 2^21 positions; each of them in 64
// bits took 160 instead of 109 us for 131072 Zipf ids over 8192 rows x 1024, this
// takes 110).  Long runs are
// joined by the workgroup's waves together, a quarter each.  Workgroups after
// them write zero rows.  Bound by latency: 4 us where no run is long; 65536 Zipf
// ids (exponent 1.1), 272 pieces in the longest run, 19.2 us with 64 MB of zero
// rows beside it.  (The whole gradient of those took 162.4, 167 and 177 us with a
// workgroup of 4, 8 and 16 waves per chunk, 159.7 us this way: most chunks have
// nothing to join.  Rows of 64 columns, 131072 Zipf ids: 60 us then, 63 now.)
template <bool OUT16>
__global__ __launch_bounds__(kBlock) void grad_join(GradArgs a, int64_t chunk0, int64_t n_chunks,
                                                   int col_blocks, unsigned join_blocks,
                                                   ZeroRows zero) {
  constexpr int kDeep = 16;  // partial sums in flight
  __shared__ f64x4 part[kWaves][64];
  __shared__ int64_t long_more[kWaves], long_slot0[kWaves];
  __shared__ uint32_t long_token[kWaves];
  if (blockIdx.x >= join_blocks) return zero_rows(zero, blockIdx.x - join_blocks, kBlock);
  const int lane = threadIdx.x & 63, wave = wave_in_block();
  const unsigned group = blockIdx.x / static_cast<unsigned>(col_blocks);
  const int64_t col = (static_cast<int64_t>(blockIdx.x - group * col_blocks) * 64 + lane) * 4;
  const int64_t c0 = chunk0 + static_cast<int64_t>(group) * kWaves;  // the workgroup's chunks

  // the chunk of this wave: how many chunks after it begin with its last token
  const int64_t c = c0 + wave, next = (c + 1) * a.chunk;
  int64_t more = 0, slot0 = 0;  // slot0: where the run's piece in this chunk is
  uint32_t token = 0;
  if (c < chunk0 + n_chunks) {
    const int64_t n = *a.count;
    token = a.key[next];  // (a place of the buffer, whatever n is)
    const uint32_t last = a.key[next - 1], first = a.key[next - a.chunk];
    const uint32_t before = a.key[c > 0 ? next - a.chunk - 1 : 0];
    slot0 = 2 * c + (first != token);
    const bool begun = c > 0 && first == token && before == token;
    if (next < n && last == token && !begun) {
      // 64 at a time, and where those all do, by the last ones of the next 64
      // times 64
      auto begin_with_it = [&](int64_t chunk) {  // how many of the lanes' chunks do
        const int64_t q = chunk * a.chunk;
        const uint64_t on = __ballot(q < n && a.key[q < n ? q : 0] == token);
        return on == ~0ull ? 64 : __builtin_ctzll(~on);
      };
      more = 1;
      for (;;) {
        const int some = begin_with_it(c + 1 + more + lane);
        more += some;
        if (some < 64) break;
        int whole;
        do {
          whole = begin_with_it(c + 1 + more + 64 * lane + 63);
          more += 64 * whole;
        } while (whole == 64);
      }
    }
  }

  // pieces i0 .. i1 - 1 of the run of chunk `of`: 0 in that chunk, i in chunk of +
  // i, at its first position; partial rows are padded past dim
  auto pieces = [&](int64_t of, int64_t slot0, int64_t i0, int64_t i1) {
    f64x4 sum = f64x4(0.0);
    if (col < a.dim) {
      for (int64_t i = i0; i < i1; i += kDeep) {
        f32x4 r[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
          const int64_t slot = i + u == 0 ? slot0 : 2 * (of + i + u);
          r[u] = f32x4(0.f);
          if (i + u < i1)
            r[u] = *reinterpret_cast<const f32x4 *>(a.partial + slot * a.partial_ld + col);
        }
        f32x4 some = f32x4(0.f);
#pragma unroll
        for (int u = 0; u < kDeep; ++u)
          if (i + u < i1) some += r[u];
        sum += __builtin_convertvector(some, f64x4);
      }
    }
    return sum;
  };
  auto write = [&](uint32_t run, f64x4 sum) {
    const f32x4 r = __builtin_convertvector(sum, f32x4);
    const float v[4] = {r[0], r[1], r[2], r[3]};
    if (col < a.dim) write_row<OUT16, 4>(a, run, col, v);
  };

  const bool alone = more < kDeep;
  if (more > 0 && alone) write(token, pieces(c, slot0, 0, more + 1));
  if (lane == 0)
    long_more[wave] = alone ? 0 : more, long_slot0[wave] = slot0, long_token[wave] = token;
  __syncthreads();
#pragma nounroll
  for (int w = 0; w < kWaves; ++w) {
    const int64_t m = long_more[w];
    if (m == 0) continue;  // the same in all waves
    const int64_t share = (m + kWaves) / kWaves, i0 = wave * share;
    part[wave][lane] = pieces(c0 + w, long_slot0[w], i0, i0 + share <= m ? i0 + share : m + 1);
    __syncthreads();
    if (wave == 0) {
      f64x4 sum = part[0][lane];
#pragma unroll
      for (int q = 1; q < kWaves; ++q) sum += part[q][lane];
      write(long_token[w], sum);
    }
    __syncthreads();
  }
}

// Workgroups for `rows` rows of zeros: about `span` bytes each (a row's flag
// costs as much as 64).  Of 1024 threads beside the sort, us of the whole gradient
// with 64 KB / 256 KB / 1 MB each: 8192 ids over 75968 rows of bf16 30.5 / 30.2 /
// 38.3; 65536 Zipf ids over 151936 fp32 rows 161.2 / 159.4 / 166.5, uniform ones
// 166.0 / 165.0 / 171.6; 131072 Zipf ids over as many bf16 rows 149.9 / 153.8 /
// 161.4.  Of 256 threads beside the sums, with 64 / 256 KB: 65536 Zipf ids 159.6 /
// 161.4, uniform ones 165.1 / 167.6.
unsigned zero_blocks(int64_t rows, int64_t row_bytes, double span = 262144.0) {
  if (rows <= 0) return 0;
  const double bytes = static_cast<double>(rows) * std::max(64.0, static_cast<double>(row_bytes));
  return static_cast<unsigned>(std::max(1.0, std::min(bytes / span, 65536.0)));
}

template <bool IN16, bool OUT16>
int launch_sums(GradArgs a, int64_t n, ZeroRows zero, ZeroRows join_zero, hipStream_t st) {
  // 16-byte vectors on the wider side
  constexpr int kEpv = IN16 && OUT16 ? 8 : 4;
  const int64_t chunks = (n + a.chunk - 1) / a.chunk;
  const int64_t blocks = (a.dim + 64 * kEpv - 1) / (64 * kEpv);
  a.col_blocks = static_cast<int>(blocks);
  // chunks per launch: grids stay inside the 32-bit range
  const int64_t step = std::max<int64_t>(1, (int64_t(1) << 24) / blocks);
  for (int64_t c = 0; c < chunks; c += step) {
    const int64_t nc = std::min(step, chunks - c);
    const unsigned cb = static_cast<unsigned>((nc * blocks + kWaves - 1) / kWaves);
    hipLaunchKernelGGL((grad_chunks<IN16, OUT16, kEpv>), dim3(cb + zero.blocks), dim3(kBlock), 0,
                       st, a, c, nc, cb, zero);
    zero.blocks = 0;
  }
  if (chunks > 1) {
    const int64_t join_cols = (a.dim + 255) / 256;
    const int64_t join_step = std::max<int64_t>(1, (int64_t(1) << 22) / join_cols) * kWaves;
    for (int64_t c = 0; c < chunks - 1; c += join_step) {
      const int64_t nc = std::min(join_step, chunks - 1 - c);
      const unsigned jb = static_cast<unsigned>((nc + kWaves - 1) / kWaves * join_cols);
      hipLaunchKernelGGL((grad_join<OUT16>), dim3(jb + join_zero.blocks), dim3(kBlock), 0, st, a, c,
                         nc, static_cast<int>(join_cols), jb, join_zero);
      join_zero.blocks = 0;
    }
  }
  return static_cast<int>(hipGetLastError());
}

template <typename IdT>
int grad_any(const IdT *ids, int64_t n, GradArgs a, int64_t rows, int dtype, int gdtype,
             uint64_t start, char *ws, hipStream_t st) {
  const EmbedGradLayout l = embed_grad_layout(n, rows, a.dim);
  uint32_t *key[2] = {reinterpret_cast<uint32_t *>(ws + l.key[0]),
                      reinterpret_cast<uint32_t *>(ws + l.key[1])};
  uint32_t *pos[2] = {reinterpret_cast<uint32_t *>(ws + l.pos[0]),
                      reinterpret_cast<uint32_t *>(ws + l.pos[1])};
  uint32_t *count = reinterpret_cast<uint32_t *>(ws + l.count);
  uint32_t *hist = reinterpret_cast<uint32_t *>(ws + l.hist);
  const int key_bits = std::max(1, ceil_log2(rows));
  const int passes = (key_bits + 8) / 9;
  const int bits = (key_bits + passes - 1) / passes;
  const uint64_t urows = static_cast<uint64_t>(rows);
  const int64_t zero_to = a.accumulate ? 0 : rows;
  const int64_t row_bytes = a.dim * (gdtype == 1 ? 2 : 4);
  ZeroRows zero{a.dw, row_bytes, 0, 0, nullptr, 0, std::min(6, ceil_log2((row_bytes + 15) / 16))};
  ZeroRows join_zero = zero;
  int last = 0;
  if (n <= kGradOneBlockIds) {
    // few rows have an id: all are cleared while they are sorted, and those
    // written again
    zero.row1 = zero_to;
    zero.blocks = zero_blocks(zero.row1, zero.row_bytes);
    hipLaunchKernelGGL((sort_one_block<IdT>), dim3(1 + zero.blocks), dim3(kSortThreads), 0, st,
                       ids, static_cast<int>(n), start, urows, bits, passes, key[0], pos[0], count,
                       zero);
    zero.blocks = 0;
  } else {
    // at least kSortTile items per workgroup, at most kSortMaxBlocks workgroups
    const int64_t unit = kSortTile * kSortMaxBlocks;
    SortPass ps{n, kSortTile * ((n + unit - 1) / unit), 0, 0, bits};
    ps.blocks = static_cast<unsigned>((n + ps.tile - 1) / ps.tile);
    uint8_t *flags = a.accumulate ? nullptr : reinterpret_cast<uint8_t *>(ws + l.flags);
    // The flags are complete after the first pass: each later launch of the
    // sort clears an equal part of half the rows without an id.  The first two
    // clear what fits their time, about 24 MB, with or without one (65536 Zipf ids:
    // 159.6 us, 164.5 with none, 161.8 with 12 MB, 159.7 with 48; uniform ids 165.0,
    // 168.1, 167.2 and 166.8).
    auto ride = [&](int64_t ride_rows, const uint8_t *ride_flags) {
      zero.flags = ride_flags;
      zero.row0 = zero.row1;
      zero.row1 = std::min(zero_to, zero.row0 + ride_rows);
      zero.blocks = zero_blocks(zero.row1 - zero.row0, zero.row_bytes);
    };
    const int64_t early = std::min(zero_to / 16, (int64_t(24) << 20) / zero.row_bytes);
    const int64_t later = passes > 1 ? (zero_to / 2 + 2 * passes - 3) / (2 * passes - 2) : 0;
    for (int pass = 0; pass < passes; ++pass) {
      last = pass & 1;
      ps.shift = pass * bits;
      if (pass == 0) {
        SortItems<true, IdT> it{ids, nullptr, nullptr, start, urows, flags};
        ride(early, nullptr);
        hipLaunchKernelGGL((sort_counts<true, IdT>), dim3(ps.blocks + zero.blocks),
                           dim3(kSortThreads), 0, st, it, ps, count, hist, zero);
        ride(early, nullptr);
        hipLaunchKernelGGL((sort_scatter<true, IdT>), dim3(ps.blocks + zero.blocks),
                           dim3(kSortThreads), 0, st, it, ps, count, hist, key[0], pos[0], zero);
      } else {
        SortItems<false, IdT> it{nullptr, key[1 - last], pos[1 - last], start, urows, nullptr};
        ride(later, flags);
        hipLaunchKernelGGL((sort_counts<false, IdT>), dim3(ps.blocks + zero.blocks),
                           dim3(kSortThreads), 0, st, it, ps, count, hist, zero);
        ride(later, flags);
        hipLaunchKernelGGL((sort_scatter<false, IdT>), dim3(ps.blocks + zero.blocks),
                           dim3(kSortThreads), 0, st, it, ps, count, hist, key[last], pos[last],
                           zero);
      }
    }
    // The rest beside the sums; the last 64 MB beside their join, which waits
    // for the pieces of the longest runs one after the other (65536 Zipf ids: 159.4
    // us, 163.6 with none there, 161.1 with 32 MB, 159.9 with 128; uniform ids 165.2,
    // 166.2, 164.8 and 167.7).
    const int64_t rest = zero_to - zero.row1;
    const int64_t sums_to = zero_to - std::min(rest / 2, (int64_t(64) << 20) / zero.row_bytes);
    auto beside = [&](int64_t row0, int64_t row1) {
      return ZeroRows{zero.dw, zero.row_bytes, row0, row1, flags,
                      zero_blocks(row1 - row0, zero.row_bytes, 65536.0), zero.log2g};
    };
    join_zero = beside(sums_to, zero_to);
    zero = beside(zero.row1, sums_to);
  }
  a.key = key[last], a.pos = pos[last], a.count = count;
  a.partial = reinterpret_cast<float *>(ws + l.partial);
  a.partial_ld = l.partial_ld;
  a.chunk = static_cast<int>(l.chunk);
  if (dtype == 1)
    return gdtype == 1 ? launch_sums<true, true>(a, n, zero, join_zero, st)
                       : launch_sums<true, false>(a, n, zero, join_zero, st);
  return gdtype == 1 ? launch_sums<false, true>(a, n, zero, join_zero, st)
                     : launch_sums<false, false>(a, n, zero, join_zero, st);
}

}  // namespace

int launch_embed_scaled(const void *ids, int itype, int64_t n, const void *weight, int dtype,
                        int64_t shard_rows, int64_t dim, int64_t vocab_start, float scale,
                        void *out, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // clear a stale error so the status returned is this launch's
#define VPE_SCALED_ANY(BF16, IdT)                                                              \
  scaled_any<BF16>(static_cast<const IdT *>(ids), n, weight, shard_rows, dim, vocab_start,     \
                   scale, out, st)
  if (itype == 0) return dtype == 1 ? VPE_SCALED_ANY(true, int32_t) : VPE_SCALED_ANY(false, int32_t);
  return dtype == 1 ? VPE_SCALED_ANY(true, int64_t) : VPE_SCALED_ANY(false, int64_t);
#undef VPE_SCALED_ANY
}

int launch_embed_grad(const void *ids, int itype, int64_t n, const void *grad_out, int dtype,
                      int64_t dim, int64_t vocab_start, int64_t shard_rows, float scale,
                      void *grad_weight, int gdtype, bool accumulate, void *workspace,
                      void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  GradArgs a{};
  a.dy = static_cast<const char *>(grad_out), a.dim = dim, a.scale = scale;
  a.dw = static_cast<char *>(grad_weight), a.accumulate = accumulate;
  char *ws = static_cast<char *>(workspace);
  const uint64_t start = static_cast<uint64_t>(vocab_start);
  if (itype == 0)
    return grad_any(static_cast<const int32_t *>(ids), n, a, shard_rows, dtype, gdtype, start, ws,
                    st);
  return grad_any(static_cast<const int64_t *>(ids), n, a, shard_rows, dtype, gdtype, start, ws,
                  st);
}

}  // namespace vpe
