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
//  - Sum: runs are cut into pieces at every multiple of kGradPiece sorted
//    positions, so that a token with thousands of positions (natural text) is
//    spread over the chip; pieces that are not a whole run leave fp32 partial
//    sums, which a second kernel joins in the order of the pieces.
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
// LOG2G lanes (a power of two, at most 64) serve one row; each covers VPL
// vectors per sweep, issued before any store.
template <bool BF16, int EPV, int VPL, typename IdT>
__global__ __launch_bounds__(kBlock) void scaled_rows(const IdT *__restrict__ ids, int64_t n,
                                                     const void *__restrict__ weight,
                                                     uint64_t start, uint64_t rows, int64_t dim,
                                                     float scale, int log2g,
                                                     void *__restrict__ out) {
  typedef Vec<BF16, EPV> V;
  typedef typename V::raw raw;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kBlock + threadIdx.x;
  const int64_t row = t >> log2g;
  if (row >= n) return;
  const int group = 1 << log2g;
  const int lane = static_cast<int>(t) & (group - 1);
  // one unsigned compare covers both ends (a wrapped difference is >= rows)
  const uint64_t local = static_cast<uint64_t>(static_cast<int64_t>(ids[row])) - start;
  const bool owned = local < rows;
  const int64_t vr = dim / EPV;
  const raw *src = static_cast<const raw *>(weight) + static_cast<int64_t>(owned ? local : 0) * vr;
  raw *dst = static_cast<raw *>(out) + row * vr;
  for (int64_t c0 = lane; c0 < vr; c0 += static_cast<int64_t>(VPL) * group) {
    raw r[VPL];
#pragma unroll
    for (int c = 0; c < VPL; ++c) {
      const int64_t col = c0 + c * group;
      r[c] = raw(0);
      if (owned && col < vr) r[c] = src[col];
    }
#pragma unroll
    for (int c = 0; c < VPL; ++c) {
      const int64_t col = c0 + c * group;
      float v[EPV];
      V::widen(r[c], v);
#pragma unroll
      for (int e = 0; e < EPV; ++e) v[e] *= scale;
      raw o = V::narrow(v);
      if (!owned) o = raw(0);  // +0.0, also for a negative factor
      if (col < vr) __builtin_nontemporal_store(o, dst + col);
    }
  }
}

int ceil_log2(int64_t v) {
  int l = 0;
  while ((int64_t(1) << l) < v) ++l;
  return l;
}

// Rows per launch: keeps every grid inside the 32-bit work-item range.
constexpr int64_t kRowsPerLaunch = int64_t(1) << 24;

template <bool BF16, int EPV, typename IdT>
int scaled_launch(const IdT *ids, int64_t n, const void *weight, int64_t rows, int64_t dim,
                  int64_t start, float scale, void *out, hipStream_t st) {
  const int64_t vr = dim / EPV;
  const int log2g = std::min(6, ceil_log2(vr));
  for (int64_t r0 = 0; r0 < n; r0 += kRowsPerLaunch) {
    const int64_t nr = std::min(n - r0, kRowsPerLaunch);
    const unsigned blocks = static_cast<unsigned>(((nr << log2g) + kBlock - 1) / kBlock);
    void *o = static_cast<char *>(out) + r0 * dim * (BF16 ? 2 : 4);
#define VPE_SCALED(VPL)                                                                        \
  hipLaunchKernelGGL((scaled_rows<BF16, EPV, VPL, IdT>), dim3(blocks), dim3(kBlock), 0, st,    \
                     ids + r0, nr, weight, static_cast<uint64_t>(start),                       \
                     static_cast<uint64_t>(rows), dim, scale, log2g, o)
    if (vr <= 64) VPE_SCALED(1);
    else if (vr <= 128) VPE_SCALED(2);
    else if (vr <= 256) VPE_SCALED(4);
    else VPE_SCALED(8);
#undef VPE_SCALED
  }
  return static_cast<int>(hipGetLastError());
}

// Most elements per vector that divide the row and keep every base aligned
// (`low`: the bases' addresses or-ed together, in bytes).
int pick_epv(bool bf16, int64_t dim, uint64_t low) {
  const int size = bf16 ? 2 : 4;
  for (int epv = 16 / size; epv > 1; epv /= 2)
    if (dim % epv == 0 && low % (static_cast<uint64_t>(epv) * size) == 0) return epv;
  return 1;
}

template <typename IdT>
int scaled_any(const IdT *ids, int64_t n, const void *weight, int dtype, int64_t rows, int64_t dim,
               int64_t start, float scale, void *out, hipStream_t st) {
  const int epv = pick_epv(dtype == 1, dim,
                           reinterpret_cast<uint64_t>(weight) | reinterpret_cast<uint64_t>(out));
  if (dtype == 1) {
    switch (epv) {
      case 8: return scaled_launch<true, 8>(ids, n, weight, rows, dim, start, scale, out, st);
      case 4: return scaled_launch<true, 4>(ids, n, weight, rows, dim, start, scale, out, st);
      case 2: return scaled_launch<true, 2>(ids, n, weight, rows, dim, start, scale, out, st);
      default: return scaled_launch<true, 1>(ids, n, weight, rows, dim, start, scale, out, st);
    }
  }
  switch (epv) {
    case 4: return scaled_launch<false, 4>(ids, n, weight, rows, dim, start, scale, out, st);
    case 2: return scaled_launch<false, 2>(ids, n, weight, rows, dim, start, scale, out, st);
    default: return scaled_launch<false, 1>(ids, n, weight, rows, dim, start, scale, out, st);
  }
}

// ---------------------------------------------------------------------------
// stable sort of the owned positions by token
// ---------------------------------------------------------------------------
// Lanes of the wave whose digit equals this lane's, among lanes with `valid`.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits, bool valid) {
  uint64_t mask = __ballot(valid);
  for (int b = 0; b < bits; ++b) {
    const uint64_t one = __ballot((digit >> b) & 1u);
    mask &= ((digit >> b) & 1u) ? one : ~one;
  }
  return mask;
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

constexpr int kOneThreads = 1024;
constexpr int kOneWaves = kOneThreads / 64;
constexpr int kOneItems = static_cast<int>(kGradOneBlockIds / kOneThreads);
constexpr int kDigits = static_cast<int>(kSortDigits);

// Every owned id of at most kGradOneBlockIds, sorted in LDS.  Wave w takes the
// w-th run of items; a digit's items are ranked by (wave, round, lane), which
// is their order, so the sort is stable.
template <typename IdT>
__global__ __launch_bounds__(kOneThreads) void sort_one_block(
    const IdT *__restrict__ ids, int n, uint64_t start, uint64_t rows, int bits, int passes,
    uint32_t *__restrict__ key_out, uint32_t *__restrict__ pos_out,
    uint32_t *__restrict__ count_out, uint8_t *flags) {
  __shared__ uint32_t skey[kGradOneBlockIds];
  __shared__ uint16_t spos[kGradOneBlockIds];
  __shared__ uint16_t cnt_[kOneWaves][kDigits];
  __shared__ uint32_t sums[kDigits / 64];
  // a wave reads and updates its own counters in program order
  volatile uint16_t(*cnt)[kDigits] = cnt_;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_in_block();

  if (flags != nullptr) {
    u32x4 *f = reinterpret_cast<u32x4 *>(flags);
    const int64_t nf = static_cast<int64_t>((rows + 15) / 16);
    for (int64_t i = tid; i < nf; i += kOneThreads) f[i] = u32x4(0);
  }

  uint32_t key[kOneItems], pos[kOneItems], rank[kOneItems];
  bool have[kOneItems];
  int m = n;
  int rounds = (m + kOneThreads - 1) / kOneThreads;
#pragma unroll
  for (int r = 0; r < kOneItems; ++r) {
    const int i = (wave * rounds + r) * 64 + lane;
    have[r] = false, key[r] = 0, pos[r] = 0, rank[r] = 0;
    if (r < rounds && i < m) {
      const uint64_t local = static_cast<uint64_t>(static_cast<int64_t>(ids[i])) - start;
      have[r] = local < rows;
      key[r] = static_cast<uint32_t>(local);
      pos[r] = static_cast<uint32_t>(i);
    }
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    const uint32_t low = (1u << bits) - 1;
    for (int d = tid; d < kOneWaves * kDigits / 2; d += kOneThreads)
      reinterpret_cast<uint32_t *>(cnt_)[d] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kOneItems; ++r) {
      if (r < rounds) {
        const uint32_t d = (key[r] >> shift) & low;
        const uint64_t same = same_digit(d, bits, have[r]);
        if (have[r]) {
          const uint32_t seen = cnt[wave][d];
          rank[r] = seen + below(same);
          if (below(same) == 0) cnt[wave][d] = static_cast<uint16_t>(seen + __popcll(same));
        }
      }
    }
    __syncthreads();
    // exclusive sums over (digit, wave)
    uint32_t total = 0, incl = 0;
    if (tid < kDigits) {
      for (int w = 0; w < kOneWaves; ++w) total += cnt_[w][tid];
      incl = wave_scan(total);
      if (lane == 63) sums[wave] = incl;
    }
    __syncthreads();
    if (tid < kDigits) {
      uint32_t at = incl - total;
      for (int w = 0; w < wave; ++w) at += sums[w];
      for (int w = 0; w < kOneWaves; ++w) {
        const uint32_t c = cnt_[w][tid];
        cnt_[w][tid] = static_cast<uint16_t>(at);
        at += c;
      }
    }
    uint32_t all = 0;
    for (int w = 0; w < kDigits / 64; ++w) all += sums[w];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kOneItems; ++r) {
      if (r < rounds && have[r]) {
        const uint32_t to = cnt_[wave][(key[r] >> shift) & low] + rank[r];
        skey[to] = key[r];
        spos[to] = static_cast<uint16_t>(pos[r]);
      }
    }
    __syncthreads();
    m = static_cast<int>(all);
    rounds = (m + kOneThreads - 1) / kOneThreads;
#pragma unroll
    for (int r = 0; r < kOneItems; ++r) {
      const int i = (wave * rounds + r) * 64 + lane;
      have[r] = r < rounds && i < m;
      if (have[r]) key[r] = skey[i], pos[r] = spos[i];
    }
  }
#pragma unroll
  for (int r = 0; r < kOneItems; ++r) {
    const int i = (wave * rounds + r) * 64 + lane;
    if (have[r]) {
      key_out[i] = key[r];
      pos_out[i] = pos[r];
      if (flags != nullptr) flags[key[r]] = 1;
    }
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

template <bool FIRST, typename IdT>
__global__ __launch_bounds__(kBlock) void sort_counts(SortItems<FIRST, IdT> items, int64_t n,
                                                     const uint32_t *count, int64_t tile,
                                                     int shift, int bits, uint32_t *hist,
                                                     uint8_t *flags) {
  __shared__ uint32_t h[kDigits];
  const int tid = threadIdx.x;
  if (FIRST && flags != nullptr) {
    u32x4 *f = reinterpret_cast<u32x4 *>(flags);
    const int64_t nf = static_cast<int64_t>((items.rows + 15) / 16);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBlock + tid; i < nf;
         i += static_cast<int64_t>(gridDim.x) * kBlock)
      f[i] = u32x4(0);
  }
  for (int d = tid; d < kDigits; d += kBlock) h[d] = 0;
  __syncthreads();
  const int64_t m = FIRST ? n : static_cast<int64_t>(*count);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * tile;
  const int64_t i1 = i0 + tile < m ? i0 + tile : m;
  const uint32_t low = (1u << bits) - 1;
  for (int64_t i = i0 + tid; i < i1; i += kBlock) {
    uint32_t key;
    if (items.get(i, key)) atomicAdd(&h[(key >> shift) & low], 1u);
  }
  __syncthreads();
  for (int d = tid; d < kDigits; d += kBlock)
    hist[static_cast<int64_t>(blockIdx.x) * kDigits + d] = h[d];
}

template <bool FIRST, typename IdT>
__global__ __launch_bounds__(kBlock) void sort_scatter(SortItems<FIRST, IdT> items, int64_t n,
                                                      uint32_t *count, int64_t tile, int shift,
                                                      int bits, const uint32_t *__restrict__ hist,
                                                      uint32_t *__restrict__ key_out,
                                                      uint32_t *__restrict__ pos_out,
                                                      uint8_t *flags) {
  __shared__ uint32_t at_[kWaves][kDigits];
  __shared__ uint32_t base[kDigits];
  __shared__ uint32_t sums[kWaves];
  volatile uint32_t(*at)[kDigits] = at_;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_in_block();
  const int64_t m = FIRST ? n : static_cast<int64_t>(*count);

  // where this workgroup's items of each digit go: the digits below, and the
  // same digit of the workgroups before (thread t: digits 2t and 2t + 1)
  uint32_t before0 = 0, before1 = 0, total0 = 0, total1 = 0;
  const u32x2 *h2 = reinterpret_cast<const u32x2 *>(hist);
#pragma unroll 8
  for (unsigned b = 0; b < gridDim.x; ++b) {
    const u32x2 c = h2[b * (kDigits / 2) + tid];
    if (b < blockIdx.x) before0 += c[0], before1 += c[1];
    total0 += c[0], total1 += c[1];
  }
  const uint32_t incl = wave_scan(total0 + total1);
  if (lane == 63) sums[wave] = incl;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) at_[w][2 * tid] = 0, at_[w][2 * tid + 1] = 0;
  __syncthreads();
  uint32_t first = incl - total0 - total1;
  for (int w = 0; w < wave; ++w) first += sums[w];
  base[2 * tid] = first + before0;
  base[2 * tid + 1] = first + total0 + before1;
  if (FIRST && blockIdx.x == 0 && tid == kBlock - 1) *count = first + total0 + total1;

  // counts of each wave's quarter of the tile
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * tile + wave * (tile / kWaves);
  const int64_t i1 = i0 + tile / kWaves < m ? i0 + tile / kWaves : m;
  const uint32_t low = (1u << bits) - 1;
  for (int64_t i = i0 + lane; i < i1; i += 64) {
    uint32_t key;
    if (items.get(i, key)) atomicAdd(&at_[wave][(key >> shift) & low], 1u);
  }
  __syncthreads();
  for (int d = tid; d < kDigits; d += kBlock) {
    uint32_t to = base[d];
    for (int w = 0; w < kWaves; ++w) {
      const uint32_t c = at_[w][d];
      at_[w][d] = to;
      to += c;
    }
  }
  __syncthreads();
  for (int64_t r = i0; r < i1; r += 64) {
    const int64_t i = r + lane;
    uint32_t key = 0;
    const bool have = i < i1 && items.get(i, key);
    const uint32_t d = (key >> shift) & low;
    const uint64_t same = same_digit(d, bits, have);
    if (have) {
      const uint32_t seen = at[wave][d];
      const uint32_t to = seen + below(same);
      if (below(same) == 0) at[wave][d] = seen + __popcll(same);
      key_out[to] = key;
      pos_out[to] = FIRST ? static_cast<uint32_t>(i) : items.pos_in[i];
      if (FIRST && flags != nullptr) flags[key] = 1;
    }
  }
}

// ---------------------------------------------------------------------------
// sums of the sorted rows
// ---------------------------------------------------------------------------
struct GradArgs {
  const uint32_t *key, *pos, *count;
  const void *dy;
  int64_t dim;
  float scale;
  void *dw;
  bool accumulate;
  float *partial;      // [2 * pieces][dim]
  const uint8_t *flags;
  int64_t rows;
  int col_blocks;      // waves per row
};

constexpr int kPiece = static_cast<int>(kGradPiece);
constexpr int kZeroRowsPerWave = 16;

template <bool OUT16, int EPV>
__device__ __forceinline__ void write_row(const GradArgs &a, int64_t elem, const float (&sum)[EPV]) {
  float v[EPV];
  if (a.accumulate) {
    load_vec<OUT16, EPV>(a.dw, elem, v);
#pragma unroll
    for (int e = 0; e < EPV; ++e) v[e] = v[e] + a.scale * sum[e];
  } else {
#pragma unroll
    for (int e = 0; e < EPV; ++e) v[e] = a.scale * sum[e];
  }
  store_vec_nt<OUT16, EPV>(a.dw, elem, v);
}

// Waves [0, positions * col_blocks) take one sorted position and column block
// each: the wave whose position begins a piece sums it, the others end at
// once.  The waves after them write the zero rows, kZeroRowsPerWave each.
template <bool IN16, bool OUT16, int EPV, int VPL>
__global__ __launch_bounds__(kBlock) void grad_pieces(GradArgs a, int64_t p0, int64_t n_pos,
                                                     int64_t pos_blocks, int64_t zero_row0) {
  const int lane = threadIdx.x & 63;
  const int64_t vr = a.dim / EPV;
  if (static_cast<int64_t>(blockIdx.x) >= pos_blocks) {
    const int64_t w = (static_cast<int64_t>(blockIdx.x) - pos_blocks) * kWaves + wave_in_block();
    const int64_t r0 = zero_row0 + w * kZeroRowsPerWave;
    const bool here = lane < kZeroRowsPerWave && r0 + lane < a.rows;
    uint64_t empty = __ballot(here && a.flags[here ? r0 + lane : 0] == 0);
    float zero[EPV];
#pragma unroll
    for (int e = 0; e < EPV; ++e) zero[e] = 0.f;
    while (empty) {
      const int64_t row = r0 + __builtin_ctzll(empty);
      empty &= empty - 1;
      for (int64_t c = lane; c < vr; c += 64)
        store_vec_nt<OUT16, EPV>(a.dw, row * a.dim + c * EPV, zero);
    }
    return;
  }
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * kWaves + wave_in_block();
  const int64_t rel = wave / a.col_blocks;
  if (rel >= n_pos) return;
  const int64_t p = p0 + rel;
  const int64_t n = *a.count;
  if (p >= n) return;
  const int64_t col0 = (wave - rel * a.col_blocks) * (64 * VPL);
  const uint32_t token = a.key[p];
  const bool head = p == 0 || a.key[p - 1] != token;
  if (!head && p % kPiece != 0) return;
  const int64_t limit = (p / kPiece + 1) * kPiece < n ? (p / kPiece + 1) * kPiece : n;
  const bool mine = lane < kPiece && p + lane < limit && a.key[p + lane] == token;
  const uint32_t src = mine ? a.pos[p + lane] : 0;
  const int len = __popcll(__ballot(mine));
  const bool whole = head && !(p + len == limit && limit < n && a.key[limit] == token);

  float sum[VPL][EPV];
#pragma unroll
  for (int c = 0; c < VPL; ++c)
#pragma unroll
    for (int e = 0; e < EPV; ++e) sum[c][e] = 0.f;
  constexpr int kDeep = 4;  // rows in flight
  for (int i = 0; i < len; i += kDeep) {
    float v[kDeep][VPL][EPV];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const uint32_t s = static_cast<uint32_t>(
          __builtin_amdgcn_readlane(static_cast<int>(src), i + u < len ? i + u : 0));
      const int64_t at = static_cast<int64_t>(s) * a.dim;
#pragma unroll
      for (int c = 0; c < VPL; ++c) {
        const int64_t col = col0 + c * 64 + lane;
#pragma unroll
        for (int e = 0; e < EPV; ++e) v[u][c][e] = 0.f;
        if (i + u < len && col < vr) load_vec<IN16, EPV>(a.dy, at + col * EPV, v[u][c]);
      }
    }
#pragma unroll
    for (int u = 0; u < kDeep; ++u)
#pragma unroll
      for (int c = 0; c < VPL; ++c)
#pragma unroll
        for (int e = 0; e < EPV; ++e) sum[c][e] += v[u][c][e];
  }
#pragma unroll
  for (int c = 0; c < VPL; ++c) {
    const int64_t col = col0 + c * 64 + lane;
    if (col >= vr) continue;
    if (whole) {
      write_row<OUT16, EPV>(a, static_cast<int64_t>(token) * a.dim + col * EPV, sum[c]);
    } else {
      // slot 2c: the piece that begins with chunk c; 2c + 1: the one inside it
      const int64_t slot = 2 * (p / kPiece) + (p % kPiece != 0);
      float *o = a.partial + slot * a.dim + col * EPV;
#pragma unroll
      for (int e = 0; e < EPV; ++e) o[e] = sum[c][e];
    }
  }
}

// One wave per chunk of kPiece positions and column block: the run that leaves
// the chunk having begun in it is joined from its pieces, in order.
template <bool OUT16, int EPV>
__global__ __launch_bounds__(kBlock) void grad_join(GradArgs a, int64_t chunk0, int64_t n_chunks) {
  const int lane = threadIdx.x & 63;
  const int64_t vr = a.dim / EPV;
  const int64_t blocks = (vr + 63) / 64;
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * kWaves + wave_in_block();
  const int64_t rel = wave / blocks;
  const int64_t c = chunk0 + rel;
  const int64_t n = *a.count;
  const int64_t next = (c + 1) * kPiece;
  if (rel >= n_chunks || next >= n) return;
  const uint32_t token = a.key[next];
  if (a.key[next - 1] != token) return;
  const bool whole_chunk = a.key[next - kPiece] == token;
  if (whole_chunk && c > 0 && a.key[next - kPiece - 1] == token) return;  // began before
  // chunks after c that begin with the token
  int64_t more = 1;
  for (;;) {
    const int64_t q = (c + 1 + more + lane) * kPiece;
    const uint64_t on = __ballot(q < n && a.key[q < n ? q : 0] == token);
    if (on != ~0ull) {
      more += __builtin_ctzll(~on);
      break;
    }
    more += 64;
  }
  const int64_t col = (wave - rel * blocks) * 64 + lane;
  if (col >= vr) return;
  float sum[EPV];
  load_vec<false, EPV>(a.partial + (2 * c + (whole_chunk ? 0 : 1)) * a.dim, col * EPV, sum);
#pragma unroll 8
  for (int64_t i = 1; i <= more; ++i) {
    float v[EPV];
    load_vec<false, EPV>(a.partial + 2 * (c + i) * a.dim, col * EPV, v);
#pragma unroll
    for (int e = 0; e < EPV; ++e) sum[e] += v[e];
  }
  write_row<OUT16, EPV>(a, static_cast<int64_t>(token) * a.dim + col * EPV, sum);
}

template <bool IN16, bool OUT16, int EPV, int VPL>
void launch_pieces(GradArgs a, int64_t n, hipStream_t st) {
  const int64_t vr = a.dim / EPV;
  const int64_t blocks = (vr + 64 * VPL - 1) / (64 * VPL);
  a.col_blocks = static_cast<int>(blocks);
  // positions and zero rows per launch: grids stay inside the 32-bit range
  const int64_t pos_step = std::max<int64_t>(1, (int64_t(1) << 24) / blocks);
  const int64_t zero_step = (int64_t(1) << 24) * kZeroRowsPerWave;
  const int64_t zero_rows = a.accumulate ? 0 : a.rows;
  for (int64_t p = 0, z = 0; p < n || z < zero_rows; p += pos_step, z += zero_step) {
    const int64_t np = std::max<int64_t>(0, std::min(pos_step, n - p));
    const int64_t nz = std::max<int64_t>(0, std::min(zero_step, zero_rows - z));
    const int64_t pb = (np * blocks + kWaves - 1) / kWaves;
    const int64_t zb = (nz + kZeroRowsPerWave * kWaves - 1) / (kZeroRowsPerWave * kWaves);
    hipLaunchKernelGGL((grad_pieces<IN16, OUT16, EPV, VPL>), dim3(static_cast<unsigned>(pb + zb)),
                       dim3(kBlock), 0, st, a, p, np, pb, z);
  }
}

template <bool IN16, bool OUT16, int EPV>
int launch_sums(const GradArgs &a, int64_t n, hipStream_t st) {
  if (a.dim / EPV <= 64) launch_pieces<IN16, OUT16, EPV, 1>(a, n, st);
  else launch_pieces<IN16, OUT16, EPV, 2>(a, n, st);
  if (n > kPiece) {
    const int64_t chunks = (n + kPiece - 1) / kPiece;
    const int64_t blocks = (a.dim / EPV + 63) / 64;
    const int64_t step = std::max<int64_t>(1, (int64_t(1) << 24) / blocks);
    for (int64_t c = 0; c < chunks; c += step) {
      const int64_t nc = std::min(step, chunks - c);
      hipLaunchKernelGGL((grad_join<OUT16, EPV>),
                         dim3(static_cast<unsigned>((nc * blocks + kWaves - 1) / kWaves)),
                         dim3(kBlock), 0, st, a, c, nc);
    }
  }
  return static_cast<int>(hipGetLastError());
}

template <bool IN16, bool OUT16>
int launch_sums_any(const GradArgs &a, int64_t n, hipStream_t st) {
  // vectors of the same elements on both sides, at most 16 bytes of the input
  const uint64_t dy = reinterpret_cast<uint64_t>(a.dy), dw = reinterpret_cast<uint64_t>(a.dw);
  const int epv = std::min(pick_epv(IN16, a.dim, dy), OUT16 ? pick_epv(true, a.dim, dw)
                                                      : a.dim % 8 == 0 && dw % 16 == 0
                                                          ? 8
                                                          : pick_epv(false, a.dim, dw));
  if constexpr (IN16) {
    if (epv == 8) return launch_sums<IN16, OUT16, 8>(a, n, st);
  }
  if (epv >= 4) return launch_sums<IN16, OUT16, 4>(a, n, st);
  if (epv == 2) return launch_sums<IN16, OUT16, 2>(a, n, st);
  return launch_sums<IN16, OUT16, 1>(a, n, st);
}

template <typename IdT>
int grad_any(const IdT *ids, int64_t n, GradArgs a, int dtype, int gdtype, uint64_t start,
             char *ws, hipStream_t st) {
  const EmbedGradLayout l = embed_grad_layout(n, a.rows, a.dim);
  uint32_t *key[2] = {reinterpret_cast<uint32_t *>(ws + l.key[0]),
                      reinterpret_cast<uint32_t *>(ws + l.key[1])};
  uint32_t *pos[2] = {reinterpret_cast<uint32_t *>(ws + l.pos[0]),
                      reinterpret_cast<uint32_t *>(ws + l.pos[1])};
  uint32_t *count = reinterpret_cast<uint32_t *>(ws + l.count);
  uint32_t *hist = reinterpret_cast<uint32_t *>(ws + l.hist);
  uint8_t *flags = a.accumulate ? nullptr : reinterpret_cast<uint8_t *>(ws + l.flags);
  const uint64_t rows = static_cast<uint64_t>(a.rows);
  const int key_bits = std::max(1, ceil_log2(a.rows));
  const int passes = (key_bits + 8) / 9;
  const int bits = (key_bits + passes - 1) / passes;
  int last = 0;
  if (n <= kGradOneBlockIds) {
    hipLaunchKernelGGL((sort_one_block<IdT>), dim3(1), dim3(kOneThreads), 0, st, ids,
                       static_cast<int>(n), start, rows, bits, passes, key[0], pos[0], count,
                       flags);
  } else {
    // at least kSortTile items per workgroup, at most kSortMaxBlocks workgroups
    const int64_t unit = kSortTile * kSortMaxBlocks;
    const int64_t tile = kSortTile * ((n + unit - 1) / unit);
    const unsigned blocks = static_cast<unsigned>((n + tile - 1) / tile);
    for (int pass = 0; pass < passes; ++pass) {
      last = pass & 1;
      const int shift = pass * bits;
      if (pass == 0) {
        SortItems<true, IdT> it{ids, nullptr, nullptr, start, rows};
        hipLaunchKernelGGL((sort_counts<true, IdT>), dim3(blocks), dim3(kBlock), 0, st, it, n,
                           count, tile, shift, bits, hist, flags);
        hipLaunchKernelGGL((sort_scatter<true, IdT>), dim3(blocks), dim3(kBlock), 0, st, it, n,
                           count, tile, shift, bits, hist, key[0], pos[0], flags);
      } else {
        SortItems<false, IdT> it{nullptr, key[1 - last], pos[1 - last], start, rows};
        hipLaunchKernelGGL((sort_counts<false, IdT>), dim3(blocks), dim3(kBlock), 0, st, it, n,
                           count, tile, shift, bits, hist, flags);
        hipLaunchKernelGGL((sort_scatter<false, IdT>), dim3(blocks), dim3(kBlock), 0, st, it, n,
                           count, tile, shift, bits, hist, key[last], pos[last], flags);
      }
    }
  }
  a.key = key[last], a.pos = pos[last], a.count = count, a.flags = flags;
  a.partial = reinterpret_cast<float *>(ws + l.partial);
  if (dtype == 1)
    return gdtype == 1 ? launch_sums_any<true, true>(a, n, st)
                       : launch_sums_any<true, false>(a, n, st);
  return gdtype == 1 ? launch_sums_any<false, true>(a, n, st)
                     : launch_sums_any<false, false>(a, n, st);
}

}  // namespace

int launch_embed_scaled(const void *ids, int itype, int64_t n, const void *weight, int dtype,
                        int64_t shard_rows, int64_t dim, int64_t vocab_start, float scale,
                        void *out, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // clear a stale error so the status returned is this launch's
  if (itype == 0)
    return scaled_any(static_cast<const int32_t *>(ids), n, weight, dtype, shard_rows, dim,
                      vocab_start, scale, out, st);
  return scaled_any(static_cast<const int64_t *>(ids), n, weight, dtype, shard_rows, dim,
                    vocab_start, scale, out, st);
}

int launch_embed_grad(const void *ids, int itype, int64_t n, const void *grad_out, int dtype,
                      int64_t dim, int64_t vocab_start, int64_t shard_rows, float scale,
                      void *grad_weight, int gdtype, bool accumulate, void *workspace,
                      void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  GradArgs a{};
  a.dy = grad_out, a.dim = dim, a.scale = scale, a.dw = grad_weight, a.accumulate = accumulate;
  a.rows = shard_rows;
  char *ws = static_cast<char *>(workspace);
  const uint64_t start = static_cast<uint64_t>(vocab_start);
  if (itype == 0)
    return grad_any(static_cast<const int32_t *>(ids), n, a, dtype, gdtype, start, ws, st);
  return grad_any(static_cast<const int64_t *>(ids), n, a, dtype, gdtype, start, ws, st);
}

}  // namespace vpe
