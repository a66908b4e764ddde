// Distillation from a teacher's top logits for gfx950: per-shard statistics,
// the loss, and the gradient of the logits.
//
// All of it is bound by HBM: the statistics read a rank's logits once, the
// gradient reads them once and writes once; a row's teacher entries (at most
// 1024) are small beside its columns.
//  - Statistics: waves take slices of 256 vectors of a row: their maximum first,
//    then 2^((z - maximum) log2(e) / T), one v_exp_f32 per logit, so no sum is
//    rescaled inside; the slices' (maximum, sum) pairs are joined, and one wave
//    per row takes the products with the teacher's entries.  One workgroup per
//    row does all of it; a few long rows are cut into slices over the chip, and a
//    second kernel joins their pairs from memory.
//  - Gradient: P exp(z/T - lse) for every column, and for the entries' columns
//    the entries' probabilities taken off.  Those columns are read before the
//    dense pass (the gradient may overwrite the logits) and written again
//    after it.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "vpe_device.h"
#include "vpe_train_launch.h"

namespace vpe {
namespace {

using namespace dev;

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / 64;
constexpr int kMaxEntries = 1024;
constexpr int kEntriesPerThread = kMaxEntries / kBlock;
constexpr float kMostFloat = 3.4028234663852886e38f;

__device__ __forceinline__ float neg_inf() { return -__builtin_huge_valf(); }
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Block-wide maximum and sum, the same in every thread.
__device__ __forceinline__ float block_max(float v, float *lds) {
  v = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[wave_in_block()] = v;
  __syncthreads();
  float r = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) r = fmaxf(r, lds[w]);
  return r;
}
template <typename T>
__device__ __forceinline__ T block_sum(T v, T *lds) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[wave_in_block()] = v;
  __syncthreads();
  T r = lds[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) r += lds[w];
  return r;
}

// ---------------------------------------------------------------------------
// a row's teacher entries
// ---------------------------------------------------------------------------
struct TeacherArgs {
  const void *ids, *logits;
  const float *lse;
  int itype, dtype, k;
  int64_t vocab;
  float temperature;
  float inv_t;   // 1 / T
  float to_log2; // log2(e) / T
};

// Entry e of the row: its scaled logit t_e / T, or -inf (p_e = 0) for padding.
__device__ __forceinline__ float entry(const TeacherArgs &t, int64_t row, int e, int64_t &id) {
  const int64_t i = row * t.k + e;
  id = t.itype == 0 ? static_cast<const int32_t *>(t.ids)[i]
                    : static_cast<const int64_t *>(t.ids)[i];
  if (static_cast<uint64_t>(id) >= static_cast<uint64_t>(t.vocab)) return neg_inf();
  const float v = t.dtype == 0
                      ? static_cast<const float *>(t.logits)[i]
                      : __uint_as_float(static_cast<uint32_t>(
                            static_cast<const uint16_t *>(t.logits)[i]) << 16);
  return v / t.temperature;
}

// p_e of the thread's entries e = threadIdx.x + kBlock * i, their columns in
// the shard [start, start + cols) (-1: elsewhere, or p_e = 0); returns P.
__device__ __forceinline__ float teacher_row(const TeacherArgs &t, int64_t row, int64_t start,
                                             int64_t cols, float (&p)[kEntriesPerThread],
                                             int (&col)[kEntriesPerThread], float *lds) {
  float mx = neg_inf();
#pragma unroll
  for (int i = 0; i < kEntriesPerThread; ++i) {
    const int e = threadIdx.x + kBlock * i;
    p[i] = neg_inf();
    col[i] = -1;
    if (e < t.k) {
      int64_t id;
      p[i] = entry(t, row, e, id);
      const uint64_t local = static_cast<uint64_t>(id) - static_cast<uint64_t>(start);
      if (local < static_cast<uint64_t>(cols)) col[i] = static_cast<int>(local);
    }
    mx = fmaxf(mx, p[i]);
  }
  float sum = 0.f;
  if (t.lse != nullptr) {
    const float l = t.lse[row];
#pragma unroll
    for (int i = 0; i < kEntriesPerThread; ++i) {
      p[i] = p[i] == neg_inf() ? 0.f : expf(p[i] - l);
      sum += p[i];
    }
    sum = block_sum(sum, lds);
  } else {
    mx = block_max(mx, lds);
    if (mx == neg_inf()) mx = 0.f;  // no entry counts (NaN ones stay NaN)
#pragma unroll
    for (int i = 0; i < kEntriesPerThread; ++i) p[i] = expf(p[i] - mx), sum += p[i];
    sum = block_sum(sum, lds);
    if (sum != 0.f) {
#pragma unroll
      for (int i = 0; i < kEntriesPerThread; ++i) p[i] /= sum;
      sum = sum != sum ? sum : 1.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kEntriesPerThread; ++i)
    if (p[i] == 0.f) col[i] = -1;
  return sum;
}

// ---------------------------------------------------------------------------
// student rows
// ---------------------------------------------------------------------------
template <bool BF16>
struct Row : Vec<BF16, BF16 ? 8 : 4> {
  static constexpr int kEpv = BF16 ? 8 : 4;
};

// The sum of exp(z / T) over some columns as (their largest logit, the sum of
// exp((z - largest) / T)).  The difference comes before the factor: multiples
// of a mask's lowest value would be infinite.
struct Pair {
  float mx, sum;
};
__device__ __forceinline__ Pair join(Pair a, Pair b, float to_log2) {
  const float m = fmaxf(a.mx, b.mx);
  // (of equal infinities the difference would be NaN)
  const float sa = a.mx == m ? a.sum : a.sum * exp2_fast((a.mx - m) * to_log2);
  const float sb = b.mx == m ? b.sum : b.sum * exp2_fast((b.mx - m) * to_log2);
  return Pair{m, sa + sb};
}
// In 64 bits (one value per row).
__device__ __forceinline__ float natural_log(Pair p, float temperature) {
  return static_cast<float>(static_cast<double>(p.mx) / static_cast<double>(temperature) +
                            log(static_cast<double>(p.sum)));
}

__device__ __forceinline__ Pair wave_join(Pair p, float to_log2) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2)
    p = join(p, Pair{__shfl_xor(p.mx, d), __shfl_xor(p.sum, d)}, to_log2);
  return p;
}

struct ShardArgs {
  const char *base;  // first column of row 0
  int64_t ld_bytes;
  int64_t cols, vocab_start;
  int slices;        // pieces a row is cut into
  int64_t slice;     // columns of each, a multiple of the vector length
};

constexpr int kPairVecs = 4;  // vectors per lane and pair

// Slice `s` of the row at p, by one wave: its vectors, -inf where they end.
template <bool BF16>
struct Slice {
  typedef Row<BF16> R;
  static constexpr int kEpv = R::kEpv, kSize = BF16 ? 2 : 4;
  u32x4 raw[kPairVecs];
  __device__ __forceinline__ void load(const ShardArgs &z, const char *p, int64_t s) {
    const int64_t j0 = s * z.slice + (threadIdx.x & 63) * kEpv;
#pragma unroll
    for (int u = 0; u < kPairVecs; ++u) {
      const int64_t j = j0 + u * (64 * kEpv);
      raw[u] = BF16 ? u32x4(0xff80ff80u) : u32x4(0xff800000u);  // -inf: adds nothing
      if (j + kEpv <= z.cols) raw[u] = *reinterpret_cast<const typename R::loose *>(p + j * kSize);
    }
  }
  // The maximum, and the sum with it taken off.
  __device__ __forceinline__ Pair pair(const ShardArgs &z, const char *p, int64_t s,
                                       float to_log2) const {
    // the row's last columns where they do not fill a vector: one lane's
    const int64_t j0 = s * z.slice + (threadIdx.x & 63) * kEpv, tail = z.cols - z.cols % kEpv;
    const bool ragged = tail < z.cols && j0 <= tail && (tail - j0) % (64 * kEpv) == 0 &&
                        tail - j0 < kPairVecs * 64 * kEpv;
    float mx = neg_inf();
#pragma unroll
    for (int u = 0; u < kPairVecs; ++u) {
      float v[kEpv];
      Vec<BF16, kEpv>::widen(raw[u], v);
#pragma unroll
      for (int e = 0; e < kEpv; ++e) mx = fmaxf(mx, v[e]);
    }
    if (ragged) {
#pragma nounroll
      for (int64_t i = tail; i < z.cols; ++i) mx = fmaxf(mx, load_one<BF16>(p, i));
    }
    mx = wave_max(mx);
    const float off = __builtin_isinf(mx) ? 0.f : mx;  // +inf: an infinite sum
    float sum = 0.f;
#pragma unroll
    for (int u = 0; u < kPairVecs; ++u) {
      float v[kEpv];
      Vec<BF16, kEpv>::widen(raw[u], v);
#pragma unroll
      for (int e = 0; e < kEpv; ++e) sum += exp2_fast((v[e] - off) * to_log2);
    }
    if (ragged) {
#pragma nounroll
      for (int64_t i = tail; i < z.cols; ++i)
        sum += exp2_fast((load_one<BF16>(p, i) - off) * to_log2);
    }
    return Pair{mx, wave_sum(sum)};
  }
};

// One wave per pair of a row (grid: pairs / kWaves, rows), for few long rows:
// 8 fp32 rows of 151936 take 3.1 us here and 5 us in distill_rows, latency both.
// (8 vectors per lane instead of 4: 3.2 us; 31.4 instead of 30.6 us for 1024 bf16
// rows of 75968.)
template <bool BF16>
__global__ __launch_bounds__(kBlock) void distill_pairs(ShardArgs z, float to_log2,
                                                       Pair *__restrict__ pairs) {
  const int64_t row = blockIdx.y;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * kWaves + wave_in_block();
  if (s >= z.slices) return;
  const char *p = z.base + row * z.ld_bytes;
  Slice<BF16> slice;
  slice.load(z, p, s);
  const Pair a = slice.pair(z, p, s, to_log2);
  if ((threadIdx.x & 63) == 0) pairs[row * z.slices + s] = a;
}

// A row's entries by one wave: the largest t_e / T (or the given
// log-sum-exp), that the powers are taken from.
__device__ __forceinline__ float entries_shift(const TeacherArgs &t, int64_t row) {
  if (t.lse != nullptr) return t.lse[row];
  float mx = neg_inf();
  int64_t id;
  for (int e = threadIdx.x & 63; e < t.k; e += 64) mx = fmaxf(mx, entry(t, row, e, id));
  mx = wave_max(mx);
  return mx == neg_inf() ? 0.f : mx;  // no entry counts (NaN ones stay NaN)
}

// The entries' product with the shard's logits (the row at p), by one wave.
template <bool BF16>
__device__ __forceinline__ float entries_dot(const ShardArgs &z, const TeacherArgs &t, int64_t row,
                                             const char *p) {
  const float shift = entries_shift(t, row);
  // in 64 bits: the loss is a small difference of this and the log-sum-exp
  double dot = 0.0, total = 0.0;
  for (int e = threadIdx.x & 63; e < t.k; e += 64) {
    int64_t id;
    const float v = entry(t, row, e, id);
    const float w = v == neg_inf() ? 0.f : expf(v - shift);
    total += static_cast<double>(w);
    const uint64_t local = static_cast<uint64_t>(id) - static_cast<uint64_t>(z.vocab_start);
    if (w != 0.f && local < static_cast<uint64_t>(z.cols))
      dot += static_cast<double>(w) *
             static_cast<double>(load_one<BF16>(p, static_cast<int64_t>(local)));
  }
  dot = wave_sum(dot);
  total = t.lse != nullptr ? 1.0 : wave_sum(total);
  return total == 0.0 ? 0.f : static_cast<float>(dot / total / static_cast<double>(t.temperature));
}

// One wave per row: the pairs joined (shard_lse != nullptr), and the entries'
// product.
template <bool BF16>
__global__ __launch_bounds__(kBlock) void distill_rows(ShardArgs z, TeacherArgs t, int64_t m,
                                                      const Pair *__restrict__ pairs,
                                                      float *__restrict__ shard_lse,
                                                      float *__restrict__ shard_dot) {
  const int lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWaves + wave_in_block();
  if (row >= m) return;
  const float dot = entries_dot<BF16>(z, t, row, z.base + row * z.ld_bytes);
  if (lane == 0) shard_dot[row] = dot;
  if (shard_lse == nullptr) return;
  Pair a{neg_inf(), 0.f};
  for (int s = lane; s < z.slices; s += 64) a = join(a, pairs[row * z.slices + s], t.to_log2);
  a = wave_join(a, t.to_log2);
  if (lane == 0) shard_lse[row] = natural_log(a, t.temperature);
}

// One workgroup per row: both at once, without pairs in memory.  The last wave
// takes the entries, the others the row's slices in turn, the next one's vectors
// on their way.  Bound by HBM: 1024 bf16 rows of 75968 (156 MB) in 31 us, 5.0
// TB/s, by itself, 35 us between a training step's writes; 1024 fp32 rows of
// 151936 in 109 us, 5.7 TB/s.
constexpr int kRowWaves = 8;  // at most
template <bool BF16>
__global__ __launch_bounds__(64 * (kRowWaves + 1)) void distill_whole_rows(
    ShardArgs z, TeacherArgs t, int waves, float *__restrict__ shard_lse,
    float *__restrict__ shard_dot) {
  __shared__ Pair part[kRowWaves];
  const int lane = threadIdx.x & 63, wave = wave_in_block();
  const int64_t row = blockIdx.x;
  const char *p = z.base + row * z.ld_bytes;
  if (wave == waves) {
    const float dot = entries_dot<BF16>(z, t, row, p);
    if (lane == 0) shard_dot[row] = dot;
  } else {
    Slice<BF16> next;
    next.load(z, p, wave);
    Pair a{neg_inf(), 0.f};
#pragma nounroll
    for (int s = wave; s < z.slices; s += waves) {
      const Slice<BF16> now = next;
      if (s + waves < z.slices) next.load(z, p, s + waves);
      a = join(a, now.pair(z, p, s, t.to_log2), t.to_log2);
    }
    if (lane == 0) part[wave] = a;
  }
  __syncthreads();
  if (wave != 0) return;
  const Pair a = wave_join(lane < waves ? part[lane] : Pair{neg_inf(), 0.f}, t.to_log2);
  if (lane == 0) shard_lse[row] = natural_log(a, t.temperature);
}

struct Parts {
  const float *lse[64];
  const float *dot[64];
};

// One wave per row.  Sums of a few tens of near-cancelling terms per row: the
// row's scalars are joined in 64 bits and rounded once.  Bound by the latency of
// three loads that follow each other: 4.9 us for 8 rows, 5.4 us for 1024.
__global__ __launch_bounds__(kBlock) void distill_loss_rows(Parts parts, int n_parts, int64_t m,
                                                           TeacherArgs t, float *loss,
                                                           float *lse) {
  const int lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWaves + wave_in_block();
  if (row >= m) return;
  double dot = 0.0;
  float top = neg_inf();
  for (int r = 0; r < n_parts; ++r) {
    dot += static_cast<double>(parts.dot[r][row]);
    top = fmaxf(top, parts.lse[r][row]);
  }
  const float shift = __builtin_isinf(top) ? 0.f : top;
  double total = 0.0;
  for (int r = 0; r < n_parts; ++r)
    total += exp(static_cast<double>(parts.lse[r][row]) - static_cast<double>(shift));
  const double l = static_cast<double>(shift) + log(total);

  int64_t id;
  const float mx = entries_shift(t, row);
  // w = exp(x), x = t / T - mx: sums of w and of w x
  double w_sum = 0.0, wx_sum = 0.0;
  for (int e = lane; e < t.k; e += 64) {
    const float v = entry(t, row, e, id), x = v - mx;
    const float w = v == neg_inf() ? 0.f : expf(x);
    w_sum += static_cast<double>(w);
    if (w != 0.f) wx_sum += static_cast<double>(w) * static_cast<double>(x);
  }
  w_sum = wave_sum(w_sum);
  wx_sum = wave_sum(wx_sum);
  if (lane != 0) return;
  double out = 0.0;
  if (w_sum != 0.0) {
    // given log-sum-exp: p = w; else p = w / sum w, log p = x - log(sum w)
    if (t.lse != nullptr) out = wx_sum - dot + w_sum * l;
    else out = wx_sum / w_sum - log(w_sum) - dot + l;
  }
  loss[row] = static_cast<float>(out);
  lse[row] = static_cast<float>(l);
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
constexpr int kHashBits = 8192;
constexpr int64_t kGradFill = 32768;  // workgroups wanted
constexpr int64_t kGradCols = 4096;   // columns of each, at least
constexpr int64_t kGradStream = int64_t(128) << 20;

// One workgroup per slice of a row.  Ids that occur twice are found by a table
// of kHashBits bits, and only ids whose bit was set twice are looked for among
// the others.  Bound by HBM: 4096 bf16 rows of 37984 (622 MB) in 105 us, 5.9
// TB/s; 251 bf16 rows of 75968 (76 MB) in 16 us, 4.8 TB/s.  Non-temporal stores:
// written back in whole lines while the logits are still being read.
template <bool BF16, bool STREAM>
__global__ __launch_bounds__(kBlock) void distill_grad_rows(ShardArgs z, TeacherArgs t,
                                                           const float *__restrict__ lse,
                                                           const float *__restrict__ grad_loss,
                                                           char *out_base, int64_t out_ld_bytes) {
  typedef Row<BF16> R;
  constexpr int kEpv = R::kEpv, kUnroll = 4, kSize = BF16 ? 2 : 4;
  __shared__ float red[kWaves];
  __shared__ float sp[kMaxEntries];
  __shared__ int scol[kMaxEntries];
  __shared__ uint32_t seen[kHashBits / 32], twice[kHashBits / 32];
  const int64_t row = blockIdx.x / static_cast<unsigned>(z.slices);
  const int s = static_cast<int>(blockIdx.x - row * z.slices);
  const int tid = threadIdx.x;
  const int64_t c0 = s * z.slice;
  const int64_t n = c0 + z.slice < z.cols ? z.slice : z.cols - c0;
  const char *src = z.base + row * z.ld_bytes + c0 * kSize;
  char *dst = out_base + row * out_ld_bytes + c0 * kSize;
  const int64_t nv = n / kEpv;

  float p[kEntriesPerThread];
  int col[kEntriesPerThread];
  const float g = grad_loss[row] * t.inv_t;
  float mass = 0.f;
  if (grad_loss[row] != 0.f) mass = teacher_row(t, row, z.vocab_start + c0, n, p, col, red);
  if (grad_loss[row] == 0.f || mass == 0.f) {
    for (int64_t i = tid; i < nv; i += kBlock)
      reinterpret_cast<typename R::loose *>(dst)[i] = u32x4(0);
    for (int64_t i = nv * kEpv + tid; i < n; i += kBlock) store_one<BF16>(dst, i, 0.f);
    return;
  }

  // the entries' columns: logits before they may be overwritten, and the
  // probabilities of ids that occur more than once added at the first of them
  for (int i = tid; i < kHashBits / 32; i += kBlock) seen[i] = 0, twice[i] = 0;
#pragma unroll
  for (int i = 0; i < kEntriesPerThread; ++i) {
    sp[tid + kBlock * i] = p[i];
    scol[tid + kBlock * i] = col[i];
  }
  __syncthreads();
  float zk[kEntriesPerThread];
#pragma unroll
  for (int i = 0; i < kEntriesPerThread; ++i) {
    zk[i] = 0.f;
    if (col[i] >= 0) {
      zk[i] = load_one<BF16>(src, col[i]);
      const uint32_t h = static_cast<uint32_t>(col[i]) % kHashBits, bit = 1u << (h & 31);
      if (atomicOr(&seen[h / 32], bit) & bit) atomicOr(&twice[h / 32], bit);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEntriesPerThread; ++i) {
    if (col[i] >= 0) {
      const uint32_t h = static_cast<uint32_t>(col[i]) % kHashBits;
      if ((twice[h / 32] >> (h & 31)) & 1u) {
        const int e = tid + kBlock * i;
        bool first = true;
        for (int j = 0; j < e; ++j) first = first && scol[j] != col[i];
        float sum = 0.f;
        for (int j = e; j < t.k; ++j) sum += scol[j] == col[i] ? sp[j] : 0.f;
        p[i] = sum;
        if (!first) col[i] = -1;
      }
    }
  }

  // exp(z / T - lse) = 2^((z - off) c): as in the statistics, the difference
  // comes first (a finite lse times T stays finite)
  const float c = t.to_log2;
  float off = lse[row] * t.temperature;
  if (__builtin_isinf(off) && !__builtin_isinf(lse[row])) off = copysignf(kMostFloat, off);
  const float a = g * mass;
  for (int64_t i = tid; i < nv; i += kBlock * kUnroll) {
    u32x4 r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t j = i + u * kBlock;
      r[u] = u32x4(0);
      const typename R::loose *from = reinterpret_cast<const typename R::loose *>(src) + j;
      if (j < nv) r[u] = STREAM ? __builtin_nontemporal_load(from) : *from;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t j = i + u * kBlock;
      float v[kEpv];
      Vec<BF16, kEpv>::widen(r[u], v);
#pragma unroll
      for (int e = 0; e < kEpv; ++e) v[e] = a * exp2_fast((v[e] - off) * c);
      if (j < nv)
        __builtin_nontemporal_store(Vec<BF16, kEpv>::narrow(v),
                                    reinterpret_cast<typename R::loose *>(dst) + j);
    }
  }
  for (int64_t i = nv * kEpv + tid; i < n; i += kBlock)
    store_one<BF16>(dst, i, a * exp2_fast((load_one<BF16>(src, i) - off) * c));
  __syncthreads();  // the dense pass's stores come before the entries'
#pragma unroll
  for (int i = 0; i < kEntriesPerThread; ++i)
    if (col[i] >= 0)
      store_one<BF16>(dst, col[i], g * (mass * exp2_fast((zk[i] - off) * c) - p[i]));
}

TeacherArgs args_of(const Teacher &t) {
  return TeacherArgs{
      t.ids, t.logits, t.lse, t.itype, t.dtype, t.k, t.vocab, t.temperature, 1.f / t.temperature,
      static_cast<float>(1.4426950408889634 / static_cast<double>(t.temperature))};
}

ShardArgs args_of(const LogitsShard &z, int64_t slice) {
  return ShardArgs{static_cast<const char *>(z.base), z.ld * (z.dtype == 1 ? 2 : 4), z.cols,
                   z.vocab_start, static_cast<int>((z.cols + slice - 1) / slice), slice};
}

int64_t pair_cols(int dtype) { return kPairVecs * 64 * (dtype == 1 ? 8 : 4); }

}  // namespace

int64_t distill_pairs_per_row(int64_t cols, int dtype) {
  return (cols + pair_cols(dtype) - 1) / pair_cols(dtype);
}

int launch_distill_shard(const LogitsShard &z, const Teacher &t, float *shard_lse,
                         float *shard_dot, float *pairs, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // clear a stale error so the status returned is this launch's
  const ShardArgs a = args_of(z, pair_cols(z.dtype));
  const TeacherArgs ta = args_of(t);
  Pair *pr = reinterpret_cast<Pair *>(pairs);
  // A workgroup per row, unless a few long rows would leave the chip idle; a bf16
  // slice has twice the columns of an fp32 one.  us with a workgroup per row / with
  // pairs in memory, in a graph, fp32: 8 rows of 38 slices 6.4 / 7.1, of 149 slices
  // 16.4 / 8.7; 64 rows of 75 slices 10.8 / 11.2, of 149 slices 18.4 / 14.7; 255
  // rows of 149 slices 28.9 / 33.1; 4096 rows of 4 slices 16.7 / 20.6.  bf16: 8 rows
  // of 24 slices 6.8 / 7.3, of 75 slices 13.4 / 8.5; 128 rows of 44 slices 12.0 /
  // 12.7, of 75 slices 18.3 / 15.8; 255 rows of 75 slices 21.3 / 22.1.  (Of 240
  // points of 1 to 255 rows and 24 to 149 slices the rule takes the slower side by
  // more than a tenth at one, 11%.)  Waves have two slices each where they can:
  // 4096 bf16 rows of 8 slices 30.8 with 4 waves, 34.6 with 8.
  const int64_t few = z.dtype == 1 ? 26 + z.m / 4 : 44 + z.m / 2;
  if (shard_lse && (z.m >= kDistillWholeRows || a.slices <= few)) {
    const int waves = std::min((a.slices + 1) / 2, kRowWaves);
    const dim3 grid(static_cast<unsigned>(z.m)), block(64 * (waves + 1));
    if (z.dtype == 1)
      hipLaunchKernelGGL((distill_whole_rows<true>), grid, block, 0, st, a, ta, waves, shard_lse,
                         shard_dot);
    else
      hipLaunchKernelGGL((distill_whole_rows<false>), grid, block, 0, st, a, ta, waves, shard_lse,
                         shard_dot);
    return static_cast<int>(hipGetLastError());
  }
  if (shard_lse) {
    const unsigned gx = static_cast<unsigned>((a.slices + kWaves - 1) / kWaves);
    const dim3 grid(gx, static_cast<unsigned>(z.m));
    if (z.dtype == 1)
      hipLaunchKernelGGL((distill_pairs<true>), grid, dim3(kBlock), 0, st, a, ta.to_log2, pr);
    else
      hipLaunchKernelGGL((distill_pairs<false>), grid, dim3(kBlock), 0, st, a, ta.to_log2, pr);
  }
  const dim3 rows(static_cast<unsigned>((z.m + kWaves - 1) / kWaves));
  if (z.dtype == 1)
    hipLaunchKernelGGL((distill_rows<true>), rows, dim3(kBlock), 0, st, a, ta, z.m, pr, shard_lse,
                       shard_dot);
  else
    hipLaunchKernelGGL((distill_rows<false>), rows, dim3(kBlock), 0, st, a, ta, z.m, pr, shard_lse,
                       shard_dot);
  return static_cast<int>(hipGetLastError());
}

int launch_distill_loss(const float *const *shard_lse, const float *const *shard_dot, int n_parts,
                        int64_t m, const Teacher &t, float *loss, float *lse, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  Parts parts{};
  for (int r = 0; r < n_parts; ++r) parts.lse[r] = shard_lse[r], parts.dot[r] = shard_dot[r];
  hipLaunchKernelGGL(distill_loss_rows, dim3(static_cast<unsigned>((m + kWaves - 1) / kWaves)),
                     dim3(kBlock), 0, st, parts, n_parts, m, args_of(t), loss, lse);
  return static_cast<int>(hipGetLastError());
}

int launch_distill_grad(const LogitsShard &z, const Teacher &t, const float *lse,
                        const float *grad_loss, void *grad_base, int64_t ld_grad, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  // one workgroup per row, or more where there are few rows, for at least
  // kGradCols columns each
  const int64_t want =
      std::max<int64_t>(1, std::min((kGradFill + z.m - 1) / z.m, z.cols / kGradCols));
  const ShardArgs a = args_of(z, ((z.cols + want - 1) / want + 7) / 8 * 8);
  const dim3 grid(static_cast<unsigned>(z.m * a.slices));
  const int64_t ld_bytes = ld_grad * (z.dtype == 1 ? 2 : 4);
  char *out = static_cast<char *>(grad_base);
  // logits that the last-level cache cannot hold are read past it, which leaves
  // room for what is still to be written: [1024, 151936] in two shards 177 us a
  // step against 189, [4096, 37984] 105 against 108; 38 MB ([251, 75968]) are
  // still there from their producer, and read past it 17.0 instead of 15.8 us
  const bool streamed = z.m * z.cols * (z.dtype == 1 ? 2 : 4) > kGradStream;
#define VPE_GRAD(BF16, STREAM)                                                               \
  hipLaunchKernelGGL((distill_grad_rows<BF16, STREAM>), grid, dim3(kBlock), 0, st, a,         \
                     args_of(t), lse, grad_loss, out, ld_bytes)
  if (z.dtype == 1 && streamed) VPE_GRAD(true, true);
  else if (z.dtype == 1) VPE_GRAD(true, false);
  else if (streamed) VPE_GRAD(false, true);
  else VPE_GRAD(false, false);
#undef VPE_GRAD
  return static_cast<int>(hipGetLastError());
}

}  // namespace vpe
