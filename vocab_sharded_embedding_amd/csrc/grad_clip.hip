// Global gradient norm over many tensors, and clipping, for gfx950.
//
// Both read every element once and are bound by HBM (the clip also writes every
// one).  A launch takes a table of up to kClipTable tensors in its arguments, so
// that nothing is copied to the device and a captured launch keeps it; its
// workgroups are pieces of `chunk` elements of one tensor each.  A piece's sum of
// squares is one double, and one workgroup adds all pieces in order: the same
// bits every time, whatever the order the pieces ran in.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vpe_device.h"
#include "vpe_loss_launch.h"

namespace vpe {
namespace {

constexpr int kThreads = 256;

// Up to N tensors of a launch: kClipTable, or a few (the arguments of a launch are
// copied: 2 KB of them cost a small call about 1 us).
constexpr int kFewTensors = 8;
template <int N>
struct Table {
  const void *g[N];
  int64_t count[N];
  int32_t first[N + 1];  // first workgroup of a tensor
  uint32_t bf16[(N + 31) / 32];
  int64_t chunk;
  int n;
};

template <int N>
struct Outputs {
  void *out[N];
};

// The tensor that workgroup b works on.
template <int N>
__device__ __forceinline__ int tensor_of(const Table<N> &t, int b) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Calls each(i, v) for the vectors of 16 bytes of elements [begin, end) that this
// thread takes, v the one that begins at element i; kAhead loads are in flight.
constexpr int kAhead = 4;
template <bool BF16, class Each>
__device__ __forceinline__ void vectors(const void *g, int64_t begin, int64_t end, Each each) {
  constexpr int kEpv = BF16 ? 8 : 4, kRow = kThreads * kEpv;
  int64_t i = begin + threadIdx.x * kEpv;
  for (; i + (kAhead - 1) * kRow + kEpv <= end; i += kAhead * kRow) {
    float v[kAhead][kEpv];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) dev::load_vec<BF16, kEpv>(g, i + k * kRow, end, v[k]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) each(i + k * kRow, v[k]);
  }
  for (; i < end; i += kRow) {
    float v[kEpv];
    dev::load_vec<BF16, kEpv>(g, i, end, v);
    each(i, v);
  }
}

// Squares and their sums in fp64: neither the square of a large fp32 gradient
// nor that of a small one leaves its range, and no bits are lost over 10^10 of
// them.  Four sums per thread keep the additions apart.
template <bool BF16>
__device__ __forceinline__ double squares(const void *g, int64_t begin, int64_t end) {
  constexpr int kEpv = BF16 ? 8 : 4;
  double s[4] = {0., 0., 0., 0.};
  vectors<BF16>(g, begin, end, [&](int64_t, const float (&v)[kEpv]) {
#pragma unroll
    for (int e = 0; e < kEpv; ++e) s[e & 3] = fma(double(v[e]), double(v[e]), s[e & 3]);
  });
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// Sum over the workgroup, on thread 0.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double part[16];
  v = dev::wave_sum(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.;
  if (threadIdx.x == 0)
    for (unsigned w = 0; w < blockDim.x / 64; ++w) s += part[w];
  return s;
}

// (310 tensors, 600 million elements, a third fp32, on two ranks: 300 us, 5.3 TB/s)
template <int N>
__global__ __launch_bounds__(kThreads) void sumsq_pieces(Table<N> t, double *__restrict__ partial) {
  const int at = tensor_of(t, blockIdx.x);
  const int64_t begin = (blockIdx.x - t.first[at]) * t.chunk;
  const int64_t end = begin + t.chunk < t.count[at] ? begin + t.chunk : t.count[at];
  const bool bf16 = (t.bf16[at / 32] >> (at % 32)) & 1;
  const double s = block_sum(bf16 ? squares<true>(t.g[at], begin, end)
                                  : squares<false>(t.g[at], begin, end));
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(1024) void sumsq_join(const double *__restrict__ partial, int64_t n,
                                                   double *__restrict__ sumsq) {
  double s = 0.;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += partial[i];
  s = block_sum(s);
  if (threadIdx.x == 0) *sumsq = s;
}

struct Norms {
  const double *sumsq[64];
  int n;
  double max_norm;
};

__device__ __forceinline__ double global_norm(const Norms &p) {
  double s = 0.;
  for (int r = 0; r < p.n; ++r) s += *p.sumsq[r];
  return sqrt(s);
}

template <bool BF16>
__device__ __forceinline__ void scale_piece(const void *g, void *out, int64_t begin, int64_t end,
                                            float f) {
  constexpr int kEpv = BF16 ? 8 : 4;
  vectors<BF16>(g, begin, end, [&](int64_t i, float (&v)[kEpv]) {
#pragma unroll
    for (int e = 0; e < kEpv; ++e) v[e] *= f;
    dev::store_vec_nt<BF16, kEpv>(out, i, end, v);
  });
}

// The pieces last to first: what the sum of squares read last may still be in the
// memory-side cache.  (The same tensors: 660 us, 4.9 TB/s of reads and writes; with
// the sums 967 us, 1062 first to last and with fewer loads in flight.)
template <int N>
__global__ __launch_bounds__(kThreads) void clip_pieces(Table<N> t, Outputs<N> o, Norms p,
                                                        float *__restrict__ norm) {
  const double whole = global_norm(p);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(whole);
  if (t.n == 0) return;
  const int block = t.first[t.n] - 1 - static_cast<int>(blockIdx.x);
  const double ratio = p.max_norm / (whole + 1e-6);
  const float f =
      ratio < 1. ? static_cast<float>(ratio) : (ratio != ratio ? __builtin_nanf("") : 1.f);
  const int at = tensor_of(t, block);
  const void *g = t.g[at];
  // (times 1 in place: nothing to write)
  if (f == 1.f && g == o.out[at]) return;
  const int64_t begin = (block - t.first[at]) * t.chunk;
  const int64_t end = begin + t.chunk < t.count[at] ? begin + t.chunk : t.count[at];
  if ((t.bf16[at / 32] >> (at % 32)) & 1) scale_piece<true>(g, o.out[at], begin, end, f);
  else scale_piece<false>(g, o.out[at], begin, end, f);
}

// Calls launch(table, outputs, workgroups) for the tensors that have elements, N at
// a time; `last_first`: from the last table to the first.
template <int N, class F>
void each_table(const void *const *tensors, const int64_t *counts, const int32_t *dtypes, int n,
                int64_t total, void *const *out, bool last_first, F launch) {
  int end = n;
  for (int at = 0; last_first ? end > 0 : at < n;) {
    // the tensors of this table: [lo, hi)
    int lo = at, hi = at, found = 0;
    if (last_first) {
      for (lo = hi = end; lo > 0 && found < N; --lo) found += counts[lo - 1] != 0;
      end = lo;
    } else {
      for (; hi < n && found < N; ++hi) found += counts[hi] != 0;
      at = hi;
    }
    if (found == 0) continue;
    Table<N> t{};
    Outputs<N> o{};
    t.chunk = clip_chunk(total);
    int64_t groups = 0;
    for (int i = lo; i < hi; ++i) {
      if (counts[i] == 0) continue;
      t.g[t.n] = tensors[i];
      if (out != nullptr) o.out[t.n] = out[i];
      t.count[t.n] = counts[i];
      t.first[t.n] = static_cast<int32_t>(groups);
      if (dtypes[i] == 1) t.bf16[t.n / 32] |= uint32_t(1) << (t.n % 32);
      groups += (counts[i] + t.chunk - 1) / t.chunk;
      ++t.n;
    }
    t.first[t.n] = static_cast<int32_t>(groups);
    launch(t, o, static_cast<unsigned>(groups));
  }
}

template <int N>
int run_sumsq(const void *const *tensors, const int64_t *counts, const int32_t *dtypes, int n,
              int64_t total, double *sumsq, double *partial, hipStream_t st) {
  int64_t pieces = 0;
  each_table<N>(tensors, counts, dtypes, n, total, nullptr, false,
                [&](const Table<N> &t, const Outputs<N> &, unsigned groups) {
                  hipLaunchKernelGGL(sumsq_pieces<N>, dim3(groups), dim3(kThreads), 0, st, t,
                                     partial + pieces);
                  pieces += groups;
                });
  hipLaunchKernelGGL(sumsq_join, dim3(1), dim3(1024), 0, st, partial, pieces, sumsq);
  return static_cast<int>(hipGetLastError());
}

template <int N>
int run_clip(const void *const *tensors, const int64_t *counts, const int32_t *dtypes, int n,
             int64_t total, void *const *out, const Norms &p, float *norm, hipStream_t st) {
  bool first = true;
  each_table<N>(tensors, counts, dtypes, n, total, out, true,
                [&](const Table<N> &t, const Outputs<N> &o, unsigned groups) {
                  hipLaunchKernelGGL(clip_pieces<N>, dim3(groups), dim3(kThreads), 0, st, t, o, p,
                                     first ? norm : nullptr);
                  first = false;
                });
  if (first)
    hipLaunchKernelGGL(clip_pieces<N>, dim3(1), dim3(kThreads), 0, st, Table<N>{}, Outputs<N>{}, p,
                       norm);
  return static_cast<int>(hipGetLastError());
}

}  // namespace

int launch_grad_sumsq(const void *const *tensors, const int64_t *counts, const int32_t *dtypes,
                      int n, int64_t total, double *sumsq, double *partial, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();  // clear a stale error so the status below is this launch's
  return n <= kFewTensors
             ? run_sumsq<kFewTensors>(tensors, counts, dtypes, n, total, sumsq, partial, st)
             : run_sumsq<kClipTable>(tensors, counts, dtypes, n, total, sumsq, partial, st);
}

int launch_grad_clip(const void *const *tensors, const int64_t *counts, const int32_t *dtypes,
                     int n, int64_t total, void *const *out, const double *const *sumsq,
                     int n_parts, double max_norm, float *norm, void *stream) {
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  Norms p{};
  for (int r = 0; r < n_parts; ++r) p.sumsq[r] = sumsq[r];
  p.n = n_parts, p.max_norm = max_norm;
  return n <= kFewTensors
             ? run_clip<kFewTensors>(tensors, counts, dtypes, n, total, out, p, norm, st)
             : run_clip<kClipTable>(tensors, counts, dtypes, n, total, out, p, norm, st);
}

}  // namespace vpe
