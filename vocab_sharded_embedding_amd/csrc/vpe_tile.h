// Tile products for the matrix cores, shared by the cross entropy's kernels and
// the LM head's backward: one workgroup's tile of
//
//   C[n, m] = sum_k A[n, k] B[m, k]
//
// where either operand lies in memory with k contiguous ("rows": A[n, k] at n ld
// + k, as hidden rows and table rows are for the logits) or with n or m
// contiguous ("columns": at k ld + n, as a table is for the gradient of the
// hidden rows, which sums over its rows).  Nothing is ever transposed in memory.
//
// Both operands are staged through NS stages of LDS by buffer loads that write LDS
// directly, BK values of k each, and multiplied by v_mfma_f32_32x32x16_bf16 or
// v_mfma_f32_32x32x2_f32.  A lane's fragment is consecutive values of k of one n or
// m: an operand in rows gives it in one 16-byte LDS read; one in columns, of bf16 in
// two transposing 8-byte reads (ds_read_b64_tr_b16: 16 lanes read 4 values of k x 16
// columns and get 4 values of k of one column each), of fp32 in four 4-byte reads.
// Rows have to begin at 16 bytes and hold whole 16 bytes.  Other rows pass through
// registers (`run_loose`).
//
// 256 x 256 over 8 waves, BK 64, two stages, bf16: 8192 x 8192 x 1024 in rows 104-107 us,
// 1.29-1.32 PFLOP/s; 8192^3 in rows 920-935 us, in columns 877-926 us, 1.18-1.25
// PFLOP/s, no bank conflicts, matrix cores busy 83% at the 1.4 GHz that the power allows.
// Slower there: 256 x 128 and 128 x 128 tiles, stages of 32 values of k (3 to 5 of them),
// v_mfma_f32_16x16x32_bf16 (the registers of 8 waves run out in columns: 955-1300 us).
#ifndef VPE_TILE_H
#define VPE_TILE_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "vpe_bounds.h"

namespace vpe {
namespace tile {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Most stages of a tile.
constexpr int kStages = 3;

// Tile of BN x BM of C over WN x WM waves, k in steps of BK through NS stages.
// Each wave owns FN x FM fragments of 32 x 32: fragment (i, j) of a lane holds,
// in register r, n = 32 i + 8 (r / 4) + 4 (lane / 32) + r % 4 and m = 32 j + lane % 32.
template <int BN_, int BM_, int WN_, int WM_, int BK_, int NS_>
struct Shape {
  static constexpr int BN = BN_, BM = BM_, WN = WN_, WM = WM_, BK = BK_, NS = NS_;
  static constexpr int NW = WN * WM, NT = NW * 64;
  static constexpr int TN = BN / WN, TM = BM / WM;
  static constexpr int FN = TN / 32, FM = TM / 32;
  static_assert(FN * 32 == TN && FM * 32 == TM, "a wave's tile is whole fragments");
  static_assert(NS >= 2 && NS <= kStages, "two or three stages");
};

#if defined(__HIP_DEVICE_COMPILE__)

// dword 3 of a gfx9 buffer descriptor: 32-bit data format, raw access
constexpr int kRawBuffer = 0x00020000;

constexpr int wait_vm(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4) | (0xF << 8); }

__device__ __forceinline__ int wave_id() {
  return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 __attribute__((aligned(2))) loose_u32x4;

// The first `bytes` of 16 at p, elements of E bytes, zeros behind them.
template <int E>
__device__ __forceinline__ u32x4 some_of(const char *p, int bytes) {
  u32x4 v = u32x4(0u);
#pragma unroll
  for (int i = 0; i < 16 / E; ++i)
    if ((i + 1) * E <= bytes) {
      if constexpr (E == 2)
        v[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << (i % 2 * 16);
      else
        v[i] = reinterpret_cast<const uint32_t *>(p)[i];
    }
  return v;
}

// A lane's fragment: bf16, 8 consecutive values of k of one n or m (a round of
// MFMAs takes 16 values of k, lanes 0-31 the first 8); fp32, 4 of them (8 values a
// round, in 4 MFMAs that each take one from either half of the lanes).
template <int E>
struct Frag {
  typedef bf16x8 type;
};
template <>
struct Frag<4> {
  typedef f32x4 type;
};

// One operand's side of the staging, elements of E bytes.  `COLS`: it lies in
// columns.  Row strides are at most 2^22 elements: offsets inside a tile fit an int.
template <bool COLS, int SIDE, int BK, int NW, int E>
struct Stage;

// In rows: LDS row n holds BK values as pieces of 16 bytes, piece p at slot
// p ^ f(n).  The LDS serves a 16-byte read 16 lanes at a time over 64 banks (256
// bytes), and those lanes read one piece of 16 consecutive rows: f changes with
// every 256 bytes of rows, so that they meet 16 different groups of 4 banks
// (counted bank conflicts: half of the LDS's cycles with f changing every 128
// bytes).
template <int SIDE, int BK, int NW, int E>
struct Stage<false, SIDE, BK, NW, E> {
  static constexpr int kRowBytes = BK * E, kBytes = SIDE * kRowBytes;
  static constexpr int kPieces = kRowBytes / 16, kRowsPerLoad = 64 / kPieces;
  static constexpr int kLoads = SIDE / kRowsPerLoad / NW;
  static constexpr int kReads = 1;  // of the LDS, per fragment
  static_assert(kLoads * kRowsPerLoad * NW == SIDE, "whole loads per wave");
  typedef typename Frag<E>::type frag_t;
  const char *base;
  int left;  // bytes from base to the operand's end (of SIDE rows: below 2^31)
  int voff[kLoads];
  int piece_at[2];  // this lane's piece, as bytes into a row's step, by load
  int rd[kRowBytes / 32];
  int k_left;  // bytes of a row

  static __device__ __forceinline__ int swizzle(int row) {
    constexpr int kGroup = kRowBytes >= 256 ? 1 : 256 / kRowBytes;
    return (row / kGroup) & (kPieces - 1);
  }
  // `rows` rows from p on exist, of k_limit values (whole 16 bytes) each.
  __device__ __forceinline__ void init(const void *p, int64_t ld, int64_t rows, int64_t k_limit,
                                       int side_base) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    base = static_cast<const char *>(p);
    left = static_cast<int>(rows > 0 ? (((rows < SIDE ? rows : SIDE) - 1) * ld + k_limit) * E : 0);
    k_left = static_cast<int>(k_limit * E);
    const int lrow = lane / kPieces, slot = lane % kPieces;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int row = (q * NW + wave) * kRowsPerLoad + lrow;
      const int piece = slot ^ swizzle(row);
      voff[q] = row < rows ? static_cast<int>(row * ld * E) + piece * 16 : kLoadMask;
    }
    // (two loads cover whole periods of f)
    piece_at[0] = (slot ^ swizzle(wave * kRowsPerLoad + lrow)) * 16;
    piece_at[1] = (slot ^ swizzle((NW + wave) * kRowsPerLoad + lrow)) * 16;
    static_assert(2 * NW * kRowsPerLoad % 16 == 0, "loads two apart take one piece");
    const int row = side_base + (lane & 31);
#pragma unroll
    for (int ks = 0; ks < kRowBytes / 32; ++ks)
      rd[ks] = row * kRowBytes + (((ks * 2 + (lane >> 5)) ^ swizzle(row)) << 4);
  }
  // This wave's q-th load of the next BK values of k into the stage at `dst`.
  __device__ __forceinline__ void load(char *dst, int q) const {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(base), 0, left > 0 ? left : 0, kRawBuffer);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (__attribute__((address_space(3))) void *)(dst + (q * NW + wave_id()) * 1024), 16,
        piece_at[q & 1] < k_left ? voff[q] : kLoadMask, 0, 0, 0);
  }
  __device__ __forceinline__ void advance() {
    base += kRowBytes;
    left -= kRowBytes;
    k_left -= kRowBytes;
  }
  // Loose rows.  Steps that hold BK values of every row; rows that do not exist give
  // the first one's values there, which reach no result.
  __device__ __forceinline__ int whole_steps() const { return k_left / kRowBytes; }
  template <bool WHOLE>
  __device__ __forceinline__ u32x4 fetch(int q) const {
    const bool row = voff[q] != kLoadMask;
    if constexpr (WHOLE)
      return *reinterpret_cast<const loose_u32x4 *>(base + (row ? voff[q] : 0));
    const int bytes = k_left - piece_at[q & 1];
    if (!row || bytes <= 0) return u32x4(0u);
    return bytes >= 16 ? *reinterpret_cast<const loose_u32x4 *>(base + voff[q])
                       : some_of<E>(base + voff[q], bytes);
  }
  __device__ __forceinline__ frag_t frag(const char *src, int ks, int i) const {
    return *reinterpret_cast<const frag_t *>(src + rd[ks] + i * 32 * kRowBytes);
  }
};

// In columns: LDS row k holds SIDE values.
//  - bf16: as segments of 32 bytes, segment s at s ^ f(k), f(k) = r ^ 2 r ^ (bit 3
//    of k), r = k % 4.  A transposing read takes one segment of 4 values of k per
//    16 lanes: those 4 segments, and the 8 of 32 lanes, meet different banks.
//  - fp32: the halves of every 64 values change places where bit 2 of k is set, so
//    that the two halves of the lanes, 4 values of k apart, read different banks.
template <int SIDE, int BK, int NW, int E>
struct Stage<true, SIDE, BK, NW, E> {
  static constexpr int kRowBytes = SIDE * E, kBytes = BK * kRowBytes;
  static constexpr int kPieces = kRowBytes / 16, kRowsPerLoad = 64 / kPieces;
  static constexpr int kLoads = BK / kRowsPerLoad / NW;
  static constexpr int kReads = E == 2 ? 2 : 4;
  static_assert(kLoads * kRowsPerLoad * NW == BK && kRowBytes >= 256, "whole loads per wave");
  typedef typename Frag<E>::type frag_t;
  const char *base;
  int64_t left, step;
  int voff[kLoads];
  int rd[4];
  int k_rows, row_bytes;  // (loose rows) that exist, up to SIDE of a row

  static __device__ __forceinline__ int swizzle(int k) {
    return E == 2 ? ((k & 3) ^ ((k & 3) << 1) ^ ((k >> 3) & 1)) << 1 : ((k >> 2) & 1) << 3;
  }
  // Columns from p on, `cols` of them inside a row (which ends at whole 16 bytes);
  // k_limit rows exist.
  __device__ __forceinline__ void init(const void *p, int64_t ld, int64_t cols, int64_t k_limit,
                                       int side_base) {
    constexpr int kEpp = 16 / E;
    const int lane = threadIdx.x & 63, wave = wave_id();
    base = static_cast<const char *>(p);
    left = k_limit > 0 ? ((k_limit - 1) * ld + (cols + kEpp - 1) / kEpp * kEpp) * E : 0;
    step = ld * BK * E;
    k_rows = static_cast<int>(k_limit);
    row_bytes = static_cast<int>(cols < SIDE ? (cols > 0 ? cols : 0) : SIDE) * E;
    const int lrow = lane / kPieces, slot = lane % kPieces;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int k = (q * NW + wave) * kRowsPerLoad + lrow;
      // (16 bytes that begin at or past the row's last column are another row's,
      // or lie past the end: nothing reads them)
      voff[q] = static_cast<int>(k * ld * E) + (slot ^ swizzle(k)) * 16;
    }
    const int hi = lane >> 5;
    if constexpr (E == 2) {
      const int r = (lane & 15) >> 2, b = (lane >> 4) & 1;
      const int f = swizzle(r + 8 * hi) >> 1;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        rd[i] = (8 * hi + r) * kRowBytes + (((side_base / 16 + 2 * i + b) ^ f) << 5) +
                (lane & 3) * 8;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        rd[i] = 4 * hi * kRowBytes + ((((side_base / 32 + i) ^ hi) << 5) + (lane & 31)) * 4;
    }
  }
  __device__ __forceinline__ void load(char *dst, int q) const {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(base), 0,
        static_cast<int>(left > kLoadMask ? kLoadMask : (left > 0 ? left : 0)), kRawBuffer);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (__attribute__((address_space(3))) void *)(dst + (q * NW + wave_id()) * 1024), 16,
        voff[q], 0, 0, 0);
  }
  __device__ __forceinline__ void advance() {
    base += step;
    left -= step;
    k_rows -= BK;
  }
  __device__ __forceinline__ int whole_steps() const {
    return row_bytes == kRowBytes ? k_rows / BK : 0;
  }
  template <bool WHOLE>
  __device__ __forceinline__ u32x4 fetch(int q) const {
    if constexpr (WHOLE) return *reinterpret_cast<const loose_u32x4 *>(base + voff[q]);
    const int lane = threadIdx.x & 63;
    const int k = (q * NW + wave_id()) * kRowsPerLoad + lane / kPieces;
    const int bytes = row_bytes - ((lane % kPieces) ^ swizzle(k)) * 16;
    if (k >= k_rows || bytes <= 0) return u32x4(0u);
    return bytes >= 16 ? *reinterpret_cast<const loose_u32x4 *>(base + voff[q])
                       : some_of<E>(base + voff[q], bytes);
  }
  __device__ __forceinline__ frag_t frag(const char *src, int ks, int i) const {
    if constexpr (E == 2) {
      typedef __attribute__((address_space(3))) s16x4 lds_v;
      const char *p = src + rd[i & 3] + (i >> 2) * 256 + ks * 16 * kRowBytes;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v *)(p));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v *)(p + 4 * kRowBytes));
      return __builtin_bit_cast(bf16x8,
                                __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      f32x4 f;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        f[s] = *reinterpret_cast<const float *>(src + rd[i & 3] + (i >> 2) * 512 +
                                                (ks * 8 + s) * kRowBytes);
      return f;
    }
  }
};

// The stages are LDS arrays of their own, and every access names one: the
// compiler then sees that a read does not touch the stage that a load in flight
// fills, and waits for no load on its account (it puts a wait for all of them
// before every transposing read otherwise: 8192^3 in columns 1091 against 956 us).
template <class S, int E, bool NCOLS, bool MCOLS>
struct Product {
  typedef Stage<NCOLS, S::BN, S::BK, S::NW, E> StageN;
  typedef Stage<MCOLS, S::BM, S::BK, S::NW, E> StageM;
  typedef typename Frag<E>::type frag_t;
  static constexpr int kStageBytes = StageN::kBytes + StageM::kBytes;
  static constexpr int kLoads = StageN::kLoads + StageM::kLoads;
  static constexpr int KS = S::BK * E / 32;  // rounds per step
  static constexpr int kReads = S::FN * StageN::kReads + S::FM * StageM::kReads;
  static constexpr int kMfma = S::FN * S::FM * (E == 2 ? 1 : 4);
  static_assert(KS % 2 == 0, "fragments alternate between two sets of registers");
  static_assert((S::NS - 1) * kLoads <= 63, "outstanding loads fit the counter");
  // The loads of a step go out over kSpread rounds, from the one in which its
  // stage is free: the memory path takes one load of 64 x 16 bytes per 16 cycles
  // and CU, and a wave that finds its queue full issues no MFMA either.
  static constexpr int kSpread = KS < 3 ? KS : 3;
  static constexpr int kPart = (kLoads + kSpread - 1) / kSpread;

  StageN a;
  StageM b;
  frag_t fa[2][S::FN], fb[2][S::FM];
  // fp32, one fragment a wave: every other MFMA adds to a sum of its own, which
  // halves the chain of roundings.
  static constexpr bool kTwo = E == 4 && S::FN * S::FM == 1;
  f32x16 odd;

  __device__ __forceinline__ void load(char *stage, int q) {
    if (q < StageN::kLoads) a.load(stage, q);
    else if (q < kLoads) b.load(stage + StageN::kBytes, q - StageN::kLoads);
  }
  __device__ __forceinline__ void load_parts(char *stage, int from, int to) {
#pragma unroll
    for (int q = from * kPart; q < to * kPart; ++q) load(stage, q);
    if (to == kSpread) a.advance(), b.advance();
  }
  // The fragments of round ks of a stage, and (part >= 0) a part of the loads into
  // stage `to` in turn with them.
  __device__ __forceinline__ void frags(int set, const char *stage, int ks, int part, char *to) {
    constexpr int kF = S::FN + S::FM;
#pragma unroll
    for (int f = 0; f < (kF > kPart ? kF : kPart); ++f) {
      if (f < S::FM) fb[set][f] = b.frag(stage + StageN::kBytes, ks, f);
      else if (f < kF) fa[set][f - S::FM] = a.frag(stage, ks, f - S::FM);
      if (part >= 0 && f < kPart) load(to, part * kPart + f);
    }
    if (part == kSpread - 1) a.advance(), b.advance();
  }
  __device__ __forceinline__ void mfma(int set, f32x16 (&acc)[S::FN][S::FM]) {
#pragma unroll
    for (int v = 0; v < (E == 2 ? 1 : 4); ++v)
#pragma unroll
      for (int i = 0; i < S::FN; ++i)
#pragma unroll
        for (int j = 0; j < S::FM; ++j) {
          if constexpr (E == 2)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[set][i], fb[set][j], acc[i][j],
                                                                0, 0, 0);
          else if (kTwo && v % 2 == 1)
            odd = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[set][i][v], fb[set][j][v], odd, 0, 0, 0);
          else
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[set][i][v], fb[set][j][v],
                                                             acc[i][j], 0, 0, 0);
        }
  }
  // Order of a round: the next round's reads and `loads` loads between the MFMAs;
  // nothing crosses a round's end.  (Left to the compiler, reads sink to just
  // before their use.)
  static __device__ __forceinline__ void schedule(int loads) {
    constexpr int kPer = (kReads + kMfma - 1) / kMfma;
    constexpr int kLoad = (kPart + kMfma - 1) / kMfma;
#pragma unroll
    for (int g = 0; g < kMfma; ++g) {
      if (g * kPer < kReads) __builtin_amdgcn_sched_group_barrier(0x100, kPer, 0);   // LDS reads
      if (g * kLoad < loads) __builtin_amdgcn_sched_group_barrier(0x020, kLoad, 0);  // loads
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                             // MFMAs
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  // A step whose later steps have loads to send: `prev` takes the rest of step
  // kt + NS - 1, `cur` the first of step kt + NS.
  __device__ __forceinline__ void step(char *cur, const char *next, char *prev,
                                       f32x16 (&acc)[S::FN][S::FM]) {
#pragma unroll
    for (int ks = 0; ks + 1 < KS; ++ks) {
      const bool loads = ks + 1 < kSpread;
      frags((ks + 1) & 1, cur, ks + 1, loads ? ks + 1 : -1, prev);
      mfma(ks & 1, acc);
      schedule(loads ? kPart : 0);
    }
    // step kt + 1 has landed for this wave, and this wave has read step kt; after
    // the barrier both hold for all waves
    __builtin_amdgcn_s_waitcnt(wait_vm((S::NS - 2) * kLoads));
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    frags(0, next, 0, 0, cur);
    mfma((KS - 1) & 1, acc);
    schedule(kPart);
  }
  // Loose rows: 16 bytes per lane and load, from any element on, pass through
  // registers into the places that `load` fills.  A step's loads begin three steps
  // before it, through two sets of registers, and are written a step before it.
  template <class St>
  static __device__ __forceinline__ void fetch(St &o, u32x4 (&v)[St::kLoads], bool whole) {
    if (whole) {
#pragma unroll
      for (int q = 0; q < St::kLoads; ++q) v[q] = o.template fetch<true>(q);
    } else {
#pragma unroll
      for (int q = 0; q < St::kLoads; ++q) v[q] = o.template fetch<false>(q);
    }
    o.advance();
  }
  template <int N>
  static __device__ __forceinline__ void put(char *to, const u32x4 (&v)[N]) {
    const int at = wave_id() * 1024 + (threadIdx.x & 63) * 16;
#pragma unroll
    for (int q = 0; q < N; ++q) *reinterpret_cast<u32x4 *>(to + q * S::NW * 1024 + at) = v[q];
  }
  __device__ __forceinline__ void run_loose(int nk, char *const (&st)[kStages],
                                            f32x16 (&acc)[S::FN][S::FM]) {
    if (nk <= 0) return;
    if constexpr (kTwo) odd = f32x16(0.f);
    const int whole_a = a.whole_steps(), whole_b = b.whole_steps();
    u32x4 va[2][StageN::kLoads], vb[2][StageM::kLoads];
    fetch(a, va[0], whole_a > 0), fetch(b, vb[0], whole_b > 0);
    put(st[0], va[0]), put(st[0] + StageN::kBytes, vb[0]);
    if (nk > 1) fetch(a, va[1], whole_a > 1), fetch(b, vb[1], whole_b > 1);
    if (nk > 2) fetch(a, va[0], whole_a > 2), fetch(b, vb[0], whole_b > 2);
    __syncthreads();
    for (int kt = 0; kt < nk; kt += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (kt + u >= nk) break;
        if (kt + u + 1 < nk) put(st[1 - u], va[1 - u]), put(st[1 - u] + StageN::kBytes, vb[1 - u]);
        if (kt + u + 3 < nk)
          fetch(a, va[1 - u], whole_a > kt + u + 3), fetch(b, vb[1 - u], whole_b > kt + u + 3);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          frags(ks & 1, st[u], ks, -1, nullptr);
          mfma(ks & 1, acc);
        }
        __syncthreads();
      }
    }
    if constexpr (kTwo) acc[0][0] += odd;
  }
  // acc += the product over nk steps, through the stages st (NS of them).  A wave
  // reads each fragment one round of MFMAs ahead; the loads of a step begin NS - 1
  // steps before it.  Ends with every load landed.
  __device__ __forceinline__ void run(int nk, char *const (&st)[kStages],
                                      f32x16 (&acc)[S::FN][S::FM]) {
    if (nk <= 0) return;
    start(nk, st);
    if constexpr (kTwo) odd = f32x16(0.f);
    go_on(nk, st, acc);
    if constexpr (kTwo) acc[0][0] += odd;
  }
  // Its first loads, of the first NS steps (few steps: every stage at once, nothing
  // spread),
  __device__ __forceinline__ void start(int nk, char *const (&st)[kStages]) {
#pragma unroll
    for (int s = 0; s < S::NS - 1; ++s)
      if (s < nk) load_parts(st[s], 0, kSpread);
    if (nk >= 2 * S::NS) load_parts(st[S::NS - 1], 0, 1);
    else if (S::NS - 1 < nk) load_parts(st[S::NS - 1], 0, kSpread);
  }
  // and the rest.
  __device__ __forceinline__ void go_on(int nk, char *const (&st)[kStages],
                                        f32x16 (&acc)[S::FN][S::FM]) {
    bool rest = nk >= 2 * S::NS;
    if (rest) __builtin_amdgcn_s_waitcnt(wait_vm((S::NS - 2) * kLoads + kPart));
    else if (S::NS - 1 < nk) __builtin_amdgcn_s_waitcnt(wait_vm((S::NS - 1) * kLoads));
    else __builtin_amdgcn_s_waitcnt(wait_vm(0));
    asm volatile("s_barrier" ::: "memory");
    frags(0, st[0], 0, -1, nullptr);
    int kt = 0;
    for (; kt + 2 * S::NS - 1 < nk; kt += S::NS) {
#pragma unroll
      for (int u = 0; u < S::NS; ++u)
        step(st[u], st[(u + 1) % S::NS], st[(u + S::NS - 1) % S::NS], acc);
    }
    // the last steps, at most 2 NS - 1 of them
    char *cur = st[0], *next = st[1], *prev = st[S::NS - 1];
    for (; kt < nk; ++kt) {
      if (kSpread > 1 && rest) load_parts(prev, 1, kSpread);
      rest = false;
#pragma unroll
      for (int ks = 0; ks + 1 < KS; ++ks) {
        frags((ks + 1) & 1, cur, ks + 1, -1, nullptr);
        mfma(ks & 1, acc);
        schedule(0);
      }
      if (kt + 1 < nk) {
        __builtin_amdgcn_s_waitcnt(wait_vm(0));
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        frags(0, next, 0, -1, nullptr);
        if (kt + S::NS < nk) load_parts(cur, 0, kSpread);
      }
      mfma((KS - 1) & 1, acc);
      char *const free = cur;
      cur = next;
      next = S::NS == 2 ? free : prev;
      prev = free;
    }
  }
};

#endif  // __HIP_DEVICE_COMPILE__

}  // namespace tile
}  // namespace vpe

#endif
