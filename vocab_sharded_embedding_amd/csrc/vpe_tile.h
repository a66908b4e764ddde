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
// bf16: v_mfma_f32_32x32x16_bf16.  Both operands are staged through NS stages of
// LDS by buffer loads that write LDS directly, BK values of k each.  A lane's
// fragment is 8 consecutive k of one n or m: an operand in rows gives it in one
// 16-byte LDS read, one in columns in two transposing 8-byte reads
// (ds_read_b64_tr_b16: 16 lanes read 4 values of k x 16 columns and get 4 values
// of k of one column each).
// fp32: v_mfma_f32_32x32x2_f32 on tiles kept in LDS with k outermost.
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

// One operand's side of the staging.  `COLS`: it lies in columns.
template <bool COLS, int SIDE, int BK, int NW>
struct Stage;

// In rows: LDS row n holds BK values as pieces of 16 bytes, piece p at slot
// p ^ f(n).  The LDS serves a 16-byte read 16 lanes at a time over 64 banks (256
// bytes), and those lanes read one piece of 16 consecutive rows: f changes with
// every 256 bytes of rows, so that they meet 16 different groups of 4 banks
// (counted bank conflicts: half of the LDS's cycles with f changing every 128
// bytes).
template <int SIDE, int BK, int NW>
struct Stage<false, SIDE, BK, NW> {
  static constexpr int kElems = SIDE * BK;
  static constexpr int kPieces = BK / 8, kRowsPerLoad = 64 / kPieces;
  static constexpr int kLoads = SIDE / kRowsPerLoad / NW;
  static_assert(kLoads * kRowsPerLoad * NW == SIDE, "whole loads per wave");
  const char *base;
  int left;  // bytes from base to the operand's end (of SIDE rows: below 2^31)
  int k_left;
  int voff[kLoads];
  int piece8[2];  // first k of this lane's piece, by load
  int rd[BK / 16];

  static __device__ __forceinline__ int swizzle(int row) {
    constexpr int kGroup = BK * 2 >= 256 ? 1 : 256 / (BK * 2);
    return (row / kGroup) & (kPieces - 1);
  }
  // `rows` rows from p on exist, of k_limit values (a multiple of 8) each.
  __device__ __forceinline__ void init(const uint16_t *p, int64_t ld, int64_t rows,
                                       int64_t k_limit, int side_base) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    base = reinterpret_cast<const char *>(p);
    left = static_cast<int>(rows > 0 ? ((rows < SIDE ? rows : SIDE) - 1) * ld * 2 + k_limit * 2 : 0);
    k_left = static_cast<int>(k_limit);
    const int lrow = lane / kPieces, slot = lane % kPieces;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int row = (q * NW + wave) * kRowsPerLoad + lrow;
      const int piece = slot ^ swizzle(row);
      voff[q] = row < rows ? static_cast<int>(row * ld * 2) + piece * 16 : kLoadMask;
    }
    // (two loads cover whole periods of f)
    piece8[0] = (slot ^ swizzle(wave * kRowsPerLoad + lrow)) * 8;
    piece8[1] = (slot ^ swizzle((NW + wave) * kRowsPerLoad + lrow)) * 8;
    static_assert(2 * NW * kRowsPerLoad % 16 == 0, "loads two apart take one piece");
    const int row = side_base + (lane & 31);
#pragma unroll
    for (int ks = 0; ks < BK / 16; ++ks)
      rd[ks] = row * BK + (((ks * 2 + (lane >> 5)) ^ swizzle(row)) << 3);
  }
  // This wave's q-th load of the next BK values of k into the stage at `dst`.
  __device__ __forceinline__ void load(uint16_t *dst, int q) const {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(base), 0, left > 0 ? left : 0, kRawBuffer);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (__attribute__((address_space(3))) void *)(dst + (q * NW + wave_id()) * 512), 16,
        piece8[q & 1] < k_left ? voff[q] : kLoadMask, 0, 0, 0);
  }
  __device__ __forceinline__ void advance() {
    base += BK * 2;
    left -= BK * 2;
    k_left -= BK;
  }
  __device__ __forceinline__ bf16x8 frag(const uint16_t *src, int ks, int i) const {
    return *reinterpret_cast<const bf16x8 *>(src + rd[ks] + i * 32 * BK);
  }
};

// In columns: LDS row k holds SIDE values as segments of 32 bytes, segment s at
// s ^ f(k), f(k) = r ^ 2 r ^ (bit 3 of k), r = k % 4.  A transposing read takes
// one segment of 4 values of k per 16 lanes: those 4 segments, and the 8 of 32
// lanes, meet different groups of banks.
template <int SIDE, int BK, int NW>
struct Stage<true, SIDE, BK, NW> {
  static constexpr int kElems = SIDE * BK;
  static constexpr int kPieces = SIDE / 8, kRowsPerLoad = 64 / kPieces;
  static constexpr int kLoads = BK / kRowsPerLoad / NW;
  static_assert(kLoads * kRowsPerLoad * NW == BK && SIDE >= 128, "whole loads per wave");
  const char *base;
  int64_t left, step;
  int voff[kLoads];
  int rd[4];

  static __device__ __forceinline__ int swizzle(int k) {
    return ((k & 3) ^ ((k & 3) << 1) ^ ((k >> 3) & 1)) & 7;
  }
  // Columns from p on, `cols` of them inside a row (which ends at a multiple of 8);
  // k_limit rows exist.
  __device__ __forceinline__ void init(const uint16_t *p, int64_t ld, int64_t cols,
                                       int64_t k_limit, int side_base) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    base = reinterpret_cast<const char *>(p);
    left = k_limit > 0 ? ((k_limit - 1) * ld + (cols + 7) / 8 * 8) * 2 : 0;
    step = ld * BK * 2;
    const int lrow = lane / kPieces, slot = lane % kPieces;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int k = (q * NW + wave) * kRowsPerLoad + lrow;
      const int seg = (slot >> 1) ^ swizzle(k);
      // 16 bytes that begin at or past the row's last column are another row's
      // (or lie past the end): nothing reads them
      voff[q] = static_cast<int>(k * ld * 2) + (seg * 2 + (slot & 1)) * 16;
    }
    const int r = (lane & 15) >> 2, hi = lane >> 5, b = (lane >> 4) & 1;
    const int f = swizzle(r + 8 * hi);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      rd[i] = (8 * hi + r) * SIDE + (((side_base / 16 + 2 * i + b) ^ f) << 4) + (lane & 3) * 4;
  }
  __device__ __forceinline__ void load(uint16_t *dst, int q) const {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(base), 0,
        static_cast<int>(left > kLoadMask ? kLoadMask : (left > 0 ? left : 0)), kRawBuffer);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rsrc, (__attribute__((address_space(3))) void *)(dst + (q * NW + wave_id()) * 512), 16,
        voff[q], 0, 0, 0);
  }
  __device__ __forceinline__ void advance() {
    base += step;
    left -= step;
  }
  __device__ __forceinline__ bf16x8 frag(const uint16_t *src, int ks, int i) const {
    typedef __attribute__((address_space(3))) s16x4 lds_v;
    const uint16_t *p = src + rd[i & 3] + (i >> 2) * 128 + ks * 16 * SIDE;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v *)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v *)(p + 4 * SIDE));
    return __builtin_bit_cast(bf16x8,
                              __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// The stages are LDS arrays of their own, and every access names one: the
// compiler then sees that a read does not touch the stage that a load in flight
// fills, and waits for no load on its account (it puts a wait for all of them
// before every transposing read otherwise: 8192^3 in columns 1091 against 956 us).
template <class S, bool NCOLS, bool MCOLS>
struct Product {
  typedef Stage<NCOLS, S::BN, S::BK, S::NW> StageN;
  typedef Stage<MCOLS, S::BM, S::BK, S::NW> StageM;
  static constexpr int kStageBytes = (StageN::kElems + StageM::kElems) * 2;
  static constexpr int kLoads = StageN::kLoads + StageM::kLoads;
  static constexpr int KS = S::BK / 16;
  static constexpr int kReads = S::FN * (NCOLS ? 2 : 1) + S::FM * (MCOLS ? 2 : 1);
  static constexpr int kMfma = S::FN * S::FM;
  static_assert(KS % 2 == 0, "fragments alternate between two sets of registers");
  static_assert((S::NS - 1) * kLoads <= 63, "outstanding loads fit the counter");
  // The loads of a step go out over kSpread rounds, from the one in which its
  // stage is free: the memory path takes one load of 64 x 16 bytes per 16 cycles
  // and CU, and a wave that finds its queue full issues no MFMA either.
  static constexpr int kSpread = KS < 3 ? KS : 3;
  static constexpr int kPart = (kLoads + kSpread - 1) / kSpread;

  StageN a;
  StageM b;
  bf16x8 fa[2][S::FN], fb[2][S::FM];

  __device__ __forceinline__ void load(char *stage, int q) {
    uint16_t *dst = reinterpret_cast<uint16_t *>(stage);
    if (q < StageN::kLoads) a.load(dst, q);
    else if (q < kLoads) b.load(dst + StageN::kElems, q - StageN::kLoads);
  }
  __device__ __forceinline__ void load_parts(char *stage, int from, int to) {
#pragma unroll
    for (int q = from * kPart; q < to * kPart; ++q) load(stage, q);
    if (to == kSpread) a.advance(), b.advance();
  }
  // The fragments of round ks of a stage, and (part >= 0) a part of the loads into
  // stage `to` in turn with them.
  __device__ __forceinline__ void frags(int set, const char *stage, int ks, int part, char *to) {
    const uint16_t *src = reinterpret_cast<const uint16_t *>(stage);
    constexpr int kF = S::FN + S::FM;
#pragma unroll
    for (int f = 0; f < (kF > kPart ? kF : kPart); ++f) {
      if (f < S::FM) fb[set][f] = b.frag(src + StageN::kElems, ks, f);
      else if (f < kF) fa[set][f - S::FM] = a.frag(src, ks, f - S::FM);
      if (part >= 0 && f < kPart) load(to, part * kPart + f);
    }
    if (part == kSpread - 1) a.advance(), b.advance();
  }
  __device__ __forceinline__ void mfma(int set, f32x16 (&acc)[S::FN][S::FM]) const {
#pragma unroll
    for (int i = 0; i < S::FN; ++i)
#pragma unroll
      for (int j = 0; j < S::FM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[set][i], fb[set][j], acc[i][j], 0,
                                                            0, 0);
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
  // acc += the product over nk steps, through the stages st (NS of them).  A wave
  // reads each fragment one round of MFMAs ahead; the loads of a step begin NS - 1
  // steps before it.  Ends with every load landed.
  __device__ __forceinline__ void run(int nk, char *const (&st)[kStages],
                                      f32x16 (&acc)[S::FN][S::FM]) {
    if (nk <= 0) return;
    // (few steps: every stage at once, nothing spread)
    bool rest = nk >= 2 * S::NS;
#pragma unroll
    for (int s = 0; s < S::NS - 1; ++s)
      if (s < nk) load_parts(st[s], 0, kSpread);
    if (rest) {
      load_parts(st[S::NS - 1], 0, 1);
      __builtin_amdgcn_s_waitcnt(wait_vm((S::NS - 2) * kLoads + kPart));
    } else if (S::NS - 1 < nk) {
      load_parts(st[S::NS - 1], 0, kSpread);
      __builtin_amdgcn_s_waitcnt(wait_vm((S::NS - 1) * kLoads));
    } else {
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
    }
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

// ---------------------------------------------------------------------------
// fp32
// ---------------------------------------------------------------------------
// One fp32 operand: BK values of k of SIDE rows (or columns) pass through
// registers into LDS with k outermost, whichever way they lie in memory.  The
// row stride of SIDE + 4 spreads the transposing writes of an operand in rows.
template <bool COLS, int SIDE, int BK, int NT>
struct StageF {
  static constexpr int kLd = SIDE + 4;
  static constexpr int kElems = BK * kLd;
  static constexpr int kVecs = SIDE * BK / 4 / NT;
  static_assert(kVecs * 4 * NT == SIDE * BK, "whole vectors per thread");
  const float *base;
  int64_t ld, limit, k_left, k_at;
  bool wide;
  f32x4 v[kVecs];

  // `limit_` rows (columns) from p on exist, k_limit values of k.
  __device__ __forceinline__ void init(const float *p, int64_t ld_, int64_t limit_,
                                       int64_t k_limit) {
    base = p, ld = ld_, limit = limit_, k_left = k_limit, k_at = 0;
    wide = (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld_ & 3) == 0;
  }
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int q = 0; q < kVecs; ++q) {
      const int t = q * NT + static_cast<int>(threadIdx.x);
      int64_t at, in, left;  // first element, whether its line exists, elements left in it
      if constexpr (COLS) {
        const int k = t / (SIDE / 4), i = t % (SIDE / 4) * 4;
        at = (k_at + k) * ld + i, in = k < k_left, left = limit - i;
      } else {
        const int i = t / (BK / 4), k = t % (BK / 4) * 4;
        at = i * ld + k_at + k, in = i < limit, left = k_left - k;
      }
      f32x4 r = f32x4(0.f);
      if (in && wide && left >= 4) {
        r = *reinterpret_cast<const f32x4 *>(base + at);
      } else if (in) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < left) r[e] = base[at + e];
      }
      v[q] = r;
    }
    k_at += BK;
    k_left -= BK;
  }
  __device__ __forceinline__ void store(float *dst) const {
#pragma unroll
    for (int q = 0; q < kVecs; ++q) {
      const int t = q * NT + static_cast<int>(threadIdx.x);
      if constexpr (COLS) {
        const int k = t / (SIDE / 4), i = t % (SIDE / 4) * 4;
        *reinterpret_cast<f32x4 *>(dst + k * kLd + i) = v[q];
      } else {
        const int i = t / (BK / 4), k = t % (BK / 4) * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[(k + e) * kLd + i] = v[q][e];
      }
    }
  }
};

template <class S, bool NCOLS, bool MCOLS>
struct ProductF {
  typedef StageF<NCOLS, S::BN, S::BK, S::NT> StageN;
  typedef StageF<MCOLS, S::BM, S::BK, S::NT> StageM;
  static constexpr int kStageBytes = (StageN::kElems + StageM::kElems) * 4;

  StageN a;
  StageM b;

  __device__ __forceinline__ void run(int nk, char *const (&st)[kStages], int side_n, int side_m,
                                      f32x16 (&acc)[S::FN][S::FM]) {
    static_assert(S::NS == 2, "two stages");
    if (nk <= 0) return;
    const int lane = threadIdx.x & 63, row = lane & 31, hi = lane >> 5;
    a.load();
    b.load();
    float *even = reinterpret_cast<float *>(st[0]), *odd = reinterpret_cast<float *>(st[1]);
    a.store(even);
    b.store(even + StageN::kElems);
    for (int kt = 0; kt < nk; ++kt) {
      __syncthreads();
      float *cur = kt & 1 ? odd : even, *next = kt & 1 ? even : odd;
      if (kt + 1 < nk) {
        a.load();
        b.load();
      }
#pragma unroll
      for (int k = 0; k < S::BK; k += 2) {
        float fa[S::FN], fb[S::FM];
#pragma unroll
        for (int i = 0; i < S::FN; ++i)
          fa[i] = cur[(k + hi) * StageN::kLd + side_n + i * 32 + row];
#pragma unroll
        for (int j = 0; j < S::FM; ++j)
          fb[j] = cur[StageN::kElems + (k + hi) * StageM::kLd + side_m + j * 32 + row];
#pragma unroll
        for (int j = 0; j < S::FM; ++j)
#pragma unroll
          for (int i = 0; i < S::FN; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fa[i], fb[j], acc[i][j], 0, 0, 0);
      }
      if (kt + 1 < nk) {
        a.store(next);
        b.store(next + StageN::kElems);
      }
    }
  }
};

#endif  // __HIP_DEVICE_COMPILE__

}  // namespace tile
}  // namespace vpe

#endif
