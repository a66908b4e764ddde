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
// p ^ f(n), so that the 8 lanes of an LDS pass, which read one piece of 8
// consecutive rows, meet 8 different groups of banks.
template <int SIDE, int BK, int NW>
struct Stage<false, SIDE, BK, NW> {
  static constexpr int kElems = SIDE * BK;
  static constexpr int kPieces = BK / 8, kRowsPerLoad = 64 / kPieces;
  static constexpr int kLoads = SIDE / kRowsPerLoad / NW;
  static_assert(kLoads * kRowsPerLoad * NW == SIDE, "whole loads per wave");
  const char *base;
  int64_t left;  // bytes from base to the operand's end
  int64_t k_left;
  int voff[kLoads];
  int piece8;  // first k of this lane's piece
  int rd[BK / 16];

  static __device__ __forceinline__ int swizzle(int row) {
    constexpr int kGroup = BK * 2 >= 128 ? 1 : 128 / (BK * 2);
    return (row / kGroup) & (kPieces - 1);
  }
  // `rows` rows from p on exist, of k_limit values (a multiple of 8) each.
  __device__ __forceinline__ void init(const uint16_t *p, int64_t ld, int64_t rows,
                                       int64_t k_limit, int side_base) {
    const int lane = threadIdx.x & 63, wave = wave_id();
    base = reinterpret_cast<const char *>(p);
    left = rows > 0 ? ((rows < SIDE ? rows : SIDE) - 1) * ld * 2 + k_limit * 2 : 0;
    k_left = k_limit;
    const int lrow = lane / kPieces, slot = lane % kPieces;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const int row = (q * NW + wave) * kRowsPerLoad + lrow;
      const int piece = slot ^ swizzle(row);
      voff[q] = row < rows ? static_cast<int>(row * ld * 2) + piece * 16 : kLoadMask;
    }
    // (kRowsPerLoad is a multiple of the swizzle's period: one piece for all loads)
    piece8 = (slot ^ swizzle(lrow)) * 8;
    static_assert(kRowsPerLoad % 8 == 0, "one piece per lane");
    const int row = side_base + (lane & 31);
#pragma unroll
    for (int ks = 0; ks < BK / 16; ++ks)
      rd[ks] = row * BK + (((ks * 2 + (lane >> 5)) ^ swizzle(row)) << 3);
  }
  // The next BK values of k into the stage at `dst`.
  __device__ __forceinline__ void load(uint16_t *dst) {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(base), 0, static_cast<int>(left > 0 ? left : 0), kRawBuffer);
    const int wave = wave_id();
    const bool in = piece8 < k_left;
#pragma unroll
    for (int q = 0; q < kLoads; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (__attribute__((address_space(3))) void *)(dst + (q * NW + wave) * 512), 16,
          in ? voff[q] : kLoadMask, 0, 0, 0);
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
  __device__ __forceinline__ void load(uint16_t *dst) {
    const int64_t most = kLoadMask;
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char *>(base), 0,
        static_cast<int>(left > most ? most : (left > 0 ? left : 0)), kRawBuffer);
    const int wave = wave_id();
#pragma unroll
    for (int q = 0; q < kLoads; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (__attribute__((address_space(3))) void *)(dst + (q * NW + wave) * 512), 16,
          voff[q], 0, 0, 0);
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

template <class S, bool NCOLS, bool MCOLS>
struct Product {
  typedef Stage<NCOLS, S::BN, S::BK, S::NW> StageN;
  typedef Stage<MCOLS, S::BM, S::BK, S::NW> StageM;
  static constexpr int kStageElems = StageN::kElems + StageM::kElems;
  static constexpr int kLoads = StageN::kLoads + StageM::kLoads;
  static constexpr int KS = S::BK / 16;
  static constexpr int kReads = S::FN * (NCOLS ? 2 : 1) + S::FM * (MCOLS ? 2 : 1);
  static constexpr int kMfma = S::FN * S::FM;
  static constexpr int kLdsElems = S::NS * kStageElems;
  static_assert(KS % 2 == 0, "fragments alternate between two sets of registers");
  static_assert((S::NS - 1) * kLoads <= 63, "outstanding loads fit the counter");

  // Reads, and in a step's last round the loads of a later step, go out between
  // the MFMAs: 8192 x 8192 x 1024 in rows 125 -> 123 us, 128 x 128 tiles 143 -> 139.
  static __device__ __forceinline__ void schedule(bool last) {
    constexpr int kHalf = kMfma / 2 > 0 ? kMfma / 2 : 1;
    if (!last) {
      constexpr int kPer = (kReads + kMfma - 1) / kMfma;
#pragma unroll
      for (int g = 0; g < kReads / kPer; ++g) {
        __builtin_amdgcn_sched_group_barrier(0x100, kPer, 0);  // LDS reads
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     // MFMAs
      }
      __builtin_amdgcn_sched_group_barrier(0x008, kMfma, 0);
    } else {
      constexpr int kPer = (kReads + kHalf - 1) / kHalf, kLoad = (kLoads + kHalf - 1) / kHalf;
#pragma unroll
      for (int g = 0; g < kHalf; ++g) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, kPer, 0);
      }
#pragma unroll
      for (int g = 0; g < kHalf; ++g) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, kLoad, 0);  // global loads
      }
    }
  }

  // acc += the product over nk steps.  A wave reads each fragment one MFMA round
  // ahead; the loads of a step go out NS - 1 steps before it.
  static __device__ __forceinline__ void run(StageN &a, StageM &b, int nk, uint16_t *lds,
                                             f32x16 (&acc)[S::FN][S::FM]) {
    if (nk <= 0) return;
    bf16x8 fa[2][S::FN], fb[2][S::FM];
    auto load = [&](int buf) {
      a.load(lds + buf * kStageElems);
      b.load(lds + buf * kStageElems + StageN::kElems);
    };
    auto frags = [&](int set, int buf, int ks) {
      const uint16_t *src = lds + buf * kStageElems;
#pragma unroll
      for (int i = 0; i < S::FN; ++i) fa[set][i] = a.frag(src, ks, i);
#pragma unroll
      for (int j = 0; j < S::FM; ++j) fb[set][j] = b.frag(src + StageN::kElems, ks, j);
    };
    auto mfma = [&](int set) {
#pragma unroll
      for (int j = 0; j < S::FM; ++j)
#pragma unroll
        for (int i = 0; i < S::FN; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[set][i], fb[set][j], acc[i][j],
                                                              0, 0, 0);
    };
#pragma unroll
    for (int st = 0; st < S::NS; ++st)
      if (st < nk) load(st);
    if (nk >= S::NS) __builtin_amdgcn_s_waitcnt(wait_vm((S::NS - 1) * kLoads));
    else __builtin_amdgcn_s_waitcnt(wait_vm(0));
    asm volatile("s_barrier" ::: "memory");
    frags(0, 0, 0);
    int cur = 0;
    for (int kt = 0; kt < nk; ++kt) {
      const int next = cur + 1 == S::NS ? 0 : cur + 1;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if (ks + 1 < KS) {
          frags((ks + 1) & 1, cur, ks + 1);
        } else if (kt + 1 < nk) {
          // step kt + 1 has landed for this wave, and this wave has read step kt;
          // after the barrier both hold for all waves
          if (kt + S::NS <= nk) __builtin_amdgcn_s_waitcnt(wait_vm((S::NS - 2) * kLoads));
          else __builtin_amdgcn_s_waitcnt(wait_vm(0));
          asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
          if (kt + S::NS < nk) load(cur);
          frags(0, next, 0);
        }
        mfma(ks & 1);
        schedule(ks + 1 == KS);
      }
      cur = next;
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
  static constexpr int kStageElems = StageN::kElems + StageM::kElems;
  static constexpr int kLdsElems = 2 * kStageElems;

  static __device__ __forceinline__ void run(StageN &a, StageM &b, int nk, float *lds, int side_n,
                                             int side_m, f32x16 (&acc)[S::FN][S::FM]) {
    if (nk <= 0) return;
    const int lane = threadIdx.x & 63, row = lane & 31, hi = lane >> 5;
    a.load();
    b.load();
    a.store(lds);
    b.store(lds + StageN::kElems);
    for (int kt = 0; kt < nk; ++kt) {
      __syncthreads();
      float *cur = lds + (kt & 1) * kStageElems, *next = lds + ((kt + 1) & 1) * kStageElems;
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
