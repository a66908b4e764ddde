// Device helpers shared by the training and beam-search kernels: fp32 and
// bf16 elements in vectors of 8 or 16 bytes, widened to fp32 registers.
#ifndef VPE_DEVICE_H
#define VPE_DEVICE_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vpe {
namespace dev {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 values rounded to bf16 (nearest, ties to even), packed: one
// v_cvt_pk_bf16_f32.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const f32x2 v = {a, b};
  const bf16x2 r = __builtin_convertvector(v, bf16x2);
  return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ uint16_t one_bf16(float a) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(a));
}

// EPV elements (2 or 4 bytes each) moved as one vector of 8 or 16 bytes.  Rows
// may begin at any element, so the types only ask for the element's alignment
// (global accesses of any width may: the hardware splits what crosses).
template <int BYTES> struct Raw;
template <> struct Raw<16> {
  typedef u32x4 type;
  typedef u32x4 __attribute__((aligned(2))) loose;
};
template <> struct Raw<8> {
  typedef u32x2 type;
  typedef u32x2 __attribute__((aligned(2))) loose;
};

template <bool BF16, int EPV>
struct Vec {
  static constexpr int kSize = BF16 ? 2 : 4;
  typedef typename Raw<EPV * kSize>::type raw;
  typedef typename Raw<EPV * kSize>::loose loose;

  static __device__ __forceinline__ void widen(raw r, float (&v)[EPV]) {
    if constexpr (!BF16) {
#pragma unroll
      for (int e = 0; e < EPV; ++e) v[e] = __uint_as_float(r[e]);
    } else {
#pragma unroll
      for (int e = 0; e < EPV / 2; ++e) v[2 * e] = bf16_lo(r[e]), v[2 * e + 1] = bf16_hi(r[e]);
    }
  }
  static __device__ __forceinline__ raw narrow(const float (&v)[EPV]) {
    raw r;
    if constexpr (!BF16) {
#pragma unroll
      for (int e = 0; e < EPV; ++e) r[e] = __float_as_uint(v[e]);
    } else {
#pragma unroll
      for (int e = 0; e < EPV / 2; ++e) r[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    }
    return r;
  }
};

template <bool BF16>
__device__ __forceinline__ float load_one(const void *base, int64_t i) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(base)[i]) << 16);
  return static_cast<const float *>(base)[i];
}
template <bool BF16>
__device__ __forceinline__ void store_one(void *base, int64_t i, float v) {
  if constexpr (BF16) static_cast<uint16_t *>(base)[i] = one_bf16(v);
  else static_cast<float *>(base)[i] = v;
}

// Elements [i, i + EPV) of a row of n, 0 past its end.
template <bool BF16, int EPV>
__device__ __forceinline__ void load_vec(const void *row, int64_t i, int64_t n, float (&v)[EPV]) {
  typedef Vec<BF16, EPV> V;
  if (i + EPV <= n) {
    const char *p = static_cast<const char *>(row) + i * V::kSize;
    V::widen(*reinterpret_cast<const typename V::loose *>(p), v);
  } else {
#pragma unroll
    for (int e = 0; e < EPV; ++e) v[e] = i + e < n ? load_one<BF16>(row, i + e) : 0.f;
  }
}
template <bool BF16, int EPV>
__device__ __forceinline__ void store_vec_nt(void *row, int64_t i, int64_t n,
                                             const float (&v)[EPV]) {
  typedef Vec<BF16, EPV> V;
  if (i + EPV <= n) {
    char *p = static_cast<char *>(row) + i * V::kSize;
    __builtin_nontemporal_store(V::narrow(v), reinterpret_cast<typename V::loose *>(p));
  } else {
#pragma unroll
    for (int e = 0; e < EPV; ++e)
      if (i + e < n) store_one<BF16>(row, i + e, v[e]);
  }
}

// `bytes` (even) zero bytes at p (even), by `lanes` lanes: whole 16-byte words
// where they are aligned.
template <bool NT>
__device__ __forceinline__ void zero_bytes(char *p, int64_t bytes, int64_t lane, int64_t lanes) {
  int64_t head = static_cast<int64_t>(-reinterpret_cast<uintptr_t>(p) & 15);
  if (head > bytes) head = bytes;
  const int64_t words = (bytes - head) / 16;
  u32x4 *w = reinterpret_cast<u32x4 *>(p + head);
  for (int64_t i = lane; i < words; i += lanes) {
    if constexpr (NT) __builtin_nontemporal_store(u32x4(0), w + i);
    else w[i] = u32x4(0);
  }
  if (head != 0 || (bytes & 15) != 0) {
    for (int64_t i = lane * 2; i < head; i += lanes * 2) *reinterpret_cast<uint16_t *>(p + i) = 0;
    for (int64_t i = head + words * 16 + lane * 2; i < bytes; i += lanes * 2)
      *reinterpret_cast<uint16_t *>(p + i) = 0;
  }
}

// Reductions over the wave's 64 lanes by DPP moves, within rows of 16 lanes
// (row_shr 1, 2, 4, 8) and from row to row (row_bcast 15 and 31): lane 63 ends
// with the whole, and all lanes read it there.  The order is fixed.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float old, float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL,
                                                    ROWS, 0xf, false));
}
__device__ __forceinline__ float last_lane(float v) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_max(float v) {  // NaN is passed over
  v = fmaxf(v, dpp<0x111, 0xf>(v, v));
  v = fmaxf(v, dpp<0x112, 0xf>(v, v));
  v = fmaxf(v, dpp<0x114, 0xf>(v, v));
  v = fmaxf(v, dpp<0x118, 0xf>(v, v));
  v = fmaxf(v, dpp<0x142, 0xf>(v, v));
  return last_lane(fmaxf(v, dpp<0x143, 0xf>(v, v)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111, 0xf>(0.f, v);
  v += dpp<0x112, 0xf>(0.f, v);
  v += dpp<0x114, 0xf>(0.f, v);
  v += dpp<0x118, 0xf>(0.f, v);
  v += dpp<0x142, 0xa>(0.f, v);
  return last_lane(v + dpp<0x143, 0xc>(0.f, v));
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d /= 2) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ int wave_in_block() {
  return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
}

}  // namespace dev
}  // namespace vpe

#endif
