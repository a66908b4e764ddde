// Device helpers shared by the training and beam-search kernels: fp32 and
// bf16 elements in vectors of up to 16 bytes, widened to fp32 registers.
#ifndef VPE_DEVICE_H
#define VPE_DEVICE_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vpe {
namespace dev {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
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

template <int BYTES> struct Raw;
template <> struct Raw<16> { typedef u32x4 type; };
template <> struct Raw<8> { typedef u32x2 type; };
template <> struct Raw<4> { typedef uint32_t type; };
template <> struct Raw<2> { typedef uint16_t type; };

// EPV elements (2 or 4 bytes each) moved as one vector.
template <bool BF16, int EPV>
struct Vec {
  static constexpr int kBytes = EPV * (BF16 ? 2 : 4);
  typedef typename Raw<kBytes>::type raw;

  static __device__ __forceinline__ void widen(raw r, float (&v)[EPV]) {
    if constexpr (!BF16) {
      if constexpr (EPV == 1) {
        v[0] = __uint_as_float(r);
      } else {
#pragma unroll
        for (int e = 0; e < EPV; ++e) v[e] = __uint_as_float(r[e]);
      }
    } else if constexpr (EPV == 1) {
      v[0] = __uint_as_float(static_cast<uint32_t>(r) << 16);
    } else if constexpr (EPV == 2) {
      v[0] = bf16_lo(r), v[1] = bf16_hi(r);
    } else {
#pragma unroll
      for (int e = 0; e < EPV / 2; ++e) v[2 * e] = bf16_lo(r[e]), v[2 * e + 1] = bf16_hi(r[e]);
    }
  }

  static __device__ __forceinline__ raw narrow(const float (&v)[EPV]) {
    if constexpr (!BF16) {
      if constexpr (EPV == 1) {
        return __float_as_uint(v[0]);
      } else {
        raw r;
#pragma unroll
        for (int e = 0; e < EPV; ++e) r[e] = __float_as_uint(v[e]);
        return r;
      }
    } else if constexpr (EPV == 1) {
      return one_bf16(v[0]);
    } else if constexpr (EPV == 2) {
      return pack_bf16(v[0], v[1]);
    } else {
      raw r;
#pragma unroll
      for (int e = 0; e < EPV / 2; ++e) r[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
      return r;
    }
  }
};

// Vectors of EPV elements, EPV * element size possibly 32 bytes (fp32 beside
// bf16 vectors of 8): loaded and stored in 16-byte halves.
template <bool BF16, int EPV>
__device__ __forceinline__ void load_vec(const void *base, int64_t elem, float (&v)[EPV]) {
  if constexpr (!BF16 && EPV == 8) {
    float a[4], b[4];
    load_vec<false, 4>(base, elem, a);
    load_vec<false, 4>(base, elem + 4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
  } else {
    typedef Vec<BF16, EPV> V;
    const char *p = static_cast<const char *>(base) + elem * (BF16 ? 2 : 4);
    V::widen(*reinterpret_cast<const typename V::raw *>(p), v);
  }
}

template <bool BF16, int EPV>
__device__ __forceinline__ void store_vec_nt(void *base, int64_t elem, const float (&v)[EPV]) {
  if constexpr (!BF16 && EPV == 8) {
    float a[4], b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = v[e], b[e] = v[4 + e];
    store_vec_nt<false, 4>(base, elem, a);
    store_vec_nt<false, 4>(base, elem + 4, b);
  } else {
    typedef Vec<BF16, EPV> V;
    char *p = static_cast<char *>(base) + elem * (BF16 ? 2 : 4);
    __builtin_nontemporal_store(V::narrow(v), reinterpret_cast<typename V::raw *>(p));
  }
}

__device__ __forceinline__ int wave_in_block() {
  return __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
}

}  // namespace dev
}  // namespace vpe

#endif
