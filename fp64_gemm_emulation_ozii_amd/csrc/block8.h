// Blocks of 128 in 8-bit floating point: their scales and roundings, and runs
// of eight entries of a caller's array.
//
// A block's scale is the least power of two 2^e with amax <= MAX 2^e (e >= -126;
// 1 for a block of zeros), so x 2^-e is exact and every value is rounded
// once.  An entry that is Inf or NaN becomes NaN and does not count for amax.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ozgemm.h"

namespace oz {

constexpr int BLOCK8 = 128;

typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u8 __attribute__((ext_vector_type(4)));
typedef float v4f8 __attribute__((ext_vector_type(4)));
typedef v2u v2u_at1 __attribute__((aligned(1)));
typedef v4u8 v4u_at1 __attribute__((aligned(1)));
typedef v4u8 v4u_at2 __attribute__((aligned(2)));
typedef v4f8 v4f_at4 __attribute__((aligned(4)));

// The largest value of an 8-bit type is 1.75 2^TOP.
template <int QTYPE>
struct Eight {
  static constexpr int TOP = QTYPE == OZGEMM_E4M3 ? 8 : 15;
  // four values on the type's range, as its bytes, to nearest-even
  static __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    int w = 0;
    if (QTYPE == OZGEMM_E4M3) {
      w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    } else {
      w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
      w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
    }
    return (uint32_t)w;
  }
};

// |x| as an order-preserving integer; 0 for Inf and NaN.
__device__ __forceinline__ uint32_t finite_abs(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}

// Inf as NaN: the conversion to e5m2 keeps infinities.
__device__ __forceinline__ float no_inf(float x) {
  return (__builtin_bit_cast(uint32_t, x) & 0x7fffffffu) == 0x7f800000u ? __builtin_nanf("") : x;
}

// e of the block's scale 2^e from the bits of amax.
template <int QTYPE>
__device__ __forceinline__ int scale_exponent(uint32_t amax) {
  if (amax == 0) return 0;
  // amax = 1.f 2^E; one more where 1.f > 1.75.  (A subnormal amax has E <= -127: the clamp.)
  const int E = (int)(amax >> 23) - 127;
  const int e = E - Eight<QTYPE>::TOP + ((amax & 0x7fffffu) > 0x600000u);
  return max(e, -126);
}

__device__ __forceinline__ float power_of_two(int e) {  // -126 <= e <= 127
  return __builtin_bit_cast(float, (uint32_t)(e + 127) << 23);
}

// x rounded to odd (towards zero, with the last bit set where that dropped
// something): rounding it again, to any shorter type, is rounding x once, and
// comparisons with shorter values come out as x's.
__device__ __forceinline__ float to_odd(double x) {
  uint64_t b = __builtin_bit_cast(uint64_t, x);
  if ((b & 0x1fffffffu) != 0) b = (b & ~0x1fffffffull) | 0x20000000ull;
  return (float)__builtin_bit_cast(double, b);
}

template <int TYPE>
struct Entry;
template <>
struct Entry<OZGEMM_F32> {
  typedef float T;
  static constexpr int BYTES = 4;
};
template <>
struct Entry<OZGEMM_BF16> {
  typedef __bf16 T;
  static constexpr int BYTES = 2;
};
template <>
struct Entry<OZGEMM_F16> {
  typedef _Float16 T;
  static constexpr int BYTES = 2;
};

// Eight entries next to each other, of which the first `left` exist: raw as they came, so that many can be in flight.
template <int TYPE>
struct Raw8 {
  v4u8 w[TYPE == OZGEMM_F32 ? 2 : 1];

  __device__ __forceinline__ void load(const void* base, long at, int left) {
    typedef typename Entry<TYPE>::T T;
    const T* p = (const T*)base + at;
    if (left >= 8) {
      if constexpr (TYPE == OZGEMM_F32) {
        w[0] = __builtin_bit_cast(v4u8, *reinterpret_cast<const v4f_at4*>(p));
        w[1] = __builtin_bit_cast(v4u8, *reinterpret_cast<const v4f_at4*>(p + 4));
      } else {
        w[0] = *reinterpret_cast<const v4u_at2*>(p);
      }
    } else {
      T v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = k < left ? p[k] : (T)0.f;
      __builtin_memcpy(w, v, sizeof(v));
    }
  }
  __device__ __forceinline__ void zero() {
    w[0] = v4u8{0, 0, 0, 0};
    if constexpr (TYPE == OZGEMM_F32) w[1] = w[0];
  }
  __device__ __forceinline__ float get(int k) const {
    if constexpr (TYPE == OZGEMM_F32) {
      return __builtin_bit_cast(float, (uint32_t)w[k >> 2][k & 3]);
    } else if constexpr (TYPE == OZGEMM_BF16) {
      const uint32_t u = w[0][k >> 1];
      return __builtin_bit_cast(float, (k & 1) ? u & 0xffff0000u : u << 16);
    } else {
      const uint32_t u = w[0][k >> 1];
      return (float)__builtin_bit_cast(_Float16, (uint16_t)((k & 1) ? u >> 16 : u));
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    typename Entry<TYPE>::T t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = (typename Entry<TYPE>::T)v[k];
    __builtin_memcpy(w, t, sizeof(t));
  }
  __device__ __forceinline__ void store(void* base, long at, int left) const {
    typedef typename Entry<TYPE>::T T;
    T* p = (T*)base + at;
    if (left >= 8) {
      if constexpr (TYPE == OZGEMM_F32) {
        *reinterpret_cast<v4f_at4*>(p) = __builtin_bit_cast(v4f8, w[0]);
        *reinterpret_cast<v4f_at4*>(p + 4) = __builtin_bit_cast(v4f8, w[1]);
      } else {
        *reinterpret_cast<v4u_at2*>(p) = w[0];
      }
    } else {
      T v[8];
      __builtin_memcpy(v, w, sizeof(v));
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < left) p[k] = v[k];
    }
  }
};

// Eight bytes next to each other, of which the first `left` exist.
__device__ __forceinline__ void store_bytes(uint8_t* p, v2u v, int left) {
  if (left >= 8) {
    *reinterpret_cast<v2u_at1*>(p) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) p[k] = (uint8_t)(v[k >> 2] >> (8 * (k & 3)));
  }
}

// The value of the lane N on, around the row of 16 lanes.
template <int N>
__device__ __forceinline__ uint32_t rotated(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, false);
}
template <int N>
__device__ __forceinline__ double rotated(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)rotated<N>((uint32_t)u) | (uint64_t)rotated<N>((uint32_t)(u >> 32)) << 32);
}

// The largest of 16 neighbouring lanes, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, rotated<8>(v));
  v = max(v, rotated<4>(v));
  v = max(v, rotated<2>(v));
  return max(v, rotated<1>(v));
}

// The sum of a wavefront, the same bits in all of its lanes.
__device__ __forceinline__ double sum64(double v) {
  v += rotated<8>(v);
  v += rotated<4>(v);
  v += rotated<2>(v);
  v += rotated<1>(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

}  // namespace oz
