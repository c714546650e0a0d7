// Rows of 16-bit, fp32 and 8-bit elements in the kernels: matrix instructions,
// conversions, chunks of 16 bytes at any alignment, and the 8-bit codes of a row.
#pragma once
#include "dense_launch.h"

namespace moe {

typedef _Float16 f16;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------ element types
template <int T> struct Elem;
template <> struct Elem<DT_BF16> {
  typedef f32x4 acc4;
  static constexpr int SIZE = 2;
  static __device__ __forceinline__ acc4 mma16(u32x4 p, u32x4 q, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p), __builtin_bit_cast(bf16x8, q), c,
                                                   0, 0, 0);
  }
};
template <> struct Elem<DT_F16> {
  typedef f32x4 acc4;
  static constexpr int SIZE = 2;
  static __device__ __forceinline__ acc4 mma16(u32x4 p, u32x4 q, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, p), __builtin_bit_cast(f16x8, q), c, 0,
                                                  0, 0);
  }
};
template <> struct Elem<DT_I8> {
  typedef i32x4 acc4;
  static constexpr int SIZE = 1;
  static __device__ __forceinline__ acc4 mma16(u32x4 p, u32x4 q, acc4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, p), __builtin_bit_cast(i32x4, q), c, 0, 0,
                                                 0);
  }
};

// ------------------------------------------------------------ conversions
template <int T> __device__ __forceinline__ uint16_t to16(float v) {
  if constexpr (T == DT_BF16) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (f16)v);
}
template <int T> struct Row;
template <> struct Row<DT_BF16> {
  typedef uint16_t type;
  static __device__ __forceinline__ float f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
};
template <> struct Row<DT_F16> {
  typedef uint16_t type;
  static __device__ __forceinline__ float f(uint16_t b) { return (float)__builtin_bit_cast(f16, b); }
};
template <> struct Row<DT_F32> {
  typedef float type;
  static __device__ __forceinline__ float f(float b) { return b; }
};

template <int T> __device__ __forceinline__ void unpack16(u32x4 v, float* f) {
  if constexpr (T == DT_F32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = Row<T>::f((uint16_t)v[i]);
      f[2 * i + 1] = Row<T>::f((uint16_t)(v[i] >> 16));
    }
  }
}

template <int DT> __device__ __forceinline__ u32x4 pack16(const float* f) {
  u32x4 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = to16<DT>(f[2 * k]) | (uint32_t)to16<DT>(f[2 * k + 1]) << 16;
  return v;
}
// what rounding v to 16 bits leaves (nothing where that is not finite)
template <int DT> __device__ __forceinline__ float low_part(float v) {
  const float hi = Row<DT>::f(to16<DT>(v));
  return __builtin_fabsf(hi) < __builtin_inff() ? v - hi : 0.f;
}
// -------------------------------------------------- rows at any alignment
// 16 bytes of a row from byte `byte` on, of elements of ES bytes, zero from
// byte `end` on. Global loads take any alignment. SHIFT: a chunk that passes the
// end is the row's last 16 bytes, shifted, instead of up to 15 loads (8-bit
// 333 x 1288 -> 776, both operands copied: 10.9 us for 11.6); the decode kernel
// has no registers left for it.
template <int ES, bool SHIFT = false>
__device__ __forceinline__ u32x4 load_chunk(const void* row, int64_t byte, int64_t end) {
  const uint8_t* at = static_cast<const uint8_t*>(row) + byte;
  u32x4 v = {0, 0, 0, 0};
  if (byte + 16 <= end) {
    __builtin_memcpy(&v, at, 16);
  } else if (SHIFT && end >= 16) {
    __builtin_memcpy(&v, static_cast<const uint8_t*>(row) + (end - 16), 16);
    const int n = (int)min(byte + 16 - end, (int64_t)16) * 8;
    uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
    lo = n < 64 ? lo >> n | hi << 1 << (63 - n) : n < 128 ? hi >> (n - 64) : 0;
    hi = n < 64 ? hi >> n : 0;
    v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  } else {
    uint8_t* b = reinterpret_cast<uint8_t*>(&v);
#pragma unroll
    for (int i = 0; i < 16; i += ES)
      if (byte + i < end) __builtin_memcpy(b + i, at + i, ES);
  }
  return v;
}

// ---------------------------------------------------------------- quantising
// Scale of a row whose largest |x| has the bits m, and its codes: q =
// round-half-even of the exact x / s, |q| <= 127, 0 where s is not positive.
// The fp32 product with the reciprocal (off by less than 1.15e-5: 127 2^-24 from
// the reciprocal's rounding, 2^-18 from a product between 64 and 128) decides,
// four values at a time, unless one of them lies within 2e-5
// of a half-integer or the reciprocal overflows (a subnormal scale); then
// 53-bit quotients do: x - s (n + 1/2) is zero or at least 2^-32 of x, so 53
// bits tell the two apart. (A wider margin sends whole waves there: with 1e-3 the
// 8-bit block of 1 x 2048 -> 2 x 512 takes 5.5 us instead of 5.2.)
struct RowScale {
  float s, inv;
  bool fast;
  __device__ __forceinline__ explicit RowScale(uint32_t m) {
    s = m < 0x7F800000u ? __uint_as_float(m) / 127.f : __builtin_nanf("");
    inv = s > 0.f ? 1.f / s : 0.f;
    fast = s > 0.f && inv < 3e38f;
  }
  __device__ __forceinline__ uint32_t exact(float x) const {
    const double q = __builtin_rint((double)x / (double)s);
    return s > 0.f ? (uint32_t)(int)__builtin_fmin(__builtin_fmax(q, -127.0), 127.0) & 255u : 0u;
  }
  // four codes, the first in the low byte
  __device__ __forceinline__ uint32_t codes4(const float* f) const {
    float n[4], far = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = f[e] * inv;
      n[e] = __builtin_rintf(t);
      far = __builtin_fmaxf(far, __builtin_fabsf(t - n[e]));
    }
    uint32_t o = 0;
    if (fast && far < 0.49998f) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o |= ((uint32_t)(int)n[e] & 255u) << (8 * e);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) o |= exact(f[e]) << (8 * e);
    }
    return o;
  }
};
template <int T, int N> __device__ __forceinline__ uint32_t top_bits(const float* f, uint32_t m) {
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}

}  // namespace moe
