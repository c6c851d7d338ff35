// float_types.hpp -- the row types of the float operators (f32, bf16, f16):
// conversions and 16-byte pieces of a row at element alignment.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>

#include "../../include/qpack.h"

namespace qp {

// bf16 held as its bits; f16 is the compiler's own type.
struct bf16_t {
  uint16_t u;
};
typedef _Float16 f16_t;

inline int elem_bytes(int32_t dtype) { return dtype == QP_F32 ? 4 : 2; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) {
  return __builtin_bit_cast(float, (uint32_t)v.u << 16);
}
__device__ __forceinline__ float to_f32(f16_t v) { return (float)v; }

// Round to nearest, ties to even; a NaN stays one.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ f16_t from_f32<f16_t>(float v) {
  return (f16_t)v;
}
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) {
  const __bf16 b = (__bf16)v;
  return bf16_t{__builtin_bit_cast(uint16_t, b)};
}

// 16 bytes at any address a 2- or 4-byte element can have.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// 16 bytes of a row.  Rows may start at any multiple of the element size:
// the card's global loads and stores take a 16-byte access at any address,
// so an odd row length costs no separate path, only the last piece does.
template <typename T>
struct Piece {
  static constexpr int kPer = 16 / sizeof(T);
  typedef uint32_t vec __attribute__((ext_vector_type(4)));
  vec v;
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) {
      const uint32_t u = v[i];
      return __builtin_bit_cast(float, u);
    } else {
      const uint32_t u = v[i / 2];
      const uint16_t h = (uint16_t)(i & 1 ? u >> 16 : u & 0xffffu);
      return to_f32(__builtin_bit_cast(T, h));
    }
  }
};

// The first n elements at p (none for n <= 0), the rest of the piece zero; p[0]
// must be readable in any case.  A cut piece's elements are loaded without a
// branch each, so that they come in together.
template <typename T>
__device__ __forceinline__ Piece<T> load_piece(const T* p, int n) {
  Piece<T> r;
  if (n >= Piece<T>::kPer) {
    r.v = *reinterpret_cast<const u32x4_any*>(p);
  } else {
    T e[Piece<T>::kPer];
#pragma unroll
    for (int i = 0; i < Piece<T>::kPer; ++i) e[i] = p[i < n ? i : 0];
    r.v = typename Piece<T>::vec{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < Piece<T>::kPer; ++i) {
      if constexpr (sizeof(T) == 4)
        r.v[i] = i < n ? __builtin_bit_cast(uint32_t, e[i]) : 0u;
      else
        r.v[i / 2] |= (i < n ? (uint32_t)__builtin_bit_cast(uint16_t, e[i]) : 0u) << (16 * (i & 1));
    }
  }
  return r;
}

// The first n of a piece's values, each rounded to T.
template <typename T>
__device__ __forceinline__ void store_piece(T* p, const float (&f)[16 / sizeof(T)], int n) {
  constexpr int kPer = 16 / sizeof(T);
  if (n >= kPer) {
    u32x4_any v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4)
        v[i] = __builtin_bit_cast(uint32_t, f[i]);
      else
        v[i] = (uint32_t)__builtin_bit_cast(uint16_t, from_f32<T>(f[2 * i])) |
               (uint32_t)__builtin_bit_cast(uint16_t, from_f32<T>(f[2 * i + 1])) << 16;
    }
    *reinterpret_cast<u32x4_any*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) p[i] = from_f32<T>(f[i]);
  }
}

}  // namespace qp
