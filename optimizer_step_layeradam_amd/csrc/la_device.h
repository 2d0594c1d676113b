// Device helpers shared by the norms' and the loss' kernels. Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace la {

// Element types (la_element_type).
struct Bf16 {
  static constexpr int bytes = 2;
  typedef uint16_t bits;
  static __device__ __forceinline__ float decode(uint16_t b) {
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
  }
  // round to nearest even, NaN -> 0x7FC0 (as in the update's kernel)
  static __device__ __forceinline__ uint16_t encode(float x) {
    const uint32_t b = __float_as_uint(x);
    const uint32_t r = (b + 0x7FFFu + ((b >> 16) & 1u)) >> 16;
    return static_cast<uint16_t>(__builtin_isnan(x) ? 0x7FC0u : r);
  }
};

struct Fp16 {
  static constexpr int bytes = 2;
  typedef uint16_t bits;
  static __device__ __forceinline__ float decode(uint16_t b) {
    return static_cast<float>(__builtin_bit_cast(_Float16, b));
  }
  static __device__ __forceinline__ uint16_t encode(float x) {
    const uint16_t h = __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
    return __builtin_isnan(x) ? uint16_t(0x7E00) : h;
  }
};

struct Fp32 {
  static constexpr int bytes = 4;
  typedef uint32_t bits;
  static __device__ __forceinline__ float decode(uint32_t b) { return __uint_as_float(b); }
  static __device__ __forceinline__ uint32_t encode(float x) { return __float_as_uint(x); }
};

// 16 bytes of elements in registers.
template <typename T>
struct Vector {
  static constexpr int n = 16 / T::bytes;
  typename T::bits e[n];
};

// Elements [at, at + n) of a row of `cols`, those past it as zeros. Rows may
// start at any element: a 16-byte access needs no alignment on this GPU.
template <typename T>
__device__ __forceinline__ Vector<T> load_vector(const typename T::bits* row, int at, int cols) {
  Vector<T> v;
  if (at + v.n <= cols) {
    __builtin_memcpy(&v, row + at, 16);
  } else {
#pragma unroll
    for (int i = 0; i < v.n; ++i) v.e[i] = at + i < cols ? row[at + i] : 0;
  }
  return v;
}

template <typename T>
__device__ __forceinline__ void store_vector(typename T::bits* row, int at, int cols,
                                             const Vector<T>& v) {
  if (at + v.n <= cols) {
    __builtin_memcpy(row + at, &v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < v.n; ++i)
      if (at + i < cols) row[at + i] = v.e[i];
  }
}

}  // namespace la
