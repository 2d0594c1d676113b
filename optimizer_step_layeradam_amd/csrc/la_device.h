// Device helpers shared by the norms' and the loss' kernels. Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace la {

// Element types (la_element_type); encode rounds to nearest even.
struct Bf16 {
  static constexpr int bytes = 2;
  typedef uint16_t bits;
  typedef __bf16 native;
  static __device__ __forceinline__ float decode(uint16_t b) {
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
  }
  static __device__ __forceinline__ uint16_t encode(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
  }
};

struct Fp16 {
  static constexpr int bytes = 2;
  typedef uint16_t bits;
  typedef _Float16 native;
  static __device__ __forceinline__ float decode(uint16_t b) {
    return static_cast<float>(__builtin_bit_cast(_Float16, b));
  }
  static __device__ __forceinline__ uint16_t encode(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
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

// A vector of x, two numbers an instruction.
template <typename T>
__device__ __forceinline__ Vector<T> encode_vector(const float (&x)[Vector<T>::n]) {
  Vector<T> v;
  if constexpr (T::bytes == 4) {
    __builtin_memcpy(&v, x, 16);
  } else {
    typename T::native o __attribute__((ext_vector_type(8)));
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = static_cast<typename T::native>(x[i]);
    __builtin_memcpy(&v, &o, 16);
  }
  return v;
}

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

// How the rows of a launch end: with a whole vector, inside one, or before the
// first one does.
enum class Ends { kWhole, kInside, kTiny };

// A vector of a row as its 16 bytes come from memory. All lanes read, those past
// the row and the one whose vector passes its end the row's last 16 bytes: there
// is no branch, so several loads are under way at once. settled() makes elements
// [at, at + n) of it, zeros past the row.
typedef uint32_t u32x4_bits __attribute__((ext_vector_type(4)));
typedef unsigned __int128 bits128;

template <typename T, Ends ENDS>
__device__ __forceinline__ u32x4_bits load_raw(const typename T::bits* row, int at, int cols) {
  u32x4_bits v = {};
  if constexpr (ENDS == Ends::kTiny) {
    bits128 b = 0;
    if (at == 0)
      for (int i = 0; i < cols; ++i) b |= static_cast<bits128>(row[i]) << (8 * T::bytes * i);
    __builtin_memcpy(&v, &b, 16);
  } else {
    const int last = cols - Vector<T>::n;
    __builtin_memcpy(&v, row + (at < last ? at : last), 16);
  }
  return v;
}

template <typename T, Ends ENDS>
__device__ __forceinline__ Vector<T> settled(u32x4_bits v, int at, int cols) {
  if constexpr (ENDS == Ends::kInside) {
    const int past = at + Vector<T>::n - cols;
    if (past > 0 && at < cols) {
      bits128 b;
      __builtin_memcpy(&b, &v, 16);
      b >>= 8 * T::bytes * past;
      __builtin_memcpy(&v, &b, 16);
    }
  }
  if constexpr (ENDS != Ends::kTiny) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = at < cols ? v[i] : 0u;
  }
  return __builtin_bit_cast(Vector<T>, v);
}

}  // namespace la
