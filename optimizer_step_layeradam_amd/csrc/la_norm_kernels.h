// Pieces of the norms' kernels (la_norm.hip, la_norm_backward.h). Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "la_device.h"
#include "la_muon.h"
#include "la_norm.h"

#pragma clang fp contract(off)

namespace la {
namespace {

// Elements [at, at + N) of a parameter as binary32, `otherwise` past the row and
// where there is none. The type is the same for a whole launch.
template <typename W, Ends ENDS, int N>
__device__ __forceinline__ void load_parameter_of(float (&to)[N], const void* p, int at, int cols,
                                                  float otherwise) {
  constexpr int n = Vector<W>::n;
  const typename W::bits* row = static_cast<const typename W::bits*>(p);
  if constexpr (ENDS == Ends::kWhole) {
    // as many whole vectors of the parameter as one of the row holds, or half of one
    if (N >= n || at + n <= cols) {
#pragma unroll
      for (int k = 0; k < N; k += n) {
        const Vector<W> x = settled<W, ENDS>(load_raw<W, ENDS>(row, at + k, cols), at + k, cols);
#pragma unroll
        for (int i = 0; i < (N < n ? N : n); ++i)
          to[k + i] = at + k + i < cols ? W::decode(x.e[i]) : otherwise;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) to[i] = at + i < cols ? W::decode(row[at + i]) : otherwise;
}

template <Ends ENDS, int N>
__device__ __forceinline__ void load_parameter(float (&to)[N], const void* p, int type, int at,
                                               int cols, float otherwise) {
  if (p == nullptr) {
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = otherwise;
  } else if (type == kFp32) {
    load_parameter_of<Fp32, ENDS>(to, p, at, cols, otherwise);
  } else if (type == kFp16) {
    load_parameter_of<Fp16, ENDS>(to, p, at, cols, otherwise);
  } else {
    load_parameter_of<Bf16, ENDS>(to, p, at, cols, otherwise);
  }
}

__device__ __forceinline__ void store_parameter(void* p, int type, int64_t at, float x) {
  if (type == kFp32) static_cast<float*>(p)[at] = x;
  else static_cast<uint16_t*>(p)[at] = type == kFp16 ? Fp16::encode(x) : Bf16::encode(x);
}

// The row's start. Where all lanes of a wave are at one row (SAME) it is scalar,
// and an access takes a lane's offset alone from the vector registers.
template <typename T, bool SAME>
__device__ __forceinline__ typename T::bits* row_of(const NormRows& t, int row, int inner) {
  if constexpr (SAME) row = __builtin_amdgcn_readfirstlane(row);
  typename T::bits* p = static_cast<typename T::bits*>(t.p);
  if (inner == 1) return p + row * t.outer_stride;
  const int i = static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(inner));
  return p + i * t.outer_stride + (row - i * inner) * t.inner_stride;
}

// `at`, of which the compiler knows nothing: what follows from it (masks, addresses,
// a parameter's elements) is formed again where it is needed, and not kept in
// registers from one row to the next.
__device__ __forceinline__ int formed_again(int at) {
  asm volatile("" : "+v"(at));
  return at;
}

// Sums of N values over the G lanes that share a row; every one of them gets
// the result. Within a wave by exchanges; over a workgroup of G lanes the waves'
// sums meet in LDS, in two places in turn, so that one barrier a time is
// enough.
template <int G, int N>
struct RowSum {
  static constexpr int waves = G > 64 ? G / 64 : 1;
  float (*part)[N][waves];
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&x)[N]) {
#pragma unroll
    for (int d = (G < 64 ? G : 64) / 2; d > 0; d >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] += __shfl_xor(x[k], d, 64);
    if constexpr (G > 64) {
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) part[turn][k][threadIdx.x >> 6] = x[k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < N; ++k) {
        x[k] = part[turn][k][0];
#pragma unroll
        for (int w = 1; w < waves; ++w) x[k] += part[turn][k][w];
      }
      turn ^= 1;
    }
  }
};

template <int G>
constexpr int threads_of() {
  return G > 256 ? G : 256;
}

// ---- launches -------------------------------------------------------------------------

hipError_t launch(const void* kernel, int64_t grid, int threads, const NormArgs& a,
                  hipStream_t stream, int64_t max_grid) {
  grid = std::min({grid, kMaxWorkgroups, max_grid});
  NormArgs copy = a;
  void* params[] = {&copy};
  return hipLaunchKernel(kernel, dim3(static_cast<unsigned>(std::max<int64_t>(1, grid))),
                         dim3(threads), params, 0, stream);
}

// The lanes that share a row, the 16-byte vectors that each of them holds, and
// how rows end.
template <typename F>
auto with_shape(int64_t bytes, F f) {
  using std::integral_constant;
  auto at = [&](auto g, auto p) {
    return bytes % 16 == 0 ? f(g, p, integral_constant<Ends, Ends::kWhole>())
                           : f(g, p, integral_constant<Ends, Ends::kInside>());
  };
#define LA_SHAPE(G, P) at(integral_constant<int, G>(), integral_constant<int, P>())
  if (bytes < 16)
    return f(integral_constant<int, 4>(), integral_constant<int, 1>(),
             integral_constant<Ends, Ends::kTiny>());
  if (bytes <= 4 * 16) return LA_SHAPE(4, 1);
  if (bytes <= 16 * 16) return LA_SHAPE(16, 1);
  if (bytes <= 64 * 16) return LA_SHAPE(64, 1);
  if (bytes <= 128 * 16) return LA_SHAPE(64, 2);
  if (bytes <= 256 * 16) return LA_SHAPE(256, 1);
  if (bytes <= 512 * 16) return LA_SHAPE(256, 2);
  if (bytes <= 768 * 16) return LA_SHAPE(256, 3);
  if (bytes <= 1024 * 16) return LA_SHAPE(256, 4);
  return LA_SHAPE(1024, 2);
#undef LA_SHAPE
}

// The same for rows of more than kNormRegisterBytes, 1024 lanes to each.
template <typename T, typename F>
hipError_t with_wide_shape(int64_t bytes, F f) {
  using std::integral_constant;
  auto at = [&](auto p) {
    return bytes % 16 == 0 ? f(p, integral_constant<Ends, Ends::kWhole>())
                           : f(p, integral_constant<Ends, Ends::kInside>());
  };
  if (bytes <= 3 * 16384) return at(integral_constant<int, 3>());
  if constexpr (T::bytes == 4) {
    if (bytes > 6 * 16384) return at(integral_constant<int, 8>());
    if (bytes > 4 * 16384) return at(integral_constant<int, 6>());
  }
  return at(integral_constant<int, 4>());
}

}  // namespace
}  // namespace la
