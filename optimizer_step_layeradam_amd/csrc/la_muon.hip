// la_muon.hip -- the passes over the directions for gfx950: the momentum of
// a Muon step, sums of squares, and the normalised first iterate.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "la_muon.h"

#pragma clang fp contract(off)

namespace la {
namespace {

constexpr int kThreads = 256;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float from_bf16(uint16_t b) {
  return __uint_as_float(static_cast<uint32_t>(b) << 16);
}
__device__ __forceinline__ float from_fp16(uint16_t b) {
  return static_cast<float>(__builtin_bit_cast(_Float16, b));
}
template <bool FP16>
__device__ __forceinline__ float decode(uint16_t b) {
  return FP16 ? from_fp16(b) : from_bf16(b);
}

// Sum over the workgroup in a fixed order: across each wave by halves, then
// the waves in turn. Every thread gets the result.
__device__ __forceinline__ double block_sum(double x) {
  __shared__ double part[kThreads / 64];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = part[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) s += part[i];
  __syncthreads();
  return s;
}

// ---- momentum --------------------------------------------------------------------
// One pass over the gradients: g = (G_0 + ... + G_{R-1}) * unscale in replica
// order, B <- mu B + g in place, u = g + mu B where the Nesterov form is asked
// for (else u = B), and the sum of u^2 of each chunk in binary64 (the squares
// of binary32 values neither overflow nor vanish there). Reads 2R + 4 bytes
// and writes 4 or 8 per element: memory decides. A layer of 330 million
// parameters with eight replicas, 9.2 GB: 1.82 ms, 5.1 TB/s.

template <int R>
struct MomentumArgs {
  struct {
    float* momentum;
    float* direction;
    const uint16_t* g[R];
    double* partial;
    int64_t numel, direction_stride, chunk;
    int32_t partials, vectors;
  } t[kGroupsPerLaunch];
  int64_t end[kGroupsPerLaunch];  // cumulative workgroups
  int32_t* flag;
  const int32_t* skip;
  float mu, unscale;
  int32_t count;
};

template <int R, bool FP16>
__global__ __launch_bounds__(kThreads) void momentum_kernel(MomentumArgs<R> a) {
  if (a.skip != nullptr && *a.skip != 0) return;
  const int64_t total = a.end[a.count - 1];
  bool bad = false;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    int i = 0;
    while (w >= a.end[i]) ++i;
    const auto& t = a.t[i];
    const int64_t local = w - (i ? a.end[i - 1] : 0);
    const int64_t z = local / t.partials, c = local % t.partials;
    const int64_t first = c * t.chunk;
    const int64_t last = first + t.chunk < t.numel ? first + t.chunk : t.numel;
    const int64_t base = z * t.numel;
    float* B = t.momentum + base;
    float* U = t.direction != nullptr ? t.direction + z * t.direction_stride : nullptr;
    double sum = 0.0;
    auto one = [&](float g, float b, float& u) {
      g = g * a.unscale;
      bad |= !(__builtin_fabsf(g) < __builtin_inff());
      b = a.mu * b + g;
      u = U != nullptr ? g + a.mu * b : b;
      sum += static_cast<double>(u) * static_cast<double>(u);
      return b;
    };
    int64_t e = first + threadIdx.x * 8;
    if (t.vectors) {
      for (; e + 8 <= last; e += kThreads * 8) {
        u32x4 G[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
          G[r] = *reinterpret_cast<const u32x4*>(t.g[r] + base + e);
        f32x4 b[2] = {*reinterpret_cast<const f32x4*>(B + e),
                      *reinterpret_cast<const f32x4*>(B + e + 4)};
        f32x4 u[2];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float g = decode<FP16>(static_cast<uint16_t>(G[0][k >> 1] >> (16 * (k & 1))));
#pragma unroll
          for (int r = 1; r < R; ++r)
            g = g + decode<FP16>(static_cast<uint16_t>(G[r][k >> 1] >> (16 * (k & 1))));
          float x;
          b[k >> 2][k & 3] = one(g, b[k >> 2][k & 3], x);
          u[k >> 2][k & 3] = x;
        }
        *reinterpret_cast<f32x4*>(B + e) = b[0];
        *reinterpret_cast<f32x4*>(B + e + 4) = b[1];
        if (U != nullptr) {
          *reinterpret_cast<f32x4*>(U + e) = u[0];
          *reinterpret_cast<f32x4*>(U + e + 4) = u[1];
        }
      }
      // the thread whose eight elements pass the end takes them one by one
      for (int64_t k = e; k < last && k < e + 8; ++k) {
        float g = decode<FP16>(t.g[0][base + k]), u;
#pragma unroll
        for (int r = 1; r < R; ++r) g = g + decode<FP16>(t.g[r][base + k]);
        B[k] = one(g, B[k], u);
        if (U != nullptr) U[k] = u;
      }
    } else {
      for (int64_t k = first + threadIdx.x; k < last; k += kThreads) {
        float g = decode<FP16>(t.g[0][base + k]), u;
#pragma unroll
        for (int r = 1; r < R; ++r) g = g + decode<FP16>(t.g[r][base + k]);
        B[k] = one(g, B[k], u);
        if (U != nullptr) U[k] = u;
      }
    }
    const double s = block_sum(sum);
    if (threadIdx.x == 0) t.partial[z * t.partials + c] = s;
  }
  if (a.flag != nullptr && __any(bad) && (threadIdx.x & 63) == 0) atomicOr(a.flag, 1);
}

template <int R>
hipError_t launch_momentum_r(const MomentumGroup* groups, int count, bool fp16, float mu,
                             float unscale, int32_t* flag, const int32_t* skip,
                             hipStream_t stream, int64_t max_grid) {
  MomentumArgs<R> a = {};
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    a.t[i].momentum = groups[i].momentum;
    a.t[i].direction = groups[i].direction;
    for (int r = 0; r < R; ++r) a.t[i].g[r] = groups[i].g[r];
    a.t[i].partial = groups[i].partial;
    a.t[i].numel = groups[i].numel;
    a.t[i].direction_stride = groups[i].direction_stride;
    a.t[i].chunk = groups[i].chunk;
    a.t[i].partials = groups[i].partials;
    a.t[i].vectors = groups[i].vectors;
    total += static_cast<int64_t>(groups[i].partials) * groups[i].count;
    a.end[i] = total;
  }
  a.flag = flag;
  a.skip = skip;
  a.mu = mu;
  a.unscale = unscale;
  a.count = count;
  int64_t grid = total < kMaxWorkgroups ? total : kMaxWorkgroups;
  if (grid > max_grid) grid = max_grid;
  const void* k = fp16 ? reinterpret_cast<const void*>(&momentum_kernel<R, true>)
                       : reinterpret_cast<const void*>(&momentum_kernel<R, false>);
  void* params[] = {&a};
  return hipLaunchKernel(k, dim3(static_cast<unsigned>(grid)), dim3(kThreads), params, 0, stream);
}

// ---- sums of squares and the first iterate --------------------------------------

struct DirectionArgs {
  DirectionGroup g[kGroupsPerLaunch];
  int64_t end[kGroupsPerLaunch];  // cumulative workgroups
  double eps;
  const int32_t* skip;
  float scale;
  int32_t count;
  int32_t strip;  // normalise: tiles of a workgroup
};
static_assert(sizeof(DirectionArgs) <= 4096, "kernel arguments");

template <int TYPE>
__device__ __forceinline__ float element(const void* p, int64_t at) {
  if constexpr (TYPE == kFp32) return static_cast<const float*>(p)[at];
  else if constexpr (TYPE == kFp16) return from_fp16(static_cast<const uint16_t*>(p)[at]);
  else return from_bf16(static_cast<const uint16_t*>(p)[at]);
}

// Eight elements at once (16-byte aligned), left as they came.
template <int TYPE>
struct Eight {
  u32x4 v[TYPE == kFp32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const u32x4* from = reinterpret_cast<const u32x4*>(static_cast<const char*>(p) +
                                                       at * (TYPE == kFp32 ? 4 : 2));
    v[0] = __builtin_nontemporal_load(from);
    if constexpr (TYPE == kFp32) v[1] = __builtin_nontemporal_load(from + 1);
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (TYPE == kFp32) return __uint_as_float(v[e >> 2][e & 3]);
    const uint16_t b = static_cast<uint16_t>(v[0][e >> 1] >> (16 * (e & 1)));
    return TYPE == kFp16 ? from_fp16(b) : from_bf16(b);
  }
};

// Workgroup (z, c): rows [c, c + 1) * rows_per_partial of matrix z; a row is
// shared by a power of two of threads, as many as it has pieces (eight
// elements where they are aligned, else one). Memory decides: 178 MB of BF16
// in 38 us (4.7 TB/s), against 160 us one element at a time.
template <int TYPE>
__global__ __launch_bounds__(kThreads) void square_sum_kernel(DirectionArgs a) {
  const int64_t total = a.end[a.count - 1];
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    int i = 0;
    while (w >= a.end[i]) ++i;
    const DirectionGroup& g = a.g[i];
    const int64_t local = w - (i ? a.end[i - 1] : 0);
    const int64_t z = local / g.partials, c = local % g.partials;
    const int pieces = g.vectors ? g.cols >> 3 : g.cols;
    int across = 1;
    while (across < pieces && across < kThreads) across <<= 1;
    const int first = static_cast<int>(c * g.rows_per_partial);
    const int last = first + g.rows_per_partial < g.rows ? first + g.rows_per_partial : g.rows;
    double sum = 0.0;
    for (int r = first + threadIdx.x / across; r < last; r += kThreads / across) {
      const int64_t row = z * g.matrix_stride + r * g.row_stride;
      if (g.vectors) {
#pragma unroll 4
        for (int k = threadIdx.x % across; k < pieces; k += across) {
          Eight<TYPE> v;
          v.load(g.in, row + 8 * k);
          // added up for themselves: eight squares to one of the long sum
          double part = 0.0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const double x = v[e];
            part += x * x;
          }
          sum += part;
        }
      } else {
#pragma unroll 4
        for (int k = threadIdx.x % across; k < pieces; k += across) {
          const double x = element<TYPE>(g.in, row + k);
          sum += x * x;
        }
      }
    }
    const double s = block_sum(sum);
    if (threadIdx.x == 0) g.partial[local] = s;
  }
}

// A strip of 64 rows and up to `strip` tiles of 64 columns of X_0 =
// U / max(||U||_F, eps) per workgroup, in both layouts (the turned one through
// LDS), zeros in the padding. A norm that is not finite makes every element
// NaN, as the products would anyway. A thread takes eight neighbours of a row.
// Reads 2 or 4 bytes and writes 5 per element: memory decides (89 million BF16
// elements in 115 us, 5.4 TB/s).
constexpr int kStrip = 4;  // one where the launch has few tiles: latency counts there

template <int TYPE>
__global__ __launch_bounds__(kThreads) void normalise_kernel(DirectionArgs a) {
  // rows of 64 with their 16-byte pieces at piece ^ (row / 8): a turned read
  // meets every bank equally often
  __shared__ __align__(16) _Float16 turn[64 * 64];
  if (a.skip != nullptr && *a.skip != 0) return;
  const int64_t total = a.end[a.count - 1];
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    int i = 0;
    while (w >= a.end[i]) ++i;
    const DirectionGroup& g = a.g[i];
    const int64_t local = w - (i ? a.end[i - 1] : 0);
    const int tiles = g.ld_straight >> 6, down = g.ld_turned >> 6;
    const int across = (tiles + a.strip - 1) / a.strip;
    const int64_t z = local / (across * down);
    const int t = static_cast<int>(local % (across * down));
    const int r0 = (t / across) * 64, first = (t % across) * a.strip;
    const int last = first + a.strip < tiles ? first + a.strip : tiles;

    double sum = 0.0;
    for (int k = threadIdx.x; k < g.partials; k += kThreads) sum += g.partial[z * g.partials + k];
    sum = block_sum(sum);
    const double norm = __builtin_sqrt(sum);
    const double denominator = norm < a.eps ? a.eps : norm;  // NaN stays
    double factor = denominator > 0.0 ? static_cast<double>(a.scale) / denominator : 0.0;
    if (!(sum < __builtin_inf())) factor = __builtin_nan("");

    const int piece = threadIdx.x & 7, rx = threadIdx.x >> 3;  // and row rx + 32
    for (int c = first; c < last; ++c) {
      const int c0 = c * 64 + 8 * piece;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = rx + 32 * k, row = r0 + r;
        half8 hi = {};
        u32x2 lo = {};
        if (row < g.rows) {
          const int64_t at = z * g.matrix_stride + row * g.row_stride + c0;
          float x[8];
          if (g.vectors && c0 + 8 <= g.cols) {
            Eight<TYPE> v;
            v.load(g.in, at);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = v[e];
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)  // from inside the row: see the zeros below
              x[e] = element<TYPE>(g.in, at - c0 + (c0 + e < g.cols ? c0 + e : g.cols - 1));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = static_cast<float>(static_cast<double>(x[e]) * factor);
            if (c0 + e >= g.cols) x[e] = 0.0f;
            hi[e] = static_cast<_Float16>(x[e]);
            lo[e >> 2] |= (static_cast<uint32_t>(low_byte(x[e], hi[e])) & 0xFFu) << (8 * (e & 3));
          }
          const int64_t to = (z * g.rows + row) * g.ld_straight + c0;
          *reinterpret_cast<half8*>(reinterpret_cast<_Float16*>(g.straight) + to) = hi;
          *reinterpret_cast<u32x2*>(g.straight_lo + to) = lo;
        }
        *reinterpret_cast<half8*>(turn + r * 64 + ((piece ^ (r >> 3)) << 3)) = hi;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = rx + 32 * k, r = 8 * piece;  // of the tile, turned
        half8 h;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          h[e] = turn[(r + e) * 64 + (((col >> 3) ^ piece) << 3) + (col & 7)];
        if (c * 64 + col < g.cols)
          *reinterpret_cast<half8*>(reinterpret_cast<_Float16*>(g.turned) +
                                    (z * g.cols + c * 64 + col) * g.ld_turned + r0 + r) = h;
      }
      __syncthreads();
    }
  }
}

template <typename K>
hipError_t launch_directions(K kernel, DirectionArgs& a, int64_t total, hipStream_t stream,
                             int64_t max_grid) {
  int64_t grid = total < kMaxWorkgroups ? total : kMaxWorkgroups;
  if (grid > max_grid) grid = max_grid;
  void* params[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(static_cast<unsigned>(grid)),
                         dim3(kThreads), params, 0, stream);
}

}  // namespace

hipError_t launch_momentum(const MomentumGroup* groups, int count, int replicas, bool fp16,
                           float mu, float unscale, int32_t* flag, const int32_t* skip,
                           hipStream_t stream, int64_t max_grid) {
  switch (replicas) {
#define LA_CASE(RR)                                                                          \
  case RR:                                                                                   \
    return launch_momentum_r<RR>(groups, count, fp16, mu, unscale, flag, skip, stream, max_grid);
    LA_CASE(1) LA_CASE(2) LA_CASE(3) LA_CASE(4) LA_CASE(5) LA_CASE(6) LA_CASE(7) LA_CASE(8)
#undef LA_CASE
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_square_sums(const DirectionGroup* groups, int count, int type,
                              hipStream_t stream, int64_t max_grid) {
  DirectionArgs a = {};
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    a.g[i] = groups[i];
    total += static_cast<int64_t>(groups[i].partials) * groups[i].count;
    a.end[i] = total;
  }
  a.count = count;
  return type == kFp32   ? launch_directions(&square_sum_kernel<kFp32>, a, total, stream, max_grid)
         : type == kFp16 ? launch_directions(&square_sum_kernel<kFp16>, a, total, stream, max_grid)
                         : launch_directions(&square_sum_kernel<kBf16>, a, total, stream, max_grid);
}

hipError_t launch_normalise(const DirectionGroup* groups, int count, int type, float scale,
                            double eps, const int32_t* skip, hipStream_t stream,
                            int64_t max_grid) {
  DirectionArgs a = {};
  int64_t total = 0;
  for (int i = 0; i < count; ++i)
    total += static_cast<int64_t>(groups[i].ld_straight >> 6) * (groups[i].ld_turned >> 6) *
             groups[i].count;
  a.strip = total < 4096 ? 1 : kStrip;
  total = 0;
  for (int i = 0; i < count; ++i) {
    a.g[i] = groups[i];
    const int across = ((groups[i].ld_straight >> 6) + a.strip - 1) / a.strip;
    total += static_cast<int64_t>(across) * (groups[i].ld_turned >> 6) * groups[i].count;
    a.end[i] = total;
  }
  a.eps = eps;
  a.skip = skip;
  a.scale = scale;
  a.count = count;
  return type == kFp32   ? launch_directions(&normalise_kernel<kFp32>, a, total, stream, max_grid)
         : type == kFp16 ? launch_directions(&normalise_kernel<kFp16>, a, total, stream, max_grid)
                         : launch_directions(&normalise_kernel<kBf16>, a, total, stream, max_grid);
}

}  // namespace la
