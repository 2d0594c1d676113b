// la_norm.hip -- layer norm and RMS norm for gfx950, forward and backward.
//
//   s = x (+ residual, rounded to the type and stored)
//   mean = sum s / n (RMS norm: 0);  r = 1 / sqrt(sum (s - mean)^2 / n + eps)
//   h = (s - mean) r;  y = h w + b
//
//   g = dy w;  a = sum g / n (RMS norm: 0);  c = sum g h / n
//   dx = r (g - a - h c) (+ dsum);  dw = sum over rows of dy h;  db = sum of dy
//
// Memory bounds all of it: forward reads x and writes y once, backward reads
// dy and x and writes dx once. A row is held in the registers of the G lanes
// that share it, so its sums take no second reading; all sums are binary32, the
// variance about the mean that was found first.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "la_device.h"
#include "la_muon.h"
#include "la_norm.h"

#pragma clang fp contract(off)

namespace la {
namespace {

// Eight (four) elements of a parameter as binary32, zeros past the row. The
// type is the same for a whole launch.
template <int N>
__device__ __forceinline__ void load_parameter(float (&to)[N], const void* p, int type, int at,
                                               int cols, float otherwise) {
#pragma unroll
  for (int i = 0; i < N; ++i) to[i] = otherwise;
  if (p == nullptr) return;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (at + i >= cols) continue;
    to[i] = type == kFp32   ? static_cast<const float*>(p)[at + i]
            : type == kFp16 ? Fp16::decode(static_cast<const uint16_t*>(p)[at + i])
                            : Bf16::decode(static_cast<const uint16_t*>(p)[at + i]);
  }
}

__device__ __forceinline__ void store_parameter(void* p, int type, int64_t at, float x) {
  if (type == kFp32) static_cast<float*>(p)[at] = x;
  else static_cast<uint16_t*>(p)[at] = type == kFp16 ? Fp16::encode(x) : Bf16::encode(x);
}

template <typename T>
__device__ __forceinline__ typename T::bits* row_of(const NormRows& t, int64_t row,
                                                    int64_t inner) {
  typename T::bits* p = static_cast<typename T::bits*>(t.p);
  if (inner == 1) return p + row * t.outer_stride;
  // in 32 bits where they suffice: a 64-bit division is a routine
  int64_t i;
  if (row <= 0xffffffffll && inner <= 0xffffffffll)
    i = static_cast<uint32_t>(row) / static_cast<uint32_t>(inner);
  else
    i = row / inner;
  return p + i * t.outer_stride + (row - i * inner) * t.inner_stride;
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

// ---- forward --------------------------------------------------------------------------

template <typename T, int G, int P>
__global__ __launch_bounds__(threads_of<G>()) void forward_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n, groups = threads_of<G>() / G;
  __shared__ float part[2][1][RowSum<G, 1>::waves];
  RowSum<G, 1> row_sum{part};
  const int lane = threadIdx.x % G;
  float w[P][N], b[P][N];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    load_parameter(w[p], a.weight, a.weight_type, (p * G + lane) * N, a.cols, 1.0f);
    load_parameter(b[p], a.bias, a.weight_type, (p * G + lane) * N, a.cols, 0.0f);
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  // every lane of a wave takes part in the exchanges: rows past the end are
  // the last one again, and are not stored
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * groups; first < a.rows; first += step) {
    const int64_t wanted = first + threadIdx.x / G;
    const bool kept = wanted < a.rows;
    const int64_t row = kept ? wanted : a.rows - 1;
    const typename T::bits* x = row_of<T>(a.x, row, a.inner);
    float s[P][N];
    Vector<T> v[P];
#pragma unroll
    for (int p = 0; p < P; ++p) v[p] = load_vector<T>(x, (p * G + lane) * N, a.cols);
    if (a.residual.p != nullptr) {
      const typename T::bits* r = row_of<T>(a.residual, row, a.inner);
      typename T::bits* sum = row_of<T>(a.sum, row, a.inner);
      Vector<T> u[P];
#pragma unroll
      for (int p = 0; p < P; ++p) u[p] = load_vector<T>(r, (p * G + lane) * N, a.cols);
#pragma unroll
      for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[p].e[i] = T::encode(T::decode(v[p].e[i]) + T::decode(u[p].e[i]));
        if (kept) store_vector<T>(sum, (p * G + lane) * N, a.cols, v[p]);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < N; ++i) s[p][i] = T::decode(v[p].e[i]);
    float mean = 0.0f;
    if (a.layer) {
      float t[1] = {0.0f};
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) t[0] += s[p][i];  // zeros past the row
      row_sum(t);
      mean = t[0] * a.inverse_cols;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i)
          s[p][i] = (p * G + lane) * N + i < a.cols ? s[p][i] - mean : 0.0f;
    }
    float t[1] = {0.0f};
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < N; ++i) t[0] += s[p][i] * s[p][i];
    row_sum(t);
    const float rstd = 1.0f / __builtin_sqrtf(t[0] * a.inverse_cols + a.eps);
    if (kept && lane == 0) {
      if (a.layer && a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    typename T::bits* y = row_of<T>(a.y, row, a.inner);
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[p].e[i] = T::encode(s[p][i] * rstd * w[p][i] + b[p][i]);
      if (kept) store_vector<T>(y, (p * G + lane) * N, a.cols, v[p]);
    }
  }
}

// Rows too long for registers: a workgroup reads its row once more for each
// sum and for the result (from L2 while it holds them).
constexpr int kLongThreads = 1024;

template <typename T>
__global__ __launch_bounds__(kLongThreads) void forward_long_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n;
  __shared__ float part[2][1][kLongThreads / 64];
  RowSum<kLongThreads, 1> row_sum{part};
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const typename T::bits* x = row_of<T>(a.x, row, a.inner);
    float t[1] = {0.0f};
    const bool added = a.residual.p != nullptr;
    if (added) {
      const typename T::bits* r = row_of<T>(a.residual, row, a.inner);
      typename T::bits* sum = row_of<T>(a.sum, row, a.inner);
      for (int at = threadIdx.x * N; at < a.cols; at += kLongThreads * N) {
        Vector<T> v = load_vector<T>(x, at, a.cols);
        const Vector<T> u = load_vector<T>(r, at, a.cols);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          v.e[i] = T::encode(T::decode(v.e[i]) + T::decode(u.e[i]));
          t[0] += T::decode(v.e[i]);
        }
        store_vector<T>(sum, at, a.cols, v);
      }
      x = sum;  // a thread reads back what it wrote itself
    } else if (a.layer) {
      for (int at = threadIdx.x * N; at < a.cols; at += kLongThreads * N) {
        const Vector<T> v = load_vector<T>(x, at, a.cols);
#pragma unroll
        for (int i = 0; i < N; ++i) t[0] += T::decode(v.e[i]);
      }
    }
    float mean = 0.0f;
    if (a.layer) {
      row_sum(t);
      mean = t[0] * a.inverse_cols;
    }
    t[0] = 0.0f;
    for (int at = threadIdx.x * N; at < a.cols; at += kLongThreads * N) {
      const Vector<T> v = load_vector<T>(x, at, a.cols);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = at + i < a.cols ? T::decode(v.e[i]) - mean : 0.0f;
        t[0] += d * d;
      }
    }
    row_sum(t);
    const float rstd = 1.0f / __builtin_sqrtf(t[0] * a.inverse_cols + a.eps);
    if (threadIdx.x == 0) {
      if (a.layer && a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    typename T::bits* y = row_of<T>(a.y, row, a.inner);
    for (int at = threadIdx.x * N; at < a.cols; at += kLongThreads * N) {
      Vector<T> v = load_vector<T>(x, at, a.cols);
      float w[N], b[N];
      load_parameter(w, a.weight, a.weight_type, at, a.cols, 1.0f);
      load_parameter(b, a.bias, a.weight_type, at, a.cols, 0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i)
        v.e[i] = T::encode((T::decode(v.e[i]) - mean) * rstd * w[i] + b[i]);
      store_vector<T>(y, at, a.cols, v);
    }
  }
}

// ---- backward -------------------------------------------------------------------------
// A workgroup takes rows_per_part rows one after the other (several at once
// where a row needs fewer lanes), keeps the sums of its columns' dy h and dy in
// registers meanwhile, and leaves them in its part of the workspace; the parts
// are added up in a second launch, always in the same order.

template <typename T, int G, int P, bool BIAS>
__global__ __launch_bounds__(threads_of<G>()) void backward_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n, threads = threads_of<G>(), groups = threads / G;
  constexpr int exchange = groups > 1 ? threads * P * N : 1;
  __shared__ float part[2][2][RowSum<G, 2>::waves];
  __shared__ float lds[exchange];
  RowSum<G, 2> row_sum{part};
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  float w[P][N];
#pragma unroll
  for (int p = 0; p < P; ++p)
    load_parameter(w[p], a.weight, a.weight_type, (p * G + lane) * N, a.cols, 1.0f);
  for (int64_t wg = blockIdx.x; wg < a.parts; wg += gridDim.x) {
    float dw[P][N] = {}, db[BIAS ? P : 1][N] = {};
    const int64_t begin = wg * a.rows_per_part;
    const int64_t end = begin + a.rows_per_part < a.rows ? begin + a.rows_per_part : a.rows;
    for (int64_t first = begin; first < end; first += groups) {
      const int64_t wanted = first + group;
      const bool kept = wanted < end;
      const int64_t row = kept ? wanted : a.rows - 1;
      const typename T::bits* x = row_of<T>(a.x, row, a.inner);
      const typename T::bits* dy = row_of<T>(a.dy, row, a.inner);
      Vector<T> xv[P], dv[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        xv[p] = load_vector<T>(x, (p * G + lane) * N, a.cols);
        dv[p] = load_vector<T>(dy, (p * G + lane) * N, a.cols);
      }
      const float rstd = a.rstd[row], mean = a.layer ? a.mean[row] : 0.0f;
      float t[2] = {0.0f, 0.0f};
      // past the row dy is 0, and with it every term of a sum; a row that is
      // not kept adds nothing to the parameters' sums
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float h = (T::decode(xv[p].e[i]) - mean) * rstd, d = T::decode(dv[p].e[i]);
          const float g = d * w[p][i];
          t[0] += g;
          t[1] += g * h;
          if (kept) {
            dw[p][i] += d * h;
            if constexpr (BIAS) db[p][i] += d;
          }
        }
      row_sum(t);
      const float mean_g = a.layer ? t[0] * a.inverse_cols : 0.0f, mean_gh = t[1] * a.inverse_cols;
      if (a.dx.p != nullptr) {
        typename T::bits* dx = row_of<T>(a.dx, row, a.inner);
        const typename T::bits* ds =
            a.dsum.p != nullptr ? row_of<T>(a.dsum, row, a.inner) : nullptr;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int at = (p * G + lane) * N;
          Vector<T> sv = {}, o;
          if (ds != nullptr) sv = load_vector<T>(ds, at, a.cols);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float h = (T::decode(xv[p].e[i]) - mean) * rstd;
            const float g = T::decode(dv[p].e[i]) * w[p][i];
            float d = rstd * (g - mean_g - h * mean_gh);
            if (ds != nullptr) d += T::decode(sv.e[i]);
            o.e[i] = T::encode(d);
          }
          if (kept) store_vector<T>(dx, at, a.cols, o);
        }
      }
    }
    // the groups' sums meet in LDS, in the order of the groups
    auto leave = [&](float (&sums)[P][N], float* to) {
      if constexpr (groups > 1) {
        __syncthreads();
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < N; ++i) lds[group * (G * P * N) + (p * G + lane) * N + i] = sums[p][i];
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += threads) {
          float s = lds[c];
          for (int g = 1; g < groups; ++g) s += lds[g * (G * P * N) + c];
          to[c] = s;
        }
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < N; ++i)
            if ((p * G + lane) * N + i < a.cols) to[(p * G + lane) * N + i] = sums[p][i];
      }
    };
    if (a.dweight != nullptr) leave(dw, a.partial + wg * a.cols);
    if constexpr (BIAS) leave(db, a.partial + (a.parts + wg) * a.cols);
  }
}

// Rows too long for registers, first their sums, two per row.
template <typename T>
__global__ __launch_bounds__(kLongThreads) void backward_sums_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n;
  __shared__ float part[2][2][kLongThreads / 64];
  RowSum<kLongThreads, 2> row_sum{part};
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const typename T::bits* x = row_of<T>(a.x, row, a.inner);
    const typename T::bits* dy = row_of<T>(a.dy, row, a.inner);
    const float rstd = a.rstd[row], mean = a.layer ? a.mean[row] : 0.0f;
    float t[2] = {0.0f, 0.0f};
    for (int at = threadIdx.x * N; at < a.cols; at += kLongThreads * N) {
      const Vector<T> xv = load_vector<T>(x, at, a.cols), dv = load_vector<T>(dy, at, a.cols);
      float w[N];
      load_parameter(w, a.weight, a.weight_type, at, a.cols, 1.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float g = T::decode(dv.e[i]) * w[i];
        t[0] += g;
        t[1] += g * ((T::decode(xv.e[i]) - mean) * rstd);
      }
    }
    row_sum(t);
    if (threadIdx.x == 0) {
      a.coefficients[2 * row] = a.layer ? t[0] * a.inverse_cols : 0.0f;
      a.coefficients[2 * row + 1] = t[1] * a.inverse_cols;
    }
  }
}

// Then dx and the parts, a workgroup to 256 vectors of columns and one part.
template <typename T>
__global__ __launch_bounds__(256) void backward_long_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n;
  const int blocks = (a.cols + 256 * N - 1) / (256 * N);
  for (int64_t k = blockIdx.x; k < a.parts * blocks; k += gridDim.x) {
    const int64_t wg = k / blocks;
    const int at = (static_cast<int>(k - wg * blocks) * 256 + threadIdx.x) * N;
    if (at >= a.cols) continue;
    const int64_t begin = wg * a.rows_per_part;
    const int64_t end = begin + a.rows_per_part < a.rows ? begin + a.rows_per_part : a.rows;
    float w[N], dw[N] = {}, db[N] = {};
    load_parameter(w, a.weight, a.weight_type, at, a.cols, 1.0f);
    for (int64_t row = begin; row < end; ++row) {
      const Vector<T> xv = load_vector<T>(row_of<T>(a.x, row, a.inner), at, a.cols);
      const Vector<T> dv = load_vector<T>(row_of<T>(a.dy, row, a.inner), at, a.cols);
      const float rstd = a.rstd[row], mean = a.layer ? a.mean[row] : 0.0f;
      const float mean_g = a.coefficients[2 * row], mean_gh = a.coefficients[2 * row + 1];
      Vector<T> o, sv = {};
      if (a.dsum.p != nullptr) sv = load_vector<T>(row_of<T>(a.dsum, row, a.inner), at, a.cols);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float h = (T::decode(xv.e[i]) - mean) * rstd, d = T::decode(dv.e[i]);
        dw[i] += d * h;
        db[i] += d;
        float v = rstd * (d * w[i] - mean_g - h * mean_gh);
        if (a.dsum.p != nullptr) v += T::decode(sv.e[i]);
        o.e[i] = T::encode(v);
      }
      if (a.dx.p != nullptr) store_vector<T>(row_of<T>(a.dx, row, a.inner), at, a.cols, o);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (at + i >= a.cols) continue;
      if (a.dweight != nullptr) a.partial[wg * a.cols + at + i] = dw[i];
      if (a.dbias != nullptr) a.partial[(a.parts + wg) * a.cols + at + i] = db[i];
    }
  }
}

// The parts of a column added up: 32 columns and 32 chains a workgroup.
__global__ __launch_bounds__(1024) void reduce_kernel(NormArgs a) {
  __shared__ float lds[32][33];
  const int c = threadIdx.x & 31, chain = threadIdx.x >> 5;
  const int64_t blocks = (static_cast<int64_t>(a.cols) + 31) / 32;
  for (int64_t k = blockIdx.x; k < 2 * blocks; k += gridDim.x) {
    const bool bias = k >= blocks;
    void* to = bias ? a.dbias : a.dweight;
    if (to == nullptr) continue;
    const int64_t col = (k - (bias ? blocks : 0)) * 32 + c;
    const float* from = a.partial + (bias ? a.parts : 0) * a.cols + col;
    float s = 0.0f;
    if (col < a.cols)
      for (int64_t p = chain; p < a.parts; p += 32) s += from[p * a.cols];
    lds[chain][c] = s;
    __syncthreads();
    if (chain == 0 && col < a.cols) {
      for (int i = 1; i < 32; ++i) s += lds[i][c];
      store_parameter(to, a.grad_type, col, s);
    }
    __syncthreads();
  }
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

// The lanes that share a row and the 16-byte vectors that each of them holds.
template <typename F>
auto with_shape(int64_t bytes, F f) {
  using std::integral_constant;
#define LA_SHAPE(G, P) f(integral_constant<int, G>(), integral_constant<int, P>())
  if (bytes <= 4 * 16) return LA_SHAPE(4, 1);
  if (bytes <= 16 * 16) return LA_SHAPE(16, 1);
  if (bytes <= 64 * 16) return LA_SHAPE(64, 1);
  if (bytes <= 128 * 16) return LA_SHAPE(64, 2);
  if (bytes <= 256 * 16) return LA_SHAPE(256, 1);
  if (bytes <= 512 * 16) return LA_SHAPE(256, 2);
  if (bytes <= 768 * 16) return LA_SHAPE(256, 3);
  if (bytes <= 1024 * 16) return LA_SHAPE(256, 4);
  return LA_SHAPE(512, 4);
#undef LA_SHAPE
}

template <typename T>
hipError_t forward(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  const int64_t bytes = static_cast<int64_t>(a.cols) * T::bytes;
  if (bytes > kNormRegisterBytes)
    return launch(reinterpret_cast<const void*>(&forward_long_kernel<T>), a.rows, kLongThreads, a,
                  stream, max_grid);
  return with_shape(bytes, [&](auto g, auto p) {
    constexpr int G = decltype(g)::value, P = decltype(p)::value, threads = threads_of<G>();
    return launch(reinterpret_cast<const void*>(&forward_kernel<T, G, P>),
                  std::min<int64_t>((a.rows + threads / G - 1) / (threads / G), 2048), threads, a,
                  stream, max_grid);
  });
}

template <typename T>
hipError_t backward(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  const int64_t bytes = static_cast<int64_t>(a.cols) * T::bytes;
  hipError_t e;
  if (bytes > kNormRegisterBytes) {
    e = launch(reinterpret_cast<const void*>(&backward_sums_kernel<T>), a.rows, kLongThreads, a,
               stream, max_grid);
    if (e != hipSuccess) return e;
    const int64_t span = 256 * Vector<T>::n;
    return launch(reinterpret_cast<const void*>(&backward_long_kernel<T>),
                  a.parts * ((a.cols + span - 1) / span), 256, a, stream, max_grid);
  }
  return with_shape(bytes, [&](auto g, auto p) {
    constexpr int G = decltype(g)::value, P = decltype(p)::value;
    return launch(a.dbias != nullptr
                      ? reinterpret_cast<const void*>(&backward_kernel<T, G, P, true>)
                      : reinterpret_cast<const void*>(&backward_kernel<T, G, P, false>),
                  a.parts, threads_of<G>(), a, stream, max_grid);
  });
}

}  // namespace

void norm_parts(int64_t rows, int64_t cols, int type, int64_t* parts, int64_t* rows_per_part) {
  const int64_t bytes = cols * (type == kFp32 ? 4 : 2);
  int64_t together = 1;  // rows that a workgroup takes at once
  if (bytes <= kNormRegisterBytes)
    together = with_shape(bytes, [](auto g, auto) -> int64_t {
      return threads_of<decltype(g)::value>() / decltype(g)::value;
    });
  const int64_t most = 512;
  *rows_per_part = (((rows + most - 1) / most + together - 1) / together) * together;
  if (*rows_per_part < together) *rows_per_part = together;
  *parts = (rows + *rows_per_part - 1) / *rows_per_part;
}

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  return a.type == kFp32   ? forward<Fp32>(a, stream, max_grid)
         : a.type == kFp16 ? forward<Fp16>(a, stream, max_grid)
                           : forward<Bf16>(a, stream, max_grid);
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  if (a.rows > 0) {
    const hipError_t e = a.type == kFp32   ? backward<Fp32>(a, stream, max_grid)
                         : a.type == kFp16 ? backward<Fp16>(a, stream, max_grid)
                                           : backward<Bf16>(a, stream, max_grid);
    if (e != hipSuccess) return e;
  }
  if (a.dweight == nullptr && a.dbias == nullptr) return hipSuccess;
  return launch(reinterpret_cast<const void*>(&reduce_kernel),
                2 * ((static_cast<int64_t>(a.cols) + 31) / 32), 1024, a, stream, max_grid);
}

}  // namespace la
