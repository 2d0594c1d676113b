// The backward pass over rows that fit registers, for one element type; each of
// the la_norm_backward_*.hip holds one, so that they compile side by side.
//
// A workgroup takes rows_per_part rows one after the other (several at once
// where a row needs fewer lanes), keeps the sums of its columns' dy h and dy in
// registers meanwhile, and leaves them in its part of the workspace; the parts
// are added up in a second launch, always in the same order.
//
// Memory bounds it, two or three streams read and one written: 32768 BF16 rows of
// 4096 161 us (5.0 TB/s), 8192 of 5120 with a residual's gradient 73 (4.6), FP32 rows of 2560
// 46 (5.5), 163840 of 128 24 (5.2). Registers decide how much of it is under way:
// h and dy w are formed twice, from the row as it came from memory. Rows of 16 to 32 KB
// fill 1024 lanes' 128 registers with their columns' sums and the weight beside them:
// nothing of the next row is under way, and 16-bit ones leave 12 to 92 bytes a lane in
// scratch, up to 228 where they end inside a vector (8192 x 12288 132 us, 4.6 TB/s, with a
// residual's gradient and a bias 231, 3.5).
#pragma once

#include "la_norm_kernels.h"

namespace la {
namespace {

// What a lane reads of a row.
template <int P, bool ADDED>
struct BackwardRow {
  u32x4_bits x[P], dy[P], dsum[ADDED ? P : 1];
  float rstd, mean;
};

// Columns [at, at + 4) of a part.
template <typename V>
__device__ __forceinline__ void leave_four(float* to, int at, int cols, const V& sums) {
  if (at + 4 <= cols) {
    __builtin_memcpy(to + at, &sums, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (at + i < cols) to[at + i] = sums[i];
  }
}

template <typename T, int G, int P, bool BIAS, bool ADDED, Ends ENDS>
__global__ __launch_bounds__(threads_of<G>()) void backward_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n, threads = threads_of<G>(), groups = threads / G;
  constexpr int exchange = groups > 1 ? threads * P * N : 1;
  constexpr bool AHEAD = G * P <= 1024;  // beyond, registers are short
  __shared__ float part[2][2][RowSum<G, 2>::waves];
  __shared__ float lds[exchange];
  RowSum<G, 2> row_sum{part};
  using Row = BackwardRow<P, ADDED>;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  auto load = [&](Row& to, int first, int end) {
    const int row = first + group < end ? first + group : end - 1;
    const typename T::bits* x = row_of<T, G >= 64>(a.x, row, a.inner);
    const typename T::bits* dy = row_of<T, G >= 64>(a.dy, row, a.inner);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      to.x[p] = load_raw<T, ENDS>(x, (p * G + lane) * N, a.cols);
      to.dy[p] = load_raw<T, ENDS>(dy, (p * G + lane) * N, a.cols);
    }
    if constexpr (ADDED) {
      const typename T::bits* ds = row_of<T, G >= 64>(a.dsum, row, a.inner);
#pragma unroll
      for (int p = 0; p < P; ++p) to.dsum[p] = load_raw<T, ENDS>(ds, (p * G + lane) * N, a.cols);
    }
    to.rstd = a.rstd[row];
    to.mean = a.layer ? a.mean[row] : 0.0f;
  };
  for (int wg = blockIdx.x; wg < a.parts; wg += gridDim.x) {
    float dw[P][N] = {}, db[BIAS ? P : 1][N] = {}, w[P][N];
    const int begin = wg * a.rows_per_part;
    const int end = begin + min(a.rows_per_part, a.rows - begin);
    // Rows `first` on are in `now`; the next ones are asked for, into `next`,
    // before the sums of these.
    auto work = [&](Row& now, Row& next, int first) {
      const bool kept = first + group < end;
      const int row = kept ? first + group : end - 1;
      if constexpr (AHEAD) load(next, first + groups, end);
      else load(now, first, end);
      const float rstd = now.rstd, mean = now.mean;
      float t[2] = {0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * G + lane) * N;
        // past the row dy is 0, and with it every term of a sum
        const Vector<T> xv = settled<T, ENDS>(now.x[p], at, a.cols);
        const Vector<T> dv = settled<T, ENDS>(now.dy[p], at, a.cols);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float h = (T::decode(xv.e[i]) - mean) * rstd, g = T::decode(dv.e[i]) * w[p][i];
          t[0] += g;
          t[1] = __builtin_fmaf(g, h, t[1]);
        }
        __builtin_amdgcn_sched_barrier(0);  // a vector at a time: registers decide
      }
      row_sum(t);
      const float mean_g = a.layer ? t[0] * a.inverse_cols : 0.0f, mean_gh = t[1] * a.inverse_cols;
      typename T::bits* dx = row_of<T, G >= 64>(a.dx, row, a.inner);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = (p * G + lane) * N;
        // h and g are formed again: kept, they would take twice the registers
        // of what they come from, and the compiler is not to know
        asm("" : "+v"(now.x[p]), "+v"(now.dy[p]));
        const Vector<T> xv = settled<T, ENDS>(now.x[p], at, a.cols);
        const Vector<T> dv = settled<T, ENDS>(now.dy[p], at, a.cols);
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float h = (T::decode(xv.e[i]) - mean) * rstd, d = T::decode(dv.e[i]);
          const float g = d * w[p][i];
          o[i] = rstd * __builtin_fmaf(-h, mean_gh, g - mean_g);
          if constexpr (groups > 1) {  // a row that is not kept adds nothing
            d = kept ? d : 0.0f;
            h = kept ? h : 0.0f;
          }
          dw[p][i] = __builtin_fmaf(d, h, dw[p][i]);
          if constexpr (BIAS) db[p][i] += d;
          // here, and not behind the stores, until when h and d would be kept
          asm volatile("" : "+v"(dw[p][i]));
          if constexpr (BIAS) asm volatile("" : "+v"(db[p][i]));
        }
        if constexpr (ADDED) {
          const Vector<T> sv = settled<T, ENDS>(now.dsum[p], at, a.cols);
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] += T::decode(sv.e[i]);
        }
        if (kept && a.dx.p != nullptr) store_vector<T>(dx, at, a.cols, encode_vector<T>(o));
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    Row one, other;
    if constexpr (AHEAD) load(one, begin, end);
#pragma unroll
    for (int p = 0; p < P; ++p)
      load_parameter<ENDS>(w[p], a.weight, a.weight_type, (p * G + lane) * N, a.cols, 1.0f);
    for (int first = begin; first < end; first += 2 * groups) {
      work(one, other, first);
      if (first + groups < end) work(other, one, first + groups);
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
          for (int i = 0; i < N; i += 4) {
            const float four[4] = {sums[p][i], sums[p][i + 1], sums[p][i + 2], sums[p][i + 3]};
            leave_four(to, (p * G + lane) * N + i, a.cols, four);
          }
      }
    };
    if (a.dweight != nullptr) leave(dw, a.partial + static_cast<int64_t>(wg) * a.cols);
    if constexpr (BIAS) leave(db, a.partial + static_cast<int64_t>(a.parts + wg) * a.cols);
  }
}

// Rows that fill the registers of 1024 lanes: x and dy as they come from memory
// and the sums of dy are there, those of dy h in LDS (read and written
// once a row, by the lane whose columns they are), and w is read twice (from L2).
// 4926 BF16 rows of 16448 182 us (2.7 TB/s), 4000 of 32768 220 (3.6), where two
// launches that each read x and dy took 380 and 583; rows of 16 to 32 KB are better off
// above (8192 of 12288: 145 us, here 202). As in the forward pass each vector's
// parameters, and its part of dsum, are waited for before the next vector's are asked
// for: 2 P to 3 P waits a row.
template <typename T, int P, bool BIAS, bool ADDED, Ends ENDS>
__global__ __launch_bounds__(1024) void backward_wide_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n, G = 1024;
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  __shared__ float part[2][2][G / 64];
  __shared__ f32x4 dw[P * N / 4][G];
  RowSum<G, 2> row_sum{part};
  const int lane = threadIdx.x;
  for (int wg = blockIdx.x; wg < a.parts; wg += gridDim.x) {
    float db[BIAS ? P : 1][N] = {};
#pragma unroll
    for (int i = 0; i < P * N / 4; ++i) dw[i][lane] = f32x4{};
    const int begin = wg * a.rows_per_part;
    const int end = begin + min(a.rows_per_part, a.rows - begin);
    for (int row = begin; row < end; ++row) {
      const typename T::bits* x = row_of<T, true>(a.x, row, a.inner);
      const typename T::bits* dy = row_of<T, true>(a.dy, row, a.inner);
      u32x4_bits xr[P], dr[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = formed_again((p * G + lane) * N);
        xr[p] = load_raw<T, ENDS>(x, at, a.cols);
        dr[p] = load_raw<T, ENDS>(dy, at, a.cols);
      }
      const float rstd = a.rstd[row], mean = a.layer ? a.mean[row] : 0.0f;
      float t[2] = {0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = formed_again((p * G + lane) * N);
        float w[N];
        load_parameter<ENDS>(w, a.weight, a.weight_type, at, a.cols, 1.0f);
        // past the row dy is 0, and with it every term of a sum
        const Vector<T> xv = settled<T, ENDS>(xr[p], at, a.cols);
        const Vector<T> dv = settled<T, ENDS>(dr[p], at, a.cols);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float h = (T::decode(xv.e[i]) - mean) * rstd, g = T::decode(dv.e[i]) * w[i];
          t[0] += g;
          t[1] = __builtin_fmaf(g, h, t[1]);
        }
        __builtin_amdgcn_sched_barrier(0);  // a vector at a time: registers decide
      }
      row_sum(t);
      const float mean_g = a.layer ? t[0] * a.inverse_cols : 0.0f, mean_gh = t[1] * a.inverse_cols;
      typename T::bits* dx = row_of<T, true>(a.dx, row, a.inner);
      const typename T::bits* ds = ADDED ? row_of<T, true>(a.dsum, row, a.inner) : nullptr;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = formed_again((p * G + lane) * N);
        u32x4_bits sr = {};
        if constexpr (ADDED) sr = load_raw<T, ENDS>(ds, at, a.cols);
        float w[N];
        load_parameter<ENDS>(w, a.weight, a.weight_type, at, a.cols, 1.0f);
        asm("" : "+v"(xr[p]), "+v"(dr[p]));
        const Vector<T> xv = settled<T, ENDS>(xr[p], at, a.cols);
        const Vector<T> dv = settled<T, ENDS>(dr[p], at, a.cols);
        float o[N];
#pragma unroll
        for (int j = 0; j < N / 4; ++j) {
          f32x4 s = dw[p * N / 4 + j][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 4 * j + e;
            const float h = (T::decode(xv.e[i]) - mean) * rstd, d = T::decode(dv.e[i]);
            o[i] = rstd * __builtin_fmaf(-h, mean_gh, d * w[i] - mean_g);
            s[e] = __builtin_fmaf(d, h, s[e]);
            if constexpr (BIAS) db[p][i] += d;
          }
          dw[p * N / 4 + j][lane] = s;
        }
        if constexpr (ADDED) {
          const Vector<T> sv = settled<T, ENDS>(sr, at, a.cols);
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] += T::decode(sv.e[i]);
        }
        if (a.dx.p != nullptr) store_vector<T>(dx, at, a.cols, encode_vector<T>(o));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    float* const to = a.partial + static_cast<int64_t>(wg) * a.cols;
    float* const to_bias = a.partial + static_cast<int64_t>(a.parts + wg) * a.cols;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = formed_again((p * G + lane) * N);
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        if (a.dweight != nullptr) leave_four(to, at + i, a.cols, dw[(p * N + i) / 4][lane]);
        if constexpr (BIAS) {
          const f32x4 four = {db[p][i], db[p][i + 1], db[p][i + 2], db[p][i + 3]};
          leave_four(to_bias, at + i, a.cols, four);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

template <typename T>
hipError_t backward_rows(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  const int64_t bytes = static_cast<int64_t>(a.cols) * T::bytes;
  const bool bias = a.dbias != nullptr, added = a.dsum.p != nullptr;
  auto with = [&](auto kernel, int threads) {
    using std::false_type;
    using std::true_type;
    return launch(bias ? added ? kernel(true_type(), true_type()) : kernel(true_type(), false_type())
                  : added ? kernel(false_type(), true_type())
                          : kernel(false_type(), false_type()),
                  a.parts, threads, a, stream, max_grid);
  };
  if (bytes > kNormRegisterBytes)
    return with_wide_shape<T>(bytes, [&](auto p, auto ends) {
      return with(
          [&](auto b, auto d) {
            return reinterpret_cast<const void*>(
                &backward_wide_kernel<T, decltype(p)::value, decltype(b)::value,
                                      decltype(d)::value, decltype(ends)::value>);
          },
          1024);
    });
  return with_shape(bytes, [&](auto g, auto p, auto ends) {
    constexpr int G = decltype(g)::value;
    return with(
        [&](auto b, auto d) {
          return reinterpret_cast<const void*>(
              &backward_kernel<T, G, decltype(p)::value, decltype(b)::value, decltype(d)::value,
                               decltype(ends)::value>);
        },
        threads_of<G>());
  });
}

}  // namespace
}  // namespace la
