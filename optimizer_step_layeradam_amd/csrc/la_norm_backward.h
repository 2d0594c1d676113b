// The backward pass over rows that fit registers, for one element type; each of
// the la_norm_backward_*.hip holds one, so that they compile side by side.
//
// A workgroup takes rows_per_part rows one after the other (several at once
// where a row needs fewer lanes), keeps the sums of its columns' dy h and dy in
// registers meanwhile, and leaves them in its part of the workspace; the parts
// are added up in a second launch, always in the same order.
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
          for (int i = 0; i < N; ++i)
            if ((p * G + lane) * N + i < a.cols) to[(p * G + lane) * N + i] = sums[p][i];
      }
    };
    if (a.dweight != nullptr) leave(dw, a.partial + static_cast<int64_t>(wg) * a.cols);
    if constexpr (BIAS) leave(db, a.partial + static_cast<int64_t>(a.parts + wg) * a.cols);
  }
}

template <typename T>
hipError_t backward_rows(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  return with_shape(static_cast<int64_t>(a.cols) * T::bytes, [&](auto g, auto p, auto ends) {
    constexpr int G = decltype(g)::value, P = decltype(p)::value;
    constexpr Ends ENDS = decltype(ends)::value;
    const bool bias = a.dbias != nullptr, added = a.dsum.p != nullptr;
    const void* kernel =
        bias ? added ? reinterpret_cast<const void*>(&backward_kernel<T, G, P, true, true, ENDS>)
                     : reinterpret_cast<const void*>(&backward_kernel<T, G, P, true, false, ENDS>)
        : added ? reinterpret_cast<const void*>(&backward_kernel<T, G, P, false, true, ENDS>)
                : reinterpret_cast<const void*>(&backward_kernel<T, G, P, false, false, ENDS>);
    return launch(kernel, a.parts, threads_of<G>(), a, stream, max_grid);
  });
}

}  // namespace
}  // namespace la
