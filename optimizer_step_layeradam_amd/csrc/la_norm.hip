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

#include "la_norm_kernels.h"

namespace la {
namespace {

// ---- forward --------------------------------------------------------------------------

// G lanes to a row, P vectors of 16 bytes to each, the fewest that hold it, and up to
// 2048 workgroups that stride over the rows (1024 or 4096: the same). 8192 BF16
// rows of 5120 with a residual 63 us (5.3 TB/s of 6.6 that a copy reaches), FP32 rows
// of 2560 32 us (5.3), 163840 of 128 16 us (5.1). Without the next row's loads ahead
// of this one's sums, and with branches at the row's end, these took half as long again.
template <typename T, int G, int P, Ends ENDS>
__global__ __launch_bounds__(threads_of<G>()) void forward_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n, groups = threads_of<G>() / G;
  __shared__ float part[2][1][RowSum<G, 1>::waves];
  RowSum<G, 1> row_sum{part};
  const int lane = threadIdx.x % G;
  const int step = gridDim.x * groups;
  const bool added = a.residual.p != nullptr;
  // The next row is asked for before the sums of this one. Every lane of a wave
  // takes part in the exchanges: rows past the end are the last one again, and
  // are not stored.
  u32x4_bits v[P], u[P];
  auto load = [&](int first) {
    const int wanted = first + threadIdx.x / G;
    const int row = wanted < a.rows ? wanted : a.rows - 1;
    const typename T::bits* x = row_of<T, G >= 64>(a.x, row, a.inner);
#pragma unroll
    for (int p = 0; p < P; ++p) v[p] = load_raw<T, ENDS>(x, (p * G + lane) * N, a.cols);
    if (added) {
      const typename T::bits* r = row_of<T, G >= 64>(a.residual, row, a.inner);
#pragma unroll
      for (int p = 0; p < P; ++p) u[p] = load_raw<T, ENDS>(r, (p * G + lane) * N, a.cols);
    }
  };
  int first = blockIdx.x * groups;
  load(first);
  float w[P][N], b[P][N];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    load_parameter<ENDS>(w[p], a.weight, a.weight_type, (p * G + lane) * N, a.cols, 1.0f);
    load_parameter<ENDS>(b[p], a.bias, a.weight_type, (p * G + lane) * N, a.cols, 0.0f);
  }
  for (; first < a.rows; first += step) {
    const int wanted = first + threadIdx.x / G;
    const bool kept = wanted < a.rows;
    const int row = kept ? wanted : a.rows - 1;
    float s[P][N];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = (p * G + lane) * N;
      Vector<T> x = settled<T, ENDS>(v[p], at, a.cols);
      if (added) {
        const Vector<T> r = settled<T, ENDS>(u[p], at, a.cols);
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = T::decode(x.e[i]) + T::decode(r.e[i]);
        x = encode_vector<T>(o);
        if (kept) store_vector<T>(row_of<T, G >= 64>(a.sum, row, a.inner), at, a.cols, x);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) s[p][i] = T::decode(x.e[i]);
    }
    load(first + step < a.rows ? first + step : first);
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
      for (int i = 0; i < N; ++i) t[0] = __builtin_fmaf(s[p][i], s[p][i], t[0]);
    row_sum(t);
    const float rstd = 1.0f / __builtin_sqrtf(t[0] * a.inverse_cols + a.eps);
    if (kept && lane == 0) {
      if (a.layer && a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    typename T::bits* y = row_of<T, G >= 64>(a.y, row, a.inner);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      float o[N];
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = __builtin_fmaf(s[p][i] * rstd, w[p][i], b[p][i]);
      if (kept) store_vector<T>(y, (p * G + lane) * N, a.cols, encode_vector<T>(o));
    }
  }
}

// Rows that fill the registers of 1024 lanes: these hold the row alone, as it
// comes from memory, and the parameters are read where they are needed (from L2).
// What overlaps a row's sums with other rows' loads is a second workgroup, where P is
// 4 at most. The parameters' type is looked at in the loop over vectors, behind which
// each of their loads is waited for before the next is asked for: P waits a row. 4926
// BF16 rows of 16448 109 us, 3.0 TB/s, where reading the row once a sum took 309; 4000
// of 32768 122 us (4.3 TB/s) and 444.
template <typename T, int P, Ends ENDS>
__global__ __launch_bounds__(1024, P <= 4 ? 8 : 4) void forward_wide_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n, G = 1024;
  __shared__ float part[2][1][G / 64];
  RowSum<G, 1> row_sum{part};
  const int lane = threadIdx.x;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const typename T::bits* x = row_of<T, true>(a.x, row, a.inner);
    u32x4_bits v[P];
#pragma unroll
    for (int p = 0; p < P; ++p) v[p] = load_raw<T, ENDS>(x, (p * G + lane) * N, a.cols);
    if (a.residual.p != nullptr) {
      const typename T::bits* r = row_of<T, true>(a.residual, row, a.inner);
      typename T::bits* sum = row_of<T, true>(a.sum, row, a.inner);
      u32x4_bits u[P];
#pragma unroll
      for (int p = 0; p < P; ++p) u[p] = load_raw<T, ENDS>(r, (p * G + lane) * N, a.cols);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int at = formed_again((p * G + lane) * N);
        const Vector<T> xv = settled<T, ENDS>(v[p], at, a.cols);
        const Vector<T> rv = settled<T, ENDS>(u[p], at, a.cols);
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = T::decode(xv.e[i]) + T::decode(rv.e[i]);
        const Vector<T> s = encode_vector<T>(o);
        store_vector<T>(sum, at, a.cols, s);
        v[p] = __builtin_bit_cast(u32x4_bits, s);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int p = 0; p < P; ++p)
        v[p] = __builtin_bit_cast(
            u32x4_bits, settled<T, ENDS>(v[p], formed_again((p * G + lane) * N), a.cols));
    }
    float mean = 0.0f, t[1] = {0.0f};
    if (a.layer) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const Vector<T> s = __builtin_bit_cast(Vector<T>, v[p]);
#pragma unroll
        for (int i = 0; i < N; ++i) t[0] += T::decode(s.e[i]);  // zeros past the row
      }
      row_sum(t);
      mean = t[0] * a.inverse_cols;
    }
    t[0] = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = formed_again((p * G + lane) * N);
      asm("" : "+v"(v[p]));  // decoded again each time: kept, it would be twice the registers
      const Vector<T> s = __builtin_bit_cast(Vector<T>, v[p]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float d = at + i < a.cols ? T::decode(s.e[i]) - mean : 0.0f;
        t[0] = __builtin_fmaf(d, d, t[0]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    row_sum(t);
    const float rstd = 1.0f / __builtin_sqrtf(t[0] * a.inverse_cols + a.eps);
    if (lane == 0) {
      if (a.layer && a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    typename T::bits* y = row_of<T, true>(a.y, row, a.inner);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int at = formed_again((p * G + lane) * N);
      float w[N], b[N], o[N];
      load_parameter<ENDS>(w, a.weight, a.weight_type, at, a.cols, 1.0f);
      load_parameter<ENDS>(b, a.bias, a.weight_type, at, a.cols, 0.0f);
      asm("" : "+v"(v[p]));
      const Vector<T> s = __builtin_bit_cast(Vector<T>, v[p]);
#pragma unroll
      for (int i = 0; i < N; ++i)
        o[i] = __builtin_fmaf((T::decode(s.e[i]) - mean) * rstd, w[i], b[i]);
      store_vector<T>(y, at, a.cols, encode_vector<T>(o));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Rows too long for registers: a workgroup reads its row once more for each
// sum and for the result (from L2 while it holds them: a fifth to a third of what a
// copy reaches; no hidden size is as long, and the loop serves every length).
constexpr int kLongThreads = 1024;

template <typename T>
__global__ __launch_bounds__(kLongThreads) void forward_long_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n;
  __shared__ float part[2][1][kLongThreads / 64];
  RowSum<kLongThreads, 1> row_sum{part};
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const typename T::bits* x = row_of<T, true>(a.x, row, a.inner);
    float t[1] = {0.0f};
    const bool added = a.residual.p != nullptr;
    if (added) {
      const typename T::bits* r = row_of<T, true>(a.residual, row, a.inner);
      typename T::bits* sum = row_of<T, true>(a.sum, row, a.inner);
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
    typename T::bits* y = row_of<T, true>(a.y, row, a.inner);
    for (int at = threadIdx.x * N; at < a.cols; at += kLongThreads * N) {
      Vector<T> v = load_vector<T>(x, at, a.cols);
      float w[N], b[N];
      load_parameter<Ends::kInside>(w, a.weight, a.weight_type, at, a.cols, 1.0f);
      load_parameter<Ends::kInside>(b, a.bias, a.weight_type, at, a.cols, 0.0f);
#pragma unroll
      for (int i = 0; i < N; ++i)
        v.e[i] = T::encode((T::decode(v.e[i]) - mean) * rstd * w[i] + b[i]);
      store_vector<T>(y, at, a.cols, v);
    }
  }
}

// ---- backward -------------------------------------------------------------------------
// Rows too long for registers, first their sums, two per row.
template <typename T>
__global__ __launch_bounds__(kLongThreads) void backward_sums_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n;
  __shared__ float part[2][2][kLongThreads / 64];
  RowSum<kLongThreads, 2> row_sum{part};
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const typename T::bits* x = row_of<T, true>(a.x, row, a.inner);
    const typename T::bits* dy = row_of<T, true>(a.dy, row, a.inner);
    const float rstd = a.rstd[row], mean = a.layer ? a.mean[row] : 0.0f;
    float t[2] = {0.0f, 0.0f};
    for (int at = threadIdx.x * N; at < a.cols; at += kLongThreads * N) {
      const Vector<T> xv = load_vector<T>(x, at, a.cols), dv = load_vector<T>(dy, at, a.cols);
      float w[N];
      load_parameter<Ends::kInside>(w, a.weight, a.weight_type, at, a.cols, 1.0f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float g = T::decode(dv.e[i]) * w[i];
        t[0] += g;
        t[1] += g * ((T::decode(xv.e[i]) - mean) * rstd);
      }
    }
    row_sum(t);
    if (threadIdx.x == 0) {
      a.coefficients[2 * static_cast<int64_t>(row)] = a.layer ? t[0] * a.inverse_cols : 0.0f;
      a.coefficients[2 * static_cast<int64_t>(row) + 1] = t[1] * a.inverse_cols;
    }
  }
}

// Then dx and the parts, a workgroup to 256 vectors of columns and one part.
template <typename T>
__global__ __launch_bounds__(256) void backward_long_kernel(NormArgs a) {
  constexpr int N = Vector<T>::n;
  const int blocks = (a.cols + 256 * N - 1) / (256 * N);
  for (int k = blockIdx.x; k < a.parts * blocks; k += gridDim.x) {
    const int wg = k / blocks;
    const int at = ((k - wg * blocks) * 256 + threadIdx.x) * N;
    if (at >= a.cols) continue;
    const int begin = wg * a.rows_per_part;
    const int end = begin + min(a.rows_per_part, a.rows - begin);
    float w[N], dw[N] = {}, db[N] = {};
    load_parameter<Ends::kInside>(w, a.weight, a.weight_type, at, a.cols, 1.0f);
    for (int row = begin; row < end; ++row) {
      const Vector<T> xv = load_vector<T>(row_of<T, true>(a.x, row, a.inner), at, a.cols);
      const Vector<T> dv = load_vector<T>(row_of<T, true>(a.dy, row, a.inner), at, a.cols);
      const float rstd = a.rstd[row], mean = a.layer ? a.mean[row] : 0.0f;
      const float* coefficients = a.coefficients + 2 * static_cast<int64_t>(row);
      const float mean_g = coefficients[0], mean_gh = coefficients[1];
      Vector<T> o, sv = {};
      if (a.dsum.p != nullptr)
        sv = load_vector<T>(row_of<T, true>(a.dsum, row, a.inner), at, a.cols);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float h = (T::decode(xv.e[i]) - mean) * rstd, d = T::decode(dv.e[i]);
        dw[i] += d * h;
        db[i] += d;
        float v = rstd * (d * w[i] - mean_g - h * mean_gh);
        if (a.dsum.p != nullptr) v += T::decode(sv.e[i]);
        o.e[i] = T::encode(v);
      }
      if (a.dx.p != nullptr) store_vector<T>(row_of<T, true>(a.dx, row, a.inner), at, a.cols, o);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (at + i >= a.cols) continue;
      if (a.dweight != nullptr) a.partial[static_cast<int64_t>(wg) * a.cols + at + i] = dw[i];
      if (a.dbias != nullptr)
        a.partial[static_cast<int64_t>(a.parts + wg) * a.cols + at + i] = db[i];
    }
  }
}

// The parts of a column added up: 32 columns and 32 chains a workgroup, whose
// sums 32 lanes then exchange. Latency bounds it: 4 to 5 us for 512 parts of 4096
// columns (8 MB), as for two of 1027.
__global__ __launch_bounds__(1024) void reduce_kernel(NormArgs a) {
  __shared__ float lds[32][33];
  const int c = threadIdx.x & 31, chain = threadIdx.x >> 5;
  const int blocks = (a.cols + 31) / 32;
  for (int k = blockIdx.x; k < 2 * blocks; k += gridDim.x) {
    const bool bias = k >= blocks;
    void* to = bias ? a.dbias : a.dweight;
    if (to == nullptr) continue;
    const int first = (k - (bias ? blocks : 0)) * 32, col = first + c;
    const float* from = a.partial + static_cast<int64_t>(bias ? a.parts : 0) * a.cols + col;
    float s = 0.0f;
    if (col < a.cols)
#pragma unroll 8
      for (int p = chain; p < a.parts; p += 32) s += from[static_cast<int64_t>(p) * a.cols];
    lds[chain][c] = s;
    __syncthreads();
    s = lds[c][chain];  // lane c of column `chain`
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor(s, d, 64);
    if (c == 0 && first + chain < a.cols) store_parameter(to, a.grad_type, first + chain, s);
    __syncthreads();
  }
}

// ---- launches -------------------------------------------------------------------------

template <typename T>
hipError_t forward(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  const int64_t bytes = static_cast<int64_t>(a.cols) * T::bytes;
  if (a.cols > kNormWideCols)
    return launch(reinterpret_cast<const void*>(&forward_long_kernel<T>), a.rows, kLongThreads, a,
                  stream, max_grid);
  if (bytes > kNormRegisterBytes)
    return with_wide_shape<T>(bytes, [&](auto p, auto ends) {
      return launch(reinterpret_cast<const void*>(
                        &forward_wide_kernel<T, decltype(p)::value, decltype(ends)::value>),
                    a.rows, 1024, a, stream, max_grid);
    });
  return with_shape(bytes, [&](auto g, auto p, auto ends) {
    constexpr int G = decltype(g)::value, P = decltype(p)::value, threads = threads_of<G>();
    return launch(reinterpret_cast<const void*>(&forward_kernel<T, G, P, decltype(ends)::value>),
                  std::min<int64_t>(
                      (static_cast<int64_t>(a.rows) + threads / G - 1) / (threads / G), 2048),
                  threads, a, stream, max_grid);
  });
}

template <typename T>
hipError_t backward(const NormArgs& a, hipStream_t stream, int64_t max_grid,
                    decltype(norm_backward_fp32)* rows) {
  if (a.cols > kNormWideCols) {
    const hipError_t e = launch(reinterpret_cast<const void*>(&backward_sums_kernel<T>), a.rows,
                                kLongThreads, a, stream, max_grid);
    if (e != hipSuccess) return e;
    const int64_t span = 256 * Vector<T>::n;
    return launch(reinterpret_cast<const void*>(&backward_long_kernel<T>),
                  static_cast<int64_t>(a.parts) * ((a.cols + span - 1) / span), 256, a, stream,
                  max_grid);
  }
  return rows(a, stream, max_grid);
}

}  // namespace

NormParts norm_parts(int64_t rows, int64_t cols, int type) {
  const int64_t bytes = cols * (type == kFp32 ? 4 : 2);
  // A few workgroups to each compute unit, so that each row's loads are under way
  // beside other rows' work: four, two or one by what a lane holds. That is what the
  // backward kernel's registers allow at once, but in two places. At two vectors a
  // lane three would fit, and take longer (32768 rows of 4096: 512 parts 171 us, 768
  // of them 189; not explained). 16-bit rows of 6145 to 8192 elements take more than 256
  // registers with a bias or a residual's gradient, or where they end inside a vector,
  // so that one workgroup fits and the two run one after the other (8192 x 8192 with a
  // residual's gradient 116 us, 4.6 TB/s, as at 5120). Each takes four rows at least, for
  // the sake of the sum over the parts, but where a row fills a compute unit: 50 rows of
  // 32768 took 67 us by four and take 25 one by one.
  int64_t together = 1, each_unit = 2, least = 4;  // together: rows taken at once
  if (cols > kNormWideCols) {
  } else if (bytes > kNormRegisterBytes) {
    each_unit = least = 1;
  } else {
    with_shape(bytes, [&](auto g, auto p, auto) {
      constexpr int G = decltype(g)::value, P = decltype(p)::value;
      together = threads_of<G>() / G;
      each_unit = G > 256 ? 1 : P == 1 ? 4 : 2;
      return 0;
    });
  }
  const int64_t most = 256 * each_unit;
  auto parts_of = [&](int64_t each) { return (rows + each - 1) / each; };
  const int64_t fewest = (least + together - 1) / together * together;
  const int64_t share = (parts_of(most) + together - 1) / together * together;
  const int64_t each = std::max(fewest, share);
  return {static_cast<int32_t>(parts_of(each)), static_cast<int32_t>(each),
          static_cast<int32_t>(std::min(most, parts_of(fewest)))};
}

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  return a.type == kFp32   ? forward<Fp32>(a, stream, max_grid)
         : a.type == kFp16 ? forward<Fp16>(a, stream, max_grid)
                           : forward<Bf16>(a, stream, max_grid);
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  if (a.rows > 0) {
    const hipError_t e = a.type == kFp32   ? backward<Fp32>(a, stream, max_grid, norm_backward_fp32)
                         : a.type == kFp16 ? backward<Fp16>(a, stream, max_grid, norm_backward_fp16)
                                           : backward<Bf16>(a, stream, max_grid, norm_backward_bf16);
    if (e != hipSuccess) return e;
  }
  if (a.dweight == nullptr && a.dbias == nullptr) return hipSuccess;
  return launch(reinterpret_cast<const void*>(&reduce_kernel),
                2 * ((static_cast<int64_t>(a.cols) + 31) / 32), 1024, a, stream, max_grid);
}

}  // namespace la
