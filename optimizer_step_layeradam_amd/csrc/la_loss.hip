// la_loss.hip -- the passes over tokens of the linear cross entropy for
// gfx950: gathering the tokens that count, the softmax, the losses.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "la_device.h"
#include "la_loss.h"
#include "la_muon.h"

#pragma clang fp contract(off)

namespace la {
namespace {

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ int64_t target_of(const LossRows& r, int t) {
  return r.wide_targets ? static_cast<const int64_t*>(r.targets)[t]
                        : static_cast<const int32_t*>(r.targets)[t];
}

// ---- gathering ------------------------------------------------------------------------

// Places of the tokens that count, in order: one workgroup, 1024 tokens at a
// time, ranked by ballots.
__global__ __launch_bounds__(1024) void index_kernel(LossRows r) {
  __shared__ int waves[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int before = 0;
  for (int first = 0; first < r.tokens; first += 1024) {
    const int t = first + threadIdx.x;
    const int64_t y = t < r.tokens ? target_of(r, t) : r.ignore_index;
    const bool counts = y != r.ignore_index;
    const uint64_t mask = __ballot(counts);
    if (lane == 0) waves[wave] = __popcll(mask);
    __syncthreads();
    int at = before;
    for (int i = 0; i < 16; ++i) {
      if (i < wave) at += waves[i];
      before += waves[i];
    }
    at += __popcll(mask & ((uint64_t(1) << lane) - 1));
    if (counts) {
      r.index[at] = t;
      r.target[at] = y >= 0 && y < r.vocab ? static_cast<int>(y) : -1;
    } else if (t < r.tokens && r.losses != nullptr) {
      r.losses[t] = 0.0f;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *r.count = before;
}

// Rows of x that count, one after the other, zeros behind each and behind the
// last; dx rows of the others become zeros.
__global__ __launch_bounds__(256) void gather_kernel(LossRows r) {
  const int n = *r.count;
  const int padded = (n + kLossDepth - 1) / kLossDepth * kLossDepth;
  for (int row = blockIdx.x; row < padded; row += gridDim.x) {
    const uint16_t* from = row < n ? r.x + r.index[row] * r.x_stride : r.x;
    const int cols = row < n ? r.hidden : 0;
    uint16_t* to = r.xc + static_cast<int64_t>(row) * r.width;
    for (int at = threadIdx.x * 8; at < r.width; at += 2048) {
      const Vector<Bf16> v = load_vector<Bf16>(from, at, cols);
      store_vector<Bf16>(to, at, r.width, v);
    }
  }
  if (r.dx == nullptr || n == r.tokens) return;
  for (int t = blockIdx.x; t < r.tokens; t += gridDim.x) {
    if (target_of(r, t) != r.ignore_index) continue;
    uint16_t* to = r.dx + t * r.dx_stride;
    const Vector<Bf16> zero = {};
    for (int at = threadIdx.x * 8; at < r.hidden; at += 2048)
      store_vector<Bf16>(to, at, r.hidden, zero);
  }
}

// A copy of rows whose length or alignment the products cannot read: zeros up
// to width.
__global__ __launch_bounds__(256) void pack_kernel(const uint16_t* from, int64_t stride,
                                                   int64_t rows, int cols, uint16_t* to, int width) {
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
    for (int at = threadIdx.x * 8; at < width; at += 2048)
      store_vector<Bf16>(to + row * width, at, width, load_vector<Bf16>(from + row * stride, at, cols));
}

// ---- softmax --------------------------------------------------------------------------

template <int THREADS, typename S>
__device__ __forceinline__ S block_sum(S x) {
  __shared__ S part[THREADS / 64];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d, 64);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  x = part[0];
#pragma unroll
  for (int i = 1; i < THREADS / 64; ++i) x += part[i];
  __syncthreads();
  return x;
}

// The chunks of a row (each its maximum and its sum of exponentials below it)
// joined to lse. A workgroup takes ROWS rows at a time, 1024 / ROWS threads
// to each, whose reads are whole lines where ROWS is 16.
template <int ROWS>
__global__ __launch_bounds__(1024) void lse_kernel(LossRows r) {
  constexpr int SHARES = 1024 / ROWS;
  __shared__ float2 parts[SHARES][ROWS];
  const int n = *r.count;
  const int share = threadIdx.x / ROWS, lane = threadIdx.x % ROWS;
  for (int first = blockIdx.x * ROWS; first < n; first += gridDim.x * ROWS) {
    const int row = min(first + lane, n - 1);
    float most = -__builtin_inff(), sum = 0.0f;
    auto join = [](float& most, float& sum, float2 x) {
      const float top = __builtin_fmaxf(most, x.x);
      // nothing so far, or nothing here: exp(-inf - top) is 0, unless top is too
      const float point = top == -__builtin_inff() ? 0.0f : top;
      sum = sum * __builtin_amdgcn_exp2f((most - point) * kLog2e) +
            x.y * __builtin_amdgcn_exp2f((x.x - point) * kLog2e);
      most = top;
    };
    const float2* sums = r.sums + row;
    int k = share;
    for (; k + 3 * SHARES < r.chunks; k += 4 * SHARES) {
      float2 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = sums[static_cast<int64_t>(k + i * SHARES) * r.tokens];
#pragma unroll
      for (int i = 0; i < 4; ++i) join(most, sum, x[i]);
    }
    for (; k < r.chunks; k += SHARES) join(most, sum, sums[static_cast<int64_t>(k) * r.tokens]);
    parts[share][lane] = make_float2(most, sum);
    __syncthreads();
    for (int step = SHARES / 2; step > 0; step >>= 1) {
      if (share < step) {
        join(most, sum, parts[share + step][lane]);
        parts[share][lane] = make_float2(most, sum);
      }
      __syncthreads();
    }
    if (share == 0 && first + lane < n) {
      // a target outside the vocabulary makes all of its token's results NaN
      const bool outside = r.target[row] < 0;
      const float log_sum = __builtin_logf(sum), nan = __builtin_nanf("");
      const float loss = outside ? nan : (most - r.target_logit[row]) + log_sum;
      r.lse[row] = outside ? nan : most + log_sum;
      r.compact_losses[row] = loss;
      if (r.losses != nullptr) r.losses[r.index[row]] = loss;
    }
    __syncthreads();
  }
}

struct ScaledBf16 : Bf16 {
  static constexpr float encode_scale = 1.0f;
};
struct ScaledFp16 : Fp16 {
  static constexpr float encode_scale = kLossScale;
};

// e of the held piece becomes g, in place: 16 rows of 2048 columns a workgroup.
constexpr int kSoftmaxRows = 16, kSoftmaxCols = 2048;

template <typename T>
__global__ __launch_bounds__(256) void softmax_kernel(LossRows r, LossPiece piece) {
  constexpr float scale = T::encode_scale;
  const int n = *r.count;
  const int padded = (n + kLossDepth - 1) / kLossDepth * kLossDepth;
  const int width = (piece.cols + kLossDepth - 1) / kLossDepth * kLossDepth;
  const int across = (width + kSoftmaxCols - 1) / kSoftmaxCols;
  const int64_t total = static_cast<int64_t>((padded + kSoftmaxRows - 1) / kSoftmaxRows) * across;
  for (int64_t k = blockIdx.x; k < total; k += gridDim.x) {
    const int first = static_cast<int>(k / across) * kSoftmaxRows;
    const int at = static_cast<int>(k % across) * kSoftmaxCols + threadIdx.x * 8;
    if (at >= width) continue;
    const float2* sums = r.sums + static_cast<int64_t>(at >> r.chunk_shift) * r.tokens;
    uint16_t* g = piece.g + static_cast<int64_t>(first) * piece.ld + at;
#pragma unroll 8
    for (int i = 0; i < kSoftmaxRows; ++i) {
      const int row = first + i;  // padded is a multiple of kSoftmaxRows
      Vector<Bf16> o = {};        // rows behind the last one are read as zeros
      if (row < n) {
        Vector<Fp16> e;
        __builtin_memcpy(&e, g + static_cast<int64_t>(i) * piece.ld, 16);
        const float f = __builtin_amdgcn_exp2f((sums[row].x - r.lse[row]) * kLog2e) *
                        (scale / kLossScale);
        const int own = r.target[row] - piece.first - at;
#pragma unroll
        for (int j = 0; j < 8; ++j) o.e[j] = T::encode(Fp16::decode(e.e[j]) * f);
        if (own >= 0 && own < 8) {
          // not 1 - p, whose difference loses what a well predicted token has
          const uint16_t t = T::encode(scale * expm1f(-r.compact_losses[row]));
#pragma unroll
          for (int j = 0; j < 8; ++j) o.e[j] = own == j ? t : o.e[j];
        }
      }
      __builtin_memcpy(g + static_cast<int64_t>(i) * piece.ld, &o, 16);
    }
  }
}

// The loss of all tokens, summed in binary64 in a fixed order.
__global__ __launch_bounds__(1024) void sum_kernel(LossRows r) {
  const int n = *r.count;
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) s += static_cast<double>(r.compact_losses[i]);
  s = block_sum<1024>(s);
  if (threadIdx.x == 0)
    *r.loss = static_cast<float>(r.mean && n > 1 ? s / static_cast<double>(n) : s);
}

// dx of the gathered tokens from the parts of their sums, in order.
template <typename T>
__global__ __launch_bounds__(256) void input_kernel(LossRows r, const float* partial, int splits) {
  const int n = *r.count;
  const float c = (r.mean && n > 1 ? r.scale / static_cast<float>(n) : r.scale) / T::encode_scale;
  const int64_t stride = static_cast<int64_t>(r.tokens) * r.width;
  for (int row = blockIdx.x; row < n; row += gridDim.x) {
    uint16_t* to = r.dx + r.index[row] * r.dx_stride;
    const float* from = partial + static_cast<int64_t>(row) * r.width;
    for (int at = threadIdx.x * 8; at < r.hidden; at += 2048) {
      float s[8] = {};
      for (int k = 0; k < splits; ++k) {
        float v[8];
        __builtin_memcpy(v, from + k * stride + at, 32);  // width is a multiple of 8
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] += v[i];
      }
      Vector<Bf16> o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.e[i] = T::encode(s[i] * c);
      store_vector<Bf16>(to, at, r.hidden, o);
    }
  }
}

template <typename... P>
hipError_t launch(void (*kernel)(P...), int64_t grid, int threads, hipStream_t stream,
                  int64_t max_grid, std::common_type_t<P>... values) {
  grid = std::max<int64_t>(1, std::min({grid, kMaxWorkgroups, max_grid}));
  void* params[] = {&values...};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel),
                         dim3(static_cast<unsigned>(grid)), dim3(threads), params, 0, stream);
}

}  // namespace

hipError_t launch_loss_gather(const LossRows& r, hipStream_t stream, int64_t max_grid) {
  const hipError_t e = launch(index_kernel, 1, 1024, stream, max_grid, r);
  if (e != hipSuccess) return e;
  const int64_t rows = (static_cast<int64_t>(r.tokens) + kLossDepth - 1) / kLossDepth * kLossDepth;
  return launch(gather_kernel, rows, 256, stream, max_grid, r);
}

hipError_t launch_pack(const uint16_t* from, int64_t stride, int64_t rows, int cols, uint16_t* to,
                       int width, hipStream_t stream, int64_t max_grid) {
  return launch(pack_kernel, rows, 256, stream, max_grid, from, stride, rows, cols, to, width);
}

hipError_t launch_loss_lse(const LossRows& r, hipStream_t stream, int64_t max_grid) {
  // few rows: a workgroup to each
  if (r.tokens <= 64) return launch(lse_kernel<1>, r.tokens, 1024, stream, max_grid, r);
  return launch(lse_kernel<16>, (r.tokens + 15) / 16, 1024, stream, max_grid, r);
}

hipError_t launch_loss_softmax(const LossRows& r, const LossPiece& piece, hipStream_t stream,
                               int64_t max_grid) {
  const int64_t rows = (static_cast<int64_t>(r.tokens) + kLossDepth - 1) / kLossDepth * kLossDepth;
  const int64_t grid = rows / kSoftmaxRows *
                       ((static_cast<int64_t>(piece.cols) + kSoftmaxCols - 1) / kSoftmaxCols);
  return launch(r.bf16 ? softmax_kernel<ScaledBf16> : softmax_kernel<ScaledFp16>, grid, 256, stream,
                max_grid, r, piece);
}

hipError_t launch_loss_sum(const LossRows& r, hipStream_t stream) {
  return launch(sum_kernel, 1, 1024, stream, 1, r);
}

hipError_t launch_loss_input(const LossRows& r, const float* partial, int splits,
                             hipStream_t stream, int64_t max_grid) {
  return launch(r.bf16 ? input_kernel<ScaledBf16> : input_kernel<ScaledFp16>, r.tokens, 256,
                stream, max_grid, r, partial, splits);
}

}  // namespace la
