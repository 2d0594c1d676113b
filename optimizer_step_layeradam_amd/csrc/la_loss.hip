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
    uint16_t* to = r.xc + static_cast<int64_t>(row) * r.ldx;
    for (int at = threadIdx.x * 8; at < r.ldx; at += 2048) {
      const Vector<Bf16> v = load_vector<Bf16>(from, at, cols);
      store_vector<Bf16>(to, at, r.ldx, v);
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
// to ld.
__global__ __launch_bounds__(256) void pack_kernel(const uint16_t* from, int64_t stride,
                                                   int64_t rows, int cols, uint16_t* to, int ld) {
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
    for (int at = threadIdx.x * 8; at < ld; at += 2048)
      store_vector<Bf16>(to + row * ld, at, ld, load_vector<Bf16>(from + row * stride, at, cols));
}

// ---- softmax --------------------------------------------------------------------------

template <int THREADS>
__device__ __forceinline__ float block_max(float x) {
  __shared__ float part[THREADS / 64];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x = __builtin_fmaxf(x, __shfl_xor(x, d, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  x = part[0];
#pragma unroll
  for (int i = 1; i < THREADS / 64; ++i) x = __builtin_fmaxf(x, part[i]);
  __syncthreads();
  return x;
}

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

constexpr int kSoftmaxThreads = 256;

// A workgroup joins its row's chunks (each its maximum and its sum of
// exponentials below it) to lse, then turns its share of e into g. Where a row
// has several workgroups each joins the chunks again: they are few beside e.
template <typename T, bool PIECE>
__global__ __launch_bounds__(kSoftmaxThreads) void softmax_kernel(LossRows r, LossPiece piece,
                                                                  int shares) {
  const int n = *r.count;
  const int padded = PIECE ? (n + kLossDepth - 1) / kLossDepth * kLossDepth : n;
  const int width = PIECE ? (piece.cols + kLossDepth - 1) / kLossDepth * kLossDepth : 0;
  const int share = ((width / 8 + shares - 1) / shares + 255) / 256 * 256;  // vectors
  for (int64_t k = blockIdx.x; k < static_cast<int64_t>(padded) * shares; k += gridDim.x) {
    const int row = static_cast<int>(k / shares), part = static_cast<int>(k - static_cast<int64_t>(row) * shares);
    uint16_t* g = PIECE ? piece.g + static_cast<int64_t>(row) * piece.ld : nullptr;
    const int begin = part * share * 8, end = min(width, begin + share * 8);
    if (row >= n) {  // rows behind the last one are read as zeros
      const Vector<Bf16> zero = {};
      if constexpr (PIECE)
        for (int at = begin + threadIdx.x * 8; at < end; at += kSoftmaxThreads * 8)
          store_vector<Bf16>(g, at, end, zero);
      continue;
    }
    const float2* sums = r.sums + static_cast<int64_t>(row) * r.chunks;
    float most = -__builtin_inff();
    for (int i = threadIdx.x; i < r.chunks; i += kSoftmaxThreads)
      most = __builtin_fmaxf(most, sums[i].x);
    most = block_max<kSoftmaxThreads>(most);
    float sum = 0.0f;
    for (int i = threadIdx.x; i < r.chunks; i += kSoftmaxThreads)
      sum += sums[i].y * __builtin_amdgcn_exp2f((sums[i].x - most) * kLog2e);
    sum = block_sum<kSoftmaxThreads>(sum);
    const int target = r.target[row];
    const float log_sum = __builtin_logf(sum);
    // a target outside the vocabulary makes all of its token's results NaN
    const float loss = target < 0 ? __builtin_nanf("")
                                  : (most - r.target_logit[row]) + log_sum;
    if (part == 0 && threadIdx.x == 0) {
      r.lse[row] = target < 0 ? __builtin_nanf("") : most + log_sum;
      r.compact_losses[row] = loss;
      if (r.losses != nullptr) r.losses[r.index[row]] = loss;
    }
    if constexpr (PIECE) {
      constexpr float scale = T::encode_scale;
      const float inverse = target < 0 ? loss : scale / (sum * kLossScale);
      const int own = target - piece.first;
      // not 1 - p, whose difference loses what a well predicted token has
      const float at_target = scale * expm1f(-loss);
      for (int at = begin + threadIdx.x * 8; at < end; at += kSoftmaxThreads * 8) {
        const Vector<Fp16> e = load_vector<Fp16>(g, at, end);
        const float f =
            __builtin_amdgcn_exp2f((sums[at >> r.chunk_shift].x - most) * kLog2e) * inverse;
        Vector<Bf16> o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = Fp16::decode(e.e[i]) * f;
          o.e[i] = T::encode(at + i == own ? at_target : p);
        }
        store_vector<Bf16>(g, at, end, o);
      }
    }
  }
}

struct ScaledBf16 : Bf16 {
  static constexpr float encode_scale = 1.0f;
};
struct ScaledFp16 : Fp16 {
  static constexpr float encode_scale = kLossScale;
};

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
  const int64_t stride = static_cast<int64_t>(r.tokens) * r.ldx;
  for (int row = blockIdx.x; row < n; row += gridDim.x) {
    uint16_t* to = r.dx + r.index[row] * r.dx_stride;
    const float* from = partial + static_cast<int64_t>(row) * r.ldx;
    for (int at = threadIdx.x * 8; at < r.hidden; at += 2048) {
      float s[8] = {};
      for (int k = 0; k < splits; ++k) {
        float v[8];
        __builtin_memcpy(v, from + k * stride + at, 32);  // ldx is a multiple of 8
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
                       int ld, hipStream_t stream, int64_t max_grid) {
  return launch(pack_kernel, rows, 256, stream, max_grid, from, stride, rows, cols, to, ld);
}

hipError_t launch_loss_softmax(const LossRows& r, const LossPiece* piece, hipStream_t stream,
                               int64_t max_grid) {
  const int64_t rows = std::max<int64_t>(
      1, (static_cast<int64_t>(r.tokens) + kLossDepth - 1) / kLossDepth * kLossDepth);
  // about 2048 workgroups, of at least 4096 columns each
  const int64_t width = piece != nullptr ? piece->cols : 0;
  const int shares = static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>((2048 + rows - 1) / rows, width / 4096)));
  const LossPiece p = piece != nullptr ? *piece : LossPiece{};
  if (piece == nullptr)
    return launch(softmax_kernel<ScaledBf16, false>, rows, kSoftmaxThreads, stream, max_grid, r, p,
                  1);
  return launch(r.bf16 ? softmax_kernel<ScaledBf16, true> : softmax_kernel<ScaledFp16, true>,
                rows * shares, kSoftmaxThreads, stream, max_grid, r, p, shares);
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
