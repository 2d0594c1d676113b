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
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *r.count = before;
}

// A token that does not count: its loss and its dx.
__device__ __forceinline__ void clear_token(const LossRows& r, int t) {
  if (threadIdx.x == 0 && r.losses != nullptr) r.losses[t] = 0.0f;
  if (r.dx == nullptr) return;
  const Vector<Bf16> zero = {};
  for (int at = threadIdx.x * 8; at < r.hidden; at += 2048)
    store_vector<Bf16>(r.dx + t * r.dx_stride, at, r.hidden, zero);
}

// Row `row` of the gathered x: token t's, zeros behind it; t < 0: zeros.
__device__ __forceinline__ void gather_row(const LossRows& r, int row, int t) {
  const uint16_t* from = t < 0 ? r.x : r.x + t * r.x_stride;
  uint16_t* to = r.xc + static_cast<int64_t>(row) * r.width;
  for (int at = threadIdx.x * 8; at < r.width; at += 2048)
    store_vector<Bf16>(to, at, r.width, load_vector<Bf16>(from, at, t < 0 ? 0 : r.hidden));
}

// Rows of x that count, one after the other, zeros behind the last up to a
// whole depth. (A copy, where the products could read through the index: theirs would
// be scattered rows in every tile. 8192 x 5120: 45 us of 30 ms, 3.7 TB/s; the index
// before it 11 us.)
__global__ __launch_bounds__(256) void gather_kernel(LossRows r) {
  const int n = *r.count;
  const int padded = (n + kLossDepth - 1) / kLossDepth * kLossDepth;
  for (int row = blockIdx.x; row < padded; row += gridDim.x)
    gather_row(r, row, row < n ? r.index[row] : -1);
  if (n == r.tokens || (r.dx == nullptr && r.losses == nullptr)) return;
  for (int t = blockIdx.x; t < r.tokens; t += gridDim.x)
    if (target_of(r, t) == r.ignore_index) clear_token(r, t);
}

// Both in one launch where there are few tokens: every workgroup counts all
// targets, those before its own token apart. Workgroups past the tokens fill
// the last depth. (1 token 3.3 us, 1003 tokens 8.3: all targets are read by each
// workgroup, from L2. The two launches take 7 and 15 us at 4096.)
constexpr int kCountedTokens = 2048;

__global__ __launch_bounds__(256) void index_gather_kernel(LossRows r) {
  __shared__ int parts[2][4];
  for (int t = blockIdx.x; t < r.tokens + kLossDepth; t += gridDim.x) {
    int before = 0, all = 0;
    for (int i = threadIdx.x; i < r.tokens; i += 256) {
      const bool counts = target_of(r, i) != r.ignore_index;
      all += counts;
      before += counts && i < t;
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
      before += __shfl_xor(before, d, 64);
      all += __shfl_xor(all, d, 64);
    }
    __syncthreads();  // the last token's parts have been read
    if ((threadIdx.x & 63) == 0) {
      parts[0][threadIdx.x >> 6] = before;
      parts[1][threadIdx.x >> 6] = all;
    }
    __syncthreads();
    before = parts[0][0] + parts[0][1] + parts[0][2] + parts[0][3];
    all = parts[1][0] + parts[1][1] + parts[1][2] + parts[1][3];
    if (t >= r.tokens) {
      const int row = all + t - r.tokens;
      if (row < (all + kLossDepth - 1) / kLossDepth * kLossDepth) gather_row(r, row, -1);
      if (t == r.tokens && threadIdx.x == 0) *r.count = all;
      continue;
    }
    const int64_t y = target_of(r, t);
    if (y == r.ignore_index) {
      clear_token(r, t);
      continue;
    }
    if (threadIdx.x == 0) {
      r.index[before] = t;
      r.target[before] = y >= 0 && y < r.vocab ? static_cast<int>(y) : -1;
    }
    gather_row(r, before, t);
  }
}

// A copy of rows whose length or alignment the products cannot read, zeros
// behind each; four pieces a thread, so that its loads overlap: memory bounds it
// (50021 x 2049 FP16 67 us, 6.2 TB/s).
constexpr int kPackPieces = 4;

__global__ __launch_bounds__(256) void pack_kernel(const uint16_t* from, int64_t stride,
                                                   int64_t rows, int cols, uint16_t* to,
                                                   int width) {
  const int pieces = width / 8;
  const int64_t total = rows * pieces, span = 256 * kPackPieces;
  for (int64_t first = blockIdx.x * span; first < total; first += gridDim.x * span) {
    Vector<Bf16> v[kPackPieces];
#pragma unroll
    for (int i = 0; i < kPackPieces; ++i) {
      const int64_t k = first + i * 256 + threadIdx.x;
      if (k >= total) continue;
      const int64_t row =
          k <= 0xffffffffll ? static_cast<uint32_t>(k) / static_cast<uint32_t>(pieces) : k / pieces;
      v[i] = load_vector<Bf16>(from + row * stride, static_cast<int>(k - row * pieces) * 8, cols);
    }
#pragma unroll
    for (int i = 0; i < kPackPieces; ++i) {
      const int64_t k = first + i * 256 + threadIdx.x;
      if (k < total) __builtin_memcpy(to + k * 8, &v[i], 16);
    }
  }
}

// The types of g, and their scale.
struct ScaledBf16 : Bf16 {
  static constexpr float encode_scale = 1.0f;
};
struct ScaledFp16 : Fp16 {
  static constexpr float encode_scale = kLossScale;
};

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
// to each, whose reads are whole lines where ROWS is 16. Latency bounds it: 77 MB of
// chunks of 8192 tokens and 150000 columns take 21 us, those of one token 4.
template <int ROWS>
__global__ __launch_bounds__(1024) void lse_kernel(LossRows r, int sum) {
  constexpr int SHARES = 1024 / ROWS;
  __shared__ float2 parts[SHARES][ROWS];
  __shared__ float own[ROWS];
  const int n = *r.count;
  const int share = threadIdx.x / ROWS, lane = threadIdx.x % ROWS;
  for (int first = blockIdx.x * ROWS; first < n; first += gridDim.x * ROWS) {
    const int row = min(first + lane, n - 1);
    float most = -__builtin_inff(), total = 0.0f;
    auto join = [](float& most, float& total, float2 x) {
      const float top = __builtin_fmaxf(most, x.x);
      // nothing so far, or nothing here: exp(-inf - top) is 0, unless top is too
      const float point = top == -__builtin_inff() ? 0.0f : top;
      total = total * __builtin_amdgcn_exp2f(most - point) +
              x.y * __builtin_amdgcn_exp2f(x.x - point);
      most = top;
    };
    const float2* sums = r.sums + row;
    int k = share;
    for (; k + 3 * SHARES < r.chunks; k += 4 * SHARES) {
      float2 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = sums[static_cast<int64_t>(k + i * SHARES) * r.tokens];
#pragma unroll
      for (int i = 0; i < 4; ++i) join(most, total, x[i]);
    }
    for (; k < r.chunks; k += SHARES) join(most, total, sums[static_cast<int64_t>(k) * r.tokens]);
    parts[share][lane] = make_float2(most, total);
    __syncthreads();
    for (int step = SHARES / 2; step > 0; step >>= 1) {
      if (share < step) {
        join(most, total, parts[share + step][lane]);
        parts[share][lane] = make_float2(most, total);
      }
      __syncthreads();
    }
    if (share == 0 && first + lane < n) {
      // a target outside the vocabulary makes all of its token's results NaN
      const bool outside = r.target[row] < 0;
      const float nan = __builtin_nanf("");
      // in binary64, since these are large beside a small loss
      const double log_sum = log(static_cast<double>(total)) - kLossExponent * kLn2;
      const double lse = static_cast<double>(most) * kLn2 + log_sum;
      const float loss =
          outside ? nan : static_cast<float>(lse - static_cast<double>(r.target_logit[row]));
      r.lse[row] = outside ? nan : static_cast<float>(lse / kLn2);
      r.compact_losses[row] = own[lane] = loss;
      if (r.losses != nullptr) r.losses[r.index[row]] = loss;
    }
    __syncthreads();
  }
  // The one workgroup of a call of few tokens adds their losses up itself.
  if (sum && threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < n; ++i) s += static_cast<double>(own[i]);
    *r.loss = static_cast<float>(r.mean && n > 1 ? s / static_cast<double>(n) : s);
  }
}

template <int THREADS>
__device__ __forceinline__ void sum_losses(const LossRows& r, int n) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += THREADS) s += static_cast<double>(r.compact_losses[i]);
  s = block_sum<THREADS>(s);
  if (threadIdx.x == 0)
    *r.loss = static_cast<float>(r.mean && n > 1 ? s / static_cast<double>(n) : s);
}

// The loss of all tokens without gradients. (Not by the last workgroup of
// lse_kernel: the fence that it would take writes back what L2 holds.)
__global__ __launch_bounds__(1024) void sum_kernel(LossRows r) { sum_losses<1024>(r, *r.count); }

// e of the held piece becomes g, in place: 16 rows of 2048 columns a workgroup,
// whose factors are formed once, in LDS. Eight rows of a thread are asked for before
// the first is needed. The first workgroup adds the losses up too, in binary64 and
// in a fixed order. Memory bounds it, two bytes an element in and two out: 8192 x
// 150000 0.94 ms, 5.2 TB/s (stores past the caches or more rows a thread: the same).
// Without it dx and dw would form the exponential anew for each read of g, or
// the logits be formed twice.
constexpr int kSoftmaxRows = 16, kSoftmaxCols = 2048;

template <typename T>
__global__ __launch_bounds__(256) void softmax_kernel(LossRows r, LossPiece piece) {
  constexpr float scale = T::encode_scale;
  constexpr int BATCH = 8;
  __shared__ float factors[kSoftmaxCols / 64][kSoftmaxRows];
  __shared__ int targets[kSoftmaxRows];
  __shared__ uint16_t at_target[kSoftmaxRows];
  const int n = *r.count;
  const int padded = (n + kLossDepth - 1) / kLossDepth * kLossDepth;
  const int width = (piece.cols + kLossDepth - 1) / kLossDepth * kLossDepth;
  const int across = (width + kSoftmaxCols - 1) / kSoftmaxCols;
  const int64_t total = static_cast<int64_t>(padded / kSoftmaxRows) * across;
  if (blockIdx.x == 0) sum_losses<256>(r, n);
  for (int64_t k = blockIdx.x; k < total; k += gridDim.x) {
    const int first = static_cast<int>(k / across) * kSoftmaxRows;
    const int col0 = static_cast<int>(k % across) * kSoftmaxCols;
    const int at = col0 + threadIdx.x * 8;
    __syncthreads();  // the last round's factors have been read
    for (int i = threadIdx.x; i < (kSoftmaxCols >> r.chunk_shift) * kSoftmaxRows; i += 256) {
      const int row = first + i % kSoftmaxRows, chunk = (col0 >> r.chunk_shift) + i / kSoftmaxRows;
      if (row < n && chunk < r.chunks)
        factors[i / kSoftmaxRows][i % kSoftmaxRows] =
            __builtin_amdgcn_exp2f(r.sums[static_cast<int64_t>(chunk) * r.tokens + row].x -
                                   r.lse[row]) *
            (scale / kLossScale);
    }
    if (threadIdx.x < kSoftmaxRows) {
      const int row = min(first + static_cast<int>(threadIdx.x), n - 1);
      targets[threadIdx.x] = r.target[row] - piece.first;
      // not 1 - p, whose difference loses what a well predicted token has
      at_target[threadIdx.x] = T::encode(scale * expm1f(-r.compact_losses[row]));
    }
    __syncthreads();
    if (at >= width) continue;
    uint16_t* g = piece.g + static_cast<int64_t>(first) * piece.ld + at;
    const float* f = factors[(at - col0) >> r.chunk_shift];
#pragma unroll
    for (int i = 0; i < kSoftmaxRows; i += BATCH) {
      Vector<Fp16> e[BATCH];
#pragma unroll
      for (int u = 0; u < BATCH; ++u)  // padded is a multiple of kSoftmaxRows
        __builtin_memcpy(&e[u], g + static_cast<int64_t>(i + u) * piece.ld, 16);
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = Fp16::decode(e[u].e[j]) * f[i + u];
        Vector<Bf16> o = __builtin_bit_cast(Vector<Bf16>, encode_vector<T>(v));
        const int own = targets[i + u] - at;
        if (own >= 0 && own < 8) {
#pragma unroll
          for (int j = 0; j < 8; ++j) o.e[j] = own == j ? at_target[i + u] : o.e[j];
        }
        if (first + i + u >= n) o = {};  // rows behind the last one are read as zeros
        __builtin_memcpy(g + static_cast<int64_t>(i + u) * piece.ld, &o, 16);
      }
    }
  }
}

// A product's results from the parts of its sum, in order, times c: 1024 columns
// of a row a workgroup. INPUT: row i is that of the token it was gathered from.
// Memory bounds it: 8192 x 5120 from two parts 75 us, 5.6 TB/s.
template <typename T, bool INPUT>
__global__ __launch_bounds__(256) void parts_kernel(LossRows r, const float* partial, int parts,
                                                    int rows, uint16_t* to, int64_t to_stride) {
  const int n = *r.count, across = (r.width + 1023) / 1024, kept = INPUT ? n : rows;
  const float c = (r.mean && n > 1 ? r.scale / static_cast<float>(n) : r.scale) / T::encode_scale;
  const int64_t stride = static_cast<int64_t>(rows) * r.width;
  for (int64_t k = blockIdx.x; k < static_cast<int64_t>(kept) * across; k += gridDim.x) {
    const int row = static_cast<int>(k / across);
    const int at = static_cast<int>(k - static_cast<int64_t>(row) * across) * 1024 + threadIdx.x * 4;
    if (at >= r.hidden) continue;
    const float* from = partial + static_cast<int64_t>(row) * r.width + at;
    float4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {  // width is a multiple of 4
      const float4 v = *reinterpret_cast<const float4*>(from + i * stride);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    uint16_t* out = to + (INPUT ? r.index[row] : row) * to_stride + at;
    const uint16_t o[4] = {T::encode(s.x * c), T::encode(s.y * c), T::encode(s.z * c),
                           T::encode(s.w * c)};
    if (at + 4 <= r.hidden) {
      __builtin_memcpy(out, o, 8);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (at + i < r.hidden) out[i] = o[i];
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
  if (r.tokens <= kCountedTokens)
    return launch(index_gather_kernel, r.tokens + kLossDepth, 256, stream, max_grid, r);
  const hipError_t e = launch(index_kernel, 1, 1024, stream, max_grid, r);
  if (e != hipSuccess) return e;
  const int64_t rows = (static_cast<int64_t>(r.tokens) + kLossDepth - 1) / kLossDepth * kLossDepth;
  return launch(gather_kernel, rows, 256, stream, max_grid, r);
}

hipError_t launch_pack(const uint16_t* from, int64_t stride, int64_t rows, int cols, uint16_t* to,
                       int width, hipStream_t stream, int64_t max_grid) {
  const int64_t span = 256 * kPackPieces;
  return launch(pack_kernel, (rows * (width / 8) + span - 1) / span, 256, stream, max_grid, from,
                stride, rows, cols, to, width);
}

hipError_t launch_loss_lse(const LossRows& r, bool sum, hipStream_t stream, int64_t max_grid) {
  // one workgroup where it is enough, a workgroup to each of few rows, then 16 rows to one
  const int now = sum;
  if (r.tokens <= 1) return launch(lse_kernel<1>, 1, 1024, stream, max_grid, r, now);
  if (r.tokens <= 16) return launch(lse_kernel<16>, 1, 1024, stream, max_grid, r, now);
  const hipError_t e =
      r.tokens <= 256 ? launch(lse_kernel<1>, r.tokens, 1024, stream, max_grid, r, 0)
                      : launch(lse_kernel<16>, (r.tokens + 15) / 16, 1024, stream, max_grid, r, 0);
  if (e != hipSuccess || !sum) return e;
  return launch(sum_kernel, 1, 1024, stream, max_grid, r);
}

hipError_t launch_loss_softmax(const LossRows& r, const LossPiece& piece, hipStream_t stream,
                               int64_t max_grid) {
  const int64_t rows = (static_cast<int64_t>(r.tokens) + kLossDepth - 1) / kLossDepth * kLossDepth;
  const int64_t grid = std::max<int64_t>(1, rows / kSoftmaxRows) *
                       ((static_cast<int64_t>(piece.cols) + kSoftmaxCols - 1) / kSoftmaxCols);
  return launch(r.bf16 ? softmax_kernel<ScaledBf16> : softmax_kernel<ScaledFp16>, grid, 256, stream,
                max_grid, r, piece);
}

hipError_t launch_loss_input(const LossRows& r, const float* partial, int parts,
                             hipStream_t stream, int64_t max_grid) {
  return launch(r.bf16 ? parts_kernel<ScaledBf16, true> : parts_kernel<ScaledFp16, true>,
                r.tokens * ((static_cast<int64_t>(r.width) + 1023) / 1024), 256, stream, max_grid,
                r, partial, parts, r.tokens, r.dx, r.dx_stride);
}

hipError_t launch_loss_weight(const LossProductArgs& a, hipStream_t stream, int64_t max_grid) {
  const LossRows& r = a.r;
  return launch(r.bf16 ? parts_kernel<ScaledBf16, false> : parts_kernel<ScaledFp16, false>,
                a.piece.cols * ((static_cast<int64_t>(r.width) + 1023) / 1024), 256, stream,
                max_grid, r, a.partial, a.shape.parts, a.piece.cols,
                a.dw + a.piece.first * a.dw_stride, a.dw_stride);
}

}  // namespace la
