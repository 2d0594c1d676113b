// la_loss_product.hip -- the matrix products of the linear cross entropy for
// gfx950: logits z = x w^T with the softmax' sums, dx = g w and dw = g^T x.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "la_device.h"
#include "la_loss.h"
#include "la_muon.h"
#include "la_tile.h"

#pragma clang fp contract(off)

namespace la {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896341f;

template <typename T>
__device__ __forceinline__ f32x16 mfma(s16x8 p, s16x8 q, f32x16 c) {
  if constexpr (std::is_same<T, Bf16>::value)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, p),
                                                   __builtin_bit_cast(bf16x8, q), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, p),
                                                  __builtin_bit_cast(half8, q), c, 0, 0, 0);
}

// Eight numbers rounded to 16 bits, to nearest even.
template <typename T>
__device__ __forceinline__ s16x8 rounded(const float (&v)[8]) {
  if constexpr (std::is_same<T, Bf16>::value) {
    bf16x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = static_cast<__bf16>(v[i]);
    return __builtin_bit_cast(s16x8, o);
  } else {
    half8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = static_cast<_Float16>(v[i]);
    return __builtin_bit_cast(s16x8, o);
  }
}

// ---- the kernel ----------------------------------------------------------------------
// A workgroup of WM x WN waves forms a tile of (32 MT WM) x (32 NT WN)
// elements of C = P Q, each wave MT x NT blocks of 32 x 32, as in the products
// of the orthogonalised update (la_product.hip): stages of 64 of the summed
// side, copied from memory straight into LDS, fragments one step of 16 ahead.
//
// What is new here is that an operand may lie either way in memory. One that is
// contiguous along the summed side is kept as rows of 128 bytes, its 16-byte
// pieces at piece ^ (row / 2 % 8). One that is contiguous along the result's
// side ("turned": w in dx = g w; both in dw = g^T x) is kept as it lies, 64
// rows of the tile's width, and read by the transposing LDS read, which hands
// each lane four elements of one column: lanes 4 i .. 4 i + 3 of 16 address row i.
// A read meets four rows 32 bytes a group of 16 lanes, rows a multiple of 256
// bytes apart: their 32-byte pieces lie at piece ^ (2 (row % 4) + row / 8 % 2),
// so that the rows of one read, and those of the other half of the wave, 8
// rows on, take different banks. No second copy of w, g or x is ever made.

template <int MT, int NT, int WM, int WN, int BUFFERS>
struct LossTile {
  static constexpr int waves = WM * WN;
  static constexpr int threads = 64 * waves;
  static constexpr int rows = 32 * MT * WM, cols = 32 * NT * WN;
  static constexpr int stage = (rows + cols) * kLossDepth;  // elements
  static constexpr int p_copies = rows / (8 * waves), q_copies = cols / (8 * waves);
  static constexpr int in_flight = (BUFFERS - 2) * (p_copies + q_copies);
  // the epilogue's part of LDS: blocks of 32 rows that a wave exchanges at once
  static constexpr int lds = BUFFERS * stage * 2;
  static constexpr int at_once =
      std::min(MT, lds / (waves * 32 * 32 * NT * 4)) >= MT ? MT : lds / (waves * 32 * 32 * NT * 4);
  static_assert(at_once >= 1 && MT % at_once == 0, "the epilogue's part of LDS");
  static_assert(rows % (8 * waves) == 0 && cols % (8 * waves) == 0, "whole rows per copy");
};

// An operand's 16-byte piece of LDS place `at` (in pieces): its row (along the
// contiguous side's other one) and its piece within the row.
template <bool TURNED, int SIDE>
__device__ __forceinline__ void place_of(int at, int& row, int& piece) {
  if constexpr (TURNED) {
    row = at / (SIDE / 8);
    piece = (at % (SIDE / 8)) ^ (((row & 3) << 2) | (((row >> 3) & 1) << 1));
  } else {
    row = at / 8;
    piece = (at % 8) ^ ((row >> 1) & 7);
  }
}

// Fragment of 32 rows of the tile from `first` on, step `step` of a stage.
template <bool TURNED, int SIDE>
__device__ __forceinline__ s16x8 fragment(const uint16_t* from, int first, int step, int lane) {
  if constexpr (TURNED) {
    const int g = lane >> 4, i = lane & 15;
    const int row = 16 * step + 8 * (g >> 1) + (i >> 2);
    const int slot = ((first >> 4) + (g & 1)) ^ (((i >> 2) << 1) | (g >> 1));
    const uint16_t* p = from + row * SIDE + slot * 16 + (i & 3) * 4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)const_cast<uint16_t*>(p));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)const_cast<uint16_t*>(p + 4 * SIDE));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    const int row = first + (lane & 31), piece = 2 * step + (lane >> 5);
    return *reinterpret_cast<const s16x8*>(from + row * kLossDepth +
                                           ((piece ^ ((row >> 1) & 7)) << 3));
  }
}

template <typename T, LossProduct WHAT, int MT, int NT, int WM, int WN, int BUFFERS>
__global__ __launch_bounds__(64 * WM * WN, 1) void loss_product_kernel(LossProductArgs a) {
  using G = LossTile<MT, NT, WM, WN, BUFFERS>;
  constexpr bool INPUT = WHAT == LossProduct::kInput, WEIGHT = WHAT == LossProduct::kWeight;
  constexpr bool PT = WEIGHT, QT = INPUT || WEIGHT;
  constexpr bool LOGITS = !INPUT && !WEIGHT;
  __shared__ __align__(1024) uint16_t lds[BUFFERS * G::stage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave / WN) * 32 * MT, wn = (wave % WN) * 32 * NT;
  const LossRows& r = a.r;
  const int n = *r.count;
  // C is M x N over K; operands have p_rows and q_rows rows of the side that is
  // not contiguous, and p_pieces and q_pieces whole pieces along the other.
  const int M = WEIGHT ? a.piece.cols : n;
  const int N = LOGITS ? a.piece.cols : r.hidden;
  const int padded = (n + kLossDepth - 1) / kLossDepth * kLossDepth;
  const int whole = (a.piece.cols + kLossDepth - 1) / kLossDepth * kLossDepth;
  const uint16_t* P = LOGITS ? r.xc : a.piece.g;
  const uint16_t* Q = WEIGHT ? r.xc : a.w + a.piece.first * a.ldw;
  const int ldp = LOGITS ? r.ldx : a.piece.ld;
  const int ldq = WEIGHT ? r.ldx : static_cast<int>(a.ldw);
  const int tiles_m = (M + G::rows - 1) / G::rows, tiles_n = (N + G::cols - 1) / G::cols;
  const int64_t tiles = static_cast<int64_t>(tiles_m) * tiles_n;
  const int64_t total = tiles * (INPUT ? a.splits : 1);

  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int64_t local = xcd_order(w, total);
    const int split = INPUT ? static_cast<int>(local / tiles) : 0;
    int ti, tj;
    rectangle(static_cast<int>(local - split * tiles), tiles_m, tiles_n, ti, tj);
    const int row0 = ti * G::rows, col0 = tj * G::cols;
    const int k0 = INPUT ? split * a.depth : 0;
    const int depth = LOGITS ? r.ldx : WEIGHT ? padded : min(a.depth, whole - k0);
    const int stages = depth > 0 ? depth / kLossDepth : 0;

    // Copies of an operand that is contiguous along the sum: rows past its
    // last one are that one again, their results are not kept. A turned one:
    // pieces past its row's last whole one likewise; rows past its last one (of
    // w, behind the vocabulary) meet zeros of g, so they have to be numbers only.
    // Offsets are 32 bits from the stage's first row (at most 256 rows of 2 MiB).
    const uint16_t* p_first = PT ? P + static_cast<int64_t>(k0) * ldp
                                 : P + static_cast<int64_t>(row0) * ldp + k0;
    const uint16_t* q_first = QT ? Q + static_cast<int64_t>(k0) * ldq
                                 : Q + static_cast<int64_t>(col0) * ldq;
    int po[G::p_copies], qo[G::q_copies], qc[QT ? G::q_copies : 1];
#pragma unroll
    for (int c = 0; c < G::p_copies; ++c) {
      int row, piece;
      place_of<PT, G::rows>((c * G::waves + wave) * 64 + lane, row, piece);
      po[c] = PT ? row * ldp * 2 + min(row0 / 8 + piece, a.piece.ld / 8 - 1) * 16
                 : min(row, M - 1 - row0) * ldp * 2 + piece * 16;
    }
#pragma unroll
    for (int c = 0; c < G::q_copies; ++c) {
      int row, piece;
      place_of<QT, G::cols>((c * G::waves + wave) * 64 + lane, row, piece);
      if constexpr (QT) {
        qo[c] = row * ldq * 2;
        qc[c] = min(col0 / 8 + piece, r.ldx / 8 - 1) * 16;
      } else {
        qo[c] = min(row, N - 1 - col0) * ldq * 2 + piece * 16;
      }
    }
    const int64_t p_step = PT ? static_cast<int64_t>(kLossDepth) * ldp : kLossDepth;
    const int64_t q_step = QT ? static_cast<int64_t>(kLossDepth) * ldq : kLossDepth;
    // copies [from, to) of stage k
    auto copy = [&](int k, int buffer, int from, int to) {
      uint16_t* base = lds + buffer * G::stage + wave * 512;
      const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t*>(p_first + k * p_step), 0, kRsrcRange, kRsrcWord3);
      const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t*>(q_first + k * q_step), 0, kRsrcRange, kRsrcWord3);
      // the last row of w that there is, from the stage's first
      int last = kRsrcRange;
      if constexpr (INPUT) {
        const int64_t rows = r.vocab - 1 - a.piece.first - k0 - static_cast<int64_t>(k) * kLossDepth;
        if (rows < kLossDepth) last = static_cast<int>(rows) * ldq * 2;
      }
#pragma unroll
      for (int c = from; c < to; ++c) {
        uint16_t* at = base + c * G::waves * 512;
        if (c < G::p_copies) {
          copy_to_lds(rp, at, po[c < G::p_copies ? c : 0], 0);
        } else {
          const int j = c - G::p_copies;
          if constexpr (QT)
            copy_to_lds(rq, at, (INPUT ? min(qo[j], last) : qo[j]) + qc[j], 0);
          else
            copy_to_lds(rq, at, qo[j], 0);
        }
      }
    };
    struct Fragments {
      s16x8 p[MT], q[NT];
    };
    auto read = [&](Fragments& f, int buffer, int step) {
      const uint16_t* from = lds + buffer * G::stage;
#pragma unroll
      for (int i = 0; i < MT; ++i) f.p[i] = fragment<PT, G::rows>(from, wm + 32 * i, step, lane);
      from += G::rows * kLossDepth;
#pragma unroll
      for (int j = 0; j < NT; ++j) f.q[j] = fragment<QT, G::cols>(from, wn + 32 * j, step, lane);
    };
    f32x16 acc[MT][NT] = {};
    auto multiply = [&](const Fragments& f) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma<T>(f.p[i], f.q[j], acc[i][j]);
    };
    constexpr int ALL = G::p_copies + G::q_copies;
    Fragments f[2];
#pragma unroll
    for (int k = 0; k < BUFFERS - 1; ++k)
      if (k < stages) copy(k, k, 0, ALL);
    if (stages >= BUFFERS - 1) wait_and_meet<G::in_flight>();
    else wait_and_meet<0>();
    if (stages > 0) read(f[0], 0, 0);
    int buffer = 0;
    for (int k = 0; k < stages; ++k) {
      const int next = buffer + 1 == BUFFERS ? 0 : buffer + 1;
      const int last = buffer == 0 ? BUFFERS - 1 : buffer - 1;
      const bool more = k + BUFFERS - 1 < stages;
      if (more) copy(k + BUFFERS - 1, last, 0, ALL);
#pragma unroll
      for (int step = 1; step < kLossDepth / 16; ++step) {
        read(f[step & 1], buffer, step);
        multiply(f[(step - 1) & 1]);
      }
      if (more) wait_and_meet<G::in_flight>();
      else wait_and_meet<0>();
      if (k + 1 < stages) read(f[0], next, 0);
      multiply(f[1]);
      buffer = next;
    }
    // Every wave is past its last read of LDS, and no copy is under way.
    if constexpr (INPUT) {
      // The accumulators as they lie (lane l: column l % 32; register e: row 8 (e / 4) + 4
      // (l / 32) + e % 4): 32 lanes store 128 bytes of a row.
      float* to = a.partial + static_cast<int64_t>(split) * r.tokens * r.ldx;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int col = col0 + wn + 32 * j + (lane & 31);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int row = row0 + wm + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
            if (row < M && col < r.ldx) {
              float* at = to + static_cast<int64_t>(row) * r.ldx + col;
              *at = a.add ? *at + acc[i][j][e] : acc[i][j][e];
            }
          }
        }
    } else {
      // The sums change to eight neighbours of a row per lane through the wave's own
      // part of LDS, at_once blocks of 32 rows at a time; every four rows the halves
      // of 64 columns are exchanged, so that both halves of a wave store to banks of
      // their own.
      constexpr int WIDTH = 32 * NT, LANES = WIDTH / 8, TOGETHER = 64 / LANES;
      float* sums = reinterpret_cast<float*>(lds) + wave * (32 * G::at_once * WIDTH);
      const int k8 = (lane % LANES) * 8, col = col0 + wn + k8;
      const float c_out = WEIGHT ? (r.mean && n > 1 ? r.scale / static_cast<float>(n) : r.scale) /
                                       (std::is_same<T, Bf16>::value ? 1.0f : kLossScale)
                                 : 0.0f;
#pragma unroll
      for (int part = 0; part < MT / G::at_once; ++part) {
#pragma unroll
        for (int i = 0; i < G::at_once; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int row = 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
              sums[row * WIDTH + ((32 * j + (lane & 31)) ^ ((lane >> 5) << 5))] =
                  acc[part * G::at_once + i][j][e];
            }
        wave_fence();
#pragma unroll 2
        for (int p = 0; p < 32 * G::at_once / TOGETHER; ++p) {
          const int local_row = p * TOGETHER + lane / LANES;
          const int row = row0 + wm + 32 * G::at_once * part + local_row;
          const float* from = sums + local_row * WIDTH + (k8 ^ (((local_row >> 2) & 1) << 5));
          float v[8];
          *reinterpret_cast<f32x4*>(v) = *reinterpret_cast<const f32x4*>(from);
          *reinterpret_cast<f32x4*>(v + 4) = *reinterpret_cast<const f32x4*>(from + 4);
          if constexpr (WEIGHT) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= c_out;
            const s16x8 o = rounded<T>(v);
            if (row < M && col < N) {
              uint16_t* to = a.dw + (a.piece.first + row) * a.dw_stride + col;
              if (a.dw_vectors && col + 8 <= N) {
                *reinterpret_cast<s16x8*>(to) = o;
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (col + e < N) to[e] = o[e];
              }
            }
          } else {
            // columns behind the piece count as exp(-inf)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (col + e >= N) v[e] = -__builtin_inff();
            const bool kept = row < M;
            const int own = kept ? r.target[row] - a.piece.first - col : -1;
            if constexpr (WHAT == LossProduct::kAgain) {
              if (kept && col0 + wn < whole) {
                const float lse = r.lse[row];
                constexpr float scale = std::is_same<T, Bf16>::value ? 1.0f : kLossScale;
                float at_target = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (own == e) at_target = scale * expm1f(v[e] - lse);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  v[e] = scale * __builtin_amdgcn_exp2f((v[e] - lse) * kLog2e);
                  if (own == e) v[e] = at_target;
                }
                if (col < a.piece.ld)
                  *reinterpret_cast<s16x8*>(a.piece.g + static_cast<int64_t>(row) * a.piece.ld +
                                            col) = rounded<T>(v);
              }
            } else {
              if (own >= 0 && own < 8) {
                float z = v[0];
#pragma unroll
                for (int e = 1; e < 8; ++e) z = own == e ? v[e] : z;
                r.target_logit[row] = z;
              }
              float most = v[0];
#pragma unroll
              for (int e = 1; e < 8; ++e) most = __builtin_fmaxf(most, v[e]);
#pragma unroll
              for (int d = LANES / 2; d > 0; d >>= 1)
                most = __builtin_fmaxf(most, __shfl_xor(most, d, 64));
              // nothing in these columns: their exponentials are 0 from any point
              const float from_here = most == -__builtin_inff() ? 0.0f : most;
              float sum = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                v[e] = __builtin_amdgcn_exp2f((v[e] - from_here) * kLog2e);
                sum += v[e];
              }
#pragma unroll
              for (int d = LANES / 2; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
              const int chunk = (a.piece.first + col0 + wn) >> r.chunk_shift;
              if (kept && lane % LANES == 0 && chunk < r.chunks)
                r.sums[static_cast<int64_t>(row) * r.chunks + chunk] = make_float2(most, sum);
              if constexpr (WHAT == LossProduct::kKeep) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= kLossScale;
                if (kept && col < a.piece.ld)
                  *reinterpret_cast<s16x8*>(a.piece.g + static_cast<int64_t>(row) * a.piece.ld +
                                            col) = rounded<Fp16>(v);
              }
            }
          }
        }
        wave_fence();
      }
    }
    wait_and_meet<0>();  // LDS is free for the next tile, and no store is counted with its copies
  }
}

template <typename T, LossProduct WHAT, int MT, int NT, int WM, int WN, int BUFFERS>
hipError_t launch_tile(const LossProductArgs& a, hipStream_t stream, int64_t max_grid) {
  using G = LossTile<MT, NT, WM, WN, BUFFERS>;
  constexpr bool INPUT = WHAT == LossProduct::kInput, WEIGHT = WHAT == LossProduct::kWeight;
  // as many as there would be if every token counted
  const int64_t m = WEIGHT ? a.piece.cols : a.r.tokens;
  const int64_t n = INPUT || WEIGHT ? a.r.hidden : a.piece.cols;
  const int64_t total = ((m + G::rows - 1) / G::rows) * ((n + G::cols - 1) / G::cols) *
                        (INPUT ? a.splits : 1);
  const int64_t grid = std::max<int64_t>(1, std::min({total, kMaxWorkgroups, max_grid}));
  LossProductArgs copy = a;
  void* params[] = {&copy};
  return hipLaunchKernel(
      reinterpret_cast<const void*>(&loss_product_kernel<T, WHAT, MT, NT, WM, WN, BUFFERS>),
      dim3(static_cast<unsigned>(grid)), dim3(G::threads), params, 0, stream);
}

template <typename T, LossProduct WHAT>
hipError_t launch_one(const LossProductArgs& a, hipStream_t stream, int64_t max_grid) {
  return launch_tile<T, WHAT, 2, 2, 2, 2, 4>(a, stream, max_grid);
}

template <typename T>
hipError_t launch_type(const LossProductArgs& a, LossProduct what, hipStream_t stream,
                       int64_t max_grid) {
  switch (what) {
    case LossProduct::kKeep: return launch_one<T, LossProduct::kKeep>(a, stream, max_grid);
    case LossProduct::kSums: return launch_one<T, LossProduct::kSums>(a, stream, max_grid);
    case LossProduct::kAgain: return launch_one<T, LossProduct::kAgain>(a, stream, max_grid);
    case LossProduct::kInput: return launch_one<T, LossProduct::kInput>(a, stream, max_grid);
    default: return launch_one<T, LossProduct::kWeight>(a, stream, max_grid);
  }
}

}  // namespace

int loss_chunk_shift(int64_t) { return 6; }

int loss_splits(int64_t tokens, int64_t hidden, int64_t columns) {
  const int64_t tiles = std::max<int64_t>(1, (tokens + 127) / 128) * ((hidden + 127) / 128);
  return static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>((512 + tiles - 1) / tiles, columns / 1024)));
}

hipError_t launch_loss_product(const LossProductArgs& a, LossProduct what, hipStream_t stream,
                               int64_t max_grid) {
  return a.r.bf16 ? launch_type<Bf16>(a, what, stream, max_grid)
                  : launch_type<Fp16>(a, what, stream, max_grid);
}

}  // namespace la
