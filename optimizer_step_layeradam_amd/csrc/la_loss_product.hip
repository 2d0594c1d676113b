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
typedef s16x8 s16x8_anywhere __attribute__((aligned(2)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

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

// A lane's value joined with those of the others in its group of 8 or 16, by
// exchanges within a row of lanes (a sum's order is then the same everywhere).
template <int CONTROL>
__device__ __forceinline__ float moved(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CONTROL, 0xF, 0xF, true));
}

// The largest of three, a NaN being none: one instruction, where the built-in
// function first makes every NaN among its operands a quiet one.
__device__ __forceinline__ float larger(float x, float y, float z) {
  float m;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(x), "v"(y), "v"(z));
  return m;
}

template <int LANES, int SIDE, typename F>
__device__ __forceinline__ void over_lanes(float (&x)[SIDE], F join) {
  static_assert(LANES == 8 || LANES == 16, "");
#pragma unroll
  for (int u = 0; u < SIDE; ++u) x[u] = join(x[u], moved<0xB1>(x[u]));   // lane ^ 1
#pragma unroll
  for (int u = 0; u < SIDE; ++u) x[u] = join(x[u], moved<0x4E>(x[u]));   // lane ^ 2
#pragma unroll
  for (int u = 0; u < SIDE; ++u) x[u] = join(x[u], moved<0x141>(x[u]));  // 7 - lane of 8
  if constexpr (LANES == 16) {
#pragma unroll
    for (int u = 0; u < SIDE; ++u) x[u] = join(x[u], moved<0x140>(x[u]));  // 15 - lane of 16
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
//
// What bounds them, at 8192 tokens, hidden 5120, vocabulary 150000, BF16, 12.6 TFLOP
// each: logits 10.2 ms, dx 9.5, dw 9.3 (1.23, 1.33, 1.36 PFLOP/s; a library product
// of 8192^3 does 1.45, and 1.36 and 1.17 in the layouts of dx and dw). Matrix units
// are busy in 73 to 88 % of the cycles, at the 1.5 to 1.7 GHz that power leaves; of a
// tile's 80 us at hidden 2560, 4 are the wait for its first stages and 12 the
// epilogue. With 24 tokens the weight's bytes decide: logits of 4096 x 128000 211
// us (5.0 TB/s), dx 172 (6.1), dw 208 (5.0); with one, 2560 x 32000 26 us (6.2 TB/s).

template <int MT, int NT, int WM, int WN, int BUFFERS>
struct Tile {
  static constexpr int waves = WM * WN;
  static constexpr int threads = 64 * waves;
  static constexpr int rows = 32 * MT * WM, cols = 32 * NT * WN;
  static constexpr int stage = (rows + cols) * kLossDepth;  // elements
  // BUFFERS 5: five halves of a stage, one operand each (rows == cols)
  static constexpr bool halves = BUFFERS == 5;
  static constexpr int elements = halves ? 5 * rows * kLossDepth : BUFFERS * stage;
  static constexpr int p_copies = rows / (8 * waves), q_copies = cols / (8 * waves);
  static constexpr int in_flight = BUFFERS > 2 ? (BUFFERS - 2) * (p_copies + q_copies) : 0;
  // the epilogue's part of LDS: blocks of 32 rows that a wave exchanges at once
  static constexpr int lds = elements * 2;
  static constexpr int at_once =
      std::min(MT, lds / (waves * 32 * 32 * NT * 4)) >= MT ? MT : lds / (waves * 32 * 32 * NT * 4);
  static_assert(!halves || rows == cols, "halves of one size");
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

typedef const __attribute__((address_space(3))) s16x4* lds_s16x4;

// Four elements of a lane's column from the rows that its 16 lanes address.
// Without `restrict` the compiler knows nothing about what the read may alias,
// takes every copy into LDS that is under way for it and waits for all of them
// before each read; the meetings of the stages order the two.
__device__ __forceinline__ s16x4 read_turned(lds_s16x4 __restrict__ p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      const_cast<__attribute__((address_space(3))) s16x4*>(p));
}

// Fragment of 32 rows of the tile from `first` on, step `step` of a stage.
template <bool TURNED, int SIDE>
__device__ __forceinline__ s16x8 fragment(const uint16_t* from, int first, int step, int lane) {
  if constexpr (TURNED) {
    const int g = lane >> 4, i = lane & 15;
    const int row = 16 * step + 8 * (g >> 1) + (i >> 2);
    const int slot = ((first >> 4) + (g & 1)) ^ (((i >> 2) << 1) | (g >> 1));
    const uint16_t* p = from + row * SIDE + slot * 16 + (i & 3) * 4;
    const s16x4 a = read_turned((lds_s16x4)p);
    const s16x4 b = read_turned((lds_s16x4)(p + 4 * SIDE));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    const int row = first + (lane & 31), piece = 2 * step + (lane >> 5);
    return *reinterpret_cast<const s16x8*>(from + row * kLossDepth +
                                           ((piece ^ ((row >> 1) & 7)) << 3));
  }
}

template <typename T, LossProduct WHAT, int MT, int NT, int WM, int WN, int BUFFERS>
__global__ __launch_bounds__(64 * WM * WN, BUFFERS == 1 ? 4 : BUFFERS == 2 ? 2 : 1)
    void loss_product_kernel(LossProductArgs a) {
  using G = Tile<MT, NT, WM, WN, BUFFERS>;
  constexpr bool INPUT = WHAT == LossProduct::kInput, WEIGHT = WHAT == LossProduct::kWeight;
  constexpr bool PT = WEIGHT, QT = INPUT || WEIGHT;
  constexpr bool LOGITS = !INPUT && !WEIGHT;
  __shared__ __align__(1024) uint16_t lds[G::elements];
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
  const int ldp = LOGITS ? r.width : a.piece.ld;
  const int ldq = WEIGHT ? r.width : static_cast<int>(a.ldw);
  const int tiles_m = (M + G::rows - 1) / G::rows, tiles_n = (N + G::cols - 1) / G::cols;
  const int64_t tiles = static_cast<int64_t>(tiles_m) * tiles_n;
  const int64_t total = tiles * (LOGITS ? 1 : a.shape.parts);

  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int64_t local = xcd_order(w, total);
    const int part_of = LOGITS ? 0 : static_cast<int>(local / tiles);
    int ti, tj;
    rectangle(static_cast<int>(local - part_of * tiles), tiles_m, tiles_n, ti, tj);
    const int row0 = ti * G::rows, col0 = tj * G::cols;
    const int k0 = LOGITS ? 0 : part_of * a.depth;
    const int depth = LOGITS ? r.width : min(a.depth, (WEIGHT ? padded : whole) - k0);
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
        qc[c] = min(col0 / 8 + piece, r.width / 8 - 1) * 16;
      } else {
        qo[c] = min(row, N - 1 - col0) * ldq * 2 + piece * 16;
      }
    }
    // Where the stages' first rows lie: copies go stage by stage, and past the end
    // the last stage is copied again, into places that nobody reads.
    struct {
      const uint16_t* at;
      int left;  // stages behind this one
    } ap = {p_first, stages - 1}, aq = {q_first, stages - 1};
    const int64_t p_step = PT ? static_cast<int64_t>(kLossDepth) * ldp : kLossDepth;
    const int64_t q_step = QT ? static_cast<int64_t>(kLossDepth) * ldq : kLossDepth;
    auto advance_p = [&] {
      ap.at += ap.left > 0 ? p_step : 0;
      --ap.left;
    };
    auto advance_q = [&] {
      aq.at += aq.left > 0 ? q_step : 0;
      aq.left -= aq.left > 0 ? 1 : 0;
    };
    // copies [from, to) of an operand's part of the stage ahead
    auto copy_p = [&](uint16_t* to, int from, int end) {
      const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t*>(ap.at), 0, kRsrcRange, kRsrcWord3);
#pragma unroll
      for (int c = from; c < end; ++c)
        copy_to_lds(rp, to + (c * G::waves + wave) * 512, po[c], 0);
    };
    auto copy_q = [&](uint16_t* to, int from, int end) {
      const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t*>(aq.at), 0, kRsrcRange, kRsrcWord3);
      // the last row of w that there is, from the stage's first
      int last = kRsrcRange;
      if constexpr (INPUT) {
        const int rows = r.vocab - 1 - a.piece.first - k0 - (stages - 1 - aq.left) * kLossDepth;
        if (rows < kLossDepth) last = rows * ldq * 2;
      }
#pragma unroll
      for (int c = from; c < end; ++c)
        copy_to_lds<MT == 1 ? kNonTemporal : 0>(rq, to + (c * G::waves + wave) * 512,
                    QT ? (INPUT ? min(qo[c], last) : qo[c]) + qc[QT ? c : 0] : qo[c], 0);
    };
    struct Fragments {
      s16x8 p[MT], q[NT];
    };
    auto read = [&](Fragments& f, const uint16_t* p, const uint16_t* q, int step) {
#pragma unroll
      for (int i = 0; i < MT; ++i) f.p[i] = fragment<PT, G::rows>(p, wm + 32 * i, step, lane);
#pragma unroll
      for (int j = 0; j < NT; ++j) f.q[j] = fragment<QT, G::cols>(q, wn + 32 * j, step, lane);
    };
    // What the wave's rows have, a lane to a row.
    struct {
      int target[MT > 2 ? 2 : 1];
      float lse[MT > 2 ? 2 : 1];
    } mine = {};
    // (kAgain in one buffer, where registers are short, reads them when it needs them.)
    constexpr bool MINE = LOGITS && !(WHAT == LossProduct::kAgain && BUFFERS == 1);
    if constexpr (MINE) {
#pragma unroll
      for (int i = 0; i < (MT > 2 ? 2 : 1); ++i) {
        const int row = min(row0 + wm + 64 * i + lane, M - 1);
        mine.target[i] = r.target[row];
        if constexpr (WHAT == LossProduct::kAgain) mine.lse[i] = r.lse[row];
      }
    }
    f32x16 acc[MT][NT] = {};
    auto multiply = [&](const Fragments& f) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mfma<T>(f.p[i], f.q[j], acc[i][j]);
    };
    // Deals a step's reads of LDS, and behind them `copies` copies, out among
    // its products (as in la_product.hip: issued in a row they hold the products up).
    auto interleave = [&](auto copies) {
      constexpr int reads = (PT ? 2 : 1) * MT + (QT ? 2 : 1) * NT, products = MT * NT;
      constexpr int n = decltype(copies)::value;
      constexpr int pairs = reads + n > products ? 2 : 1;  // reads beside one product
      constexpr int each = n == 0 && products > reads ? products / reads : 1;
#pragma unroll
      for (int i = 0; i < reads / pairs; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, pairs, 0);  // LDS read
        __builtin_amdgcn_sched_group_barrier(0x008, each, 0);   // MFMA
      }
#pragma unroll
      for (int i = 0; i < n; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);  // copy
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
      if constexpr (products > reads / pairs * each + n)
        __builtin_amdgcn_sched_group_barrier(0x008, products - reads / pairs * each - n, 0);
      __builtin_amdgcn_sched_barrier(0);
    };
    using None = std::integral_constant<int, 0>;
    Fragments f[2];
    if constexpr (G::halves) {
      // LDS holds five operands' parts, P_0 Q_0 P_1 Q_1 P_2, then Q_2 in the place of
      // P_0 and so on: part i lies at i % 5. Behind the meeting after stage k's
      // last reads its places take Q of stage k + 2, at once, and P of stage k + 3,
      // which has a whole stage more to arrive: the meeting waits for older copies
      // only. The loop has no branch that would part the products.
      if (stages > 0) {
        constexpr int half = G::rows * kLossDepth;
        copy_p(lds, 0, G::p_copies);
        copy_q(lds + half, 0, G::q_copies);
        advance_p();
        advance_q();
        copy_p(lds + 2 * half, 0, G::p_copies);
        copy_q(lds + 3 * half, 0, G::q_copies);
        advance_p();
        wait_and_meet<G::p_copies + G::q_copies>();
        read(f[0], lds, lds + half, 0);
        using Qcopies = std::integral_constant<int, G::q_copies>;
        using Phalf = std::integral_constant<int, G::p_copies / 2>;
        int at = 0;  // place of P_k
        auto place = [&](int i) { return lds + (at + i < 5 ? at + i : at + i - 5) * half; };
        uint16_t *p = place(0), *q = place(1), *later = place(4);
        for (int k = 0; k < stages; ++k) {
          // scalar work lies where products cover it, not at the stage's ends
          read(f[1], p, q, 1);
          copy_p(later, 0, G::p_copies / 2);
          advance_q();
          multiply(f[0]);
          interleave(Phalf());
          read(f[0], p, q, 2);
          copy_p(later, G::p_copies / 2, G::p_copies);
          advance_p();
          multiply(f[1]);
          interleave(Phalf());
          read(f[1], p, q, 3);
          uint16_t* const done = p;
          at = at + 2 < 5 ? at + 2 : at - 3;
          p = place(0);
          q = place(1);
          later = place(4);
          multiply(f[0]);
          interleave(None());
          wait_and_meet<G::p_copies>();
          read(f[0], p, q, 0);
          copy_q(done, 0, G::q_copies);
          multiply(f[1]);
          interleave(Qcopies());
        }
      }
      wait_and_meet<0>();
    } else {
      auto copy = [&](int buffer) {
        uint16_t* to = lds + buffer * G::stage;
        copy_p(to, 0, G::p_copies);
        copy_q(to + G::rows * kLossDepth, 0, G::q_copies);
        advance_p();
        advance_q();
      };
      auto part = [&](Fragments& to, int buffer, int step) {
        const uint16_t* from = lds + buffer * G::stage;
        read(to, from, from + G::rows * kLossDepth, step);
      };
      if constexpr (BUFFERS == 1) {  // a stage or two: several workgroups a compute unit instead
        for (int k = 0; k < stages; ++k) {
          copy(0);
          wait_and_meet<0>();
          part(f[0], 0, 0);
#pragma unroll
          for (int step = 1; step < kLossDepth / 16; ++step) {
            part(f[step & 1], 0, step);
            multiply(f[(step - 1) & 1]);
          }
          multiply(f[1]);
          wait_and_meet<0>();
        }
      } else {
#pragma unroll
        for (int k = 0; k < BUFFERS - 1; ++k)
          if (k < stages) copy(k);
        if (stages >= BUFFERS - 1) wait_and_meet<G::in_flight>();
        else wait_and_meet<0>();
        if (stages > 0) part(f[0], 0, 0);
        int buffer = 0;
        for (int k = 0; k < stages; ++k) {
          const int next = buffer + 1 == BUFFERS ? 0 : buffer + 1;
          const int last = buffer == 0 ? BUFFERS - 1 : buffer - 1;
          const bool more = k + BUFFERS - 1 < stages;
          if (more) copy(last);
#pragma unroll
          for (int step = 1; step < kLossDepth / 16; ++step) {
            part(f[step & 1], buffer, step);
            multiply(f[(step - 1) & 1]);
            interleave(None());
          }
          if (more) wait_and_meet<G::in_flight>();
          else wait_and_meet<0>();
          if (k + 1 < stages) part(f[0], next, 0);
          multiply(f[1]);
          buffer = next;
        }
      }
    }
    // Every wave is past its last read of LDS, and no copy is under way.
    // The sums change to eight neighbours of a row per lane through the wave's own
    // part of LDS, at_once blocks of 32 rows at a time; every four rows the halves
    // of 64 columns are exchanged, so that both halves of a wave store to banks of
    // their own.
    constexpr int WIDTH = 32 * NT, LANES = WIDTH / 8, TOGETHER = 64 / LANES;
    // rows of a lane that are worked on side by side: alone, a row is a chain of
    // exchanges that the wave would wait for (fewer where four workgroups share the
    // registers)
    constexpr int SIDE = !LOGITS || BUFFERS > 1 ? 4 : 2;
    constexpr int PASSES = 32 * G::at_once / TOGETHER;
    static_assert(PASSES % SIDE == 0, "whole passes");
    float* sums = reinterpret_cast<float*>(lds) + wave * (32 * G::at_once * WIDTH);
    const int k8 = (lane % LANES) * 8, col = col0 + wn + k8;
    const float c_out = !LOGITS ? (r.mean && n > 1 ? r.scale / static_cast<float>(n) : r.scale) /
                                      (std::is_same<T, Bf16>::value ? 1.0f : kLossScale)
                                : 0.0f;
    const bool edge = col0 + G::cols > N;
    const int chunk = LOGITS ? (a.piece.first + col0 + wn) >> r.chunk_shift : 0;
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
#pragma unroll 1
      for (int p = 0; p < PASSES; p += SIDE) {
        float v[SIDE][8];
        int row[SIDE];
#pragma unroll
        for (int u = 0; u < SIDE; ++u) {
          const int local_row = (p + u) * TOGETHER + lane / LANES;
          row[u] = row0 + wm + 32 * G::at_once * part + local_row;
          const float* from = sums + local_row * WIDTH + (k8 ^ (((local_row >> 2) & 1) << 5));
          *reinterpret_cast<f32x4*>(v[u]) = *reinterpret_cast<const f32x4*>(from);
          *reinterpret_cast<f32x4*>(v[u] + 4) = *reinterpret_cast<const f32x4*>(from + 4);
        }
        if constexpr (!LOGITS) {
          const bool partial = INPUT ? !a.direct : a.shape.parts > 1;
          const int64_t rows = INPUT ? r.tokens : M;
#pragma unroll
          for (int u = 0; u < SIDE; ++u) {
            if (row[u] >= M || col >= r.width) continue;
            if (partial) {
              float* to = a.partial + (part_of * rows + row[u]) * r.width + col;
              f32x4 lo = *reinterpret_cast<const f32x4*>(v[u]);
              f32x4 hi = *reinterpret_cast<const f32x4*>(v[u] + 4);
              if (INPUT && a.add) {
                lo += *reinterpret_cast<const f32x4*>(to);
                hi += *reinterpret_cast<const f32x4*>(to + 4);
              }
              *reinterpret_cast<f32x4*>(to) = lo;
              *reinterpret_cast<f32x4*>(to + 4) = hi;
              continue;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] *= c_out;
            const s16x8 o = rounded<T>(v[u]);
            uint16_t* to = INPUT ? r.dx + r.index[row[u]] * r.dx_stride
                                 : a.dw + (a.piece.first + row[u]) * a.dw_stride;
            if (col + 8 <= N) {  // at any element; nothing here reads it again
              __builtin_nontemporal_store(o, reinterpret_cast<s16x8_anywhere*>(to + col));
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (col + e < N) to[col + e] = o[e];
            }
          }
        } else {
          int own[SIDE];      // the target's place among the lane's columns
          float lse[SIDE];
#pragma unroll
          for (int u = 0; u < SIDE; ++u) {
            const int at = row[u] - row0 - wm;
            if constexpr (MINE) {
              own[u] = __shfl(mine.target[0], at & 63, 64);
              if constexpr (MT == 4) {
                const int other = __shfl(mine.target[1], at & 63, 64);
                own[u] = at < 64 ? own[u] : other;
              }
            } else {
              own[u] = r.target[min(row[u], M - 1)];
            }
            own[u] -= a.piece.first + col;
            if constexpr (WHAT == LossProduct::kAgain) {
              if constexpr (MINE) {
                lse[u] = __shfl(mine.lse[0], at & 63, 64);
                if constexpr (MT == 4) {
                  const float other = __shfl(mine.lse[1], at & 63, 64);
                  lse[u] = at < 64 ? lse[u] : other;
                }
              } else {
                lse[u] = r.lse[min(row[u], M - 1)];
              }
            }
            if (edge) {  // columns behind the piece count as exp(-inf)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (col + e >= N) v[u][e] = -__builtin_inff();
            }
          }
          if constexpr (WHAT == LossProduct::kAgain) {
#pragma unroll
            for (int u = 0; u < SIDE; ++u) {
              constexpr float scale = std::is_same<T, Bf16>::value ? 1.0f : kLossScale;
              float at_target = 0.0f;
              if (own[u] >= 0 && own[u] < 8 && row[u] < M)
                at_target = scale * expm1f(-r.compact_losses[row[u]]);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                v[u][e] = scale * __builtin_amdgcn_exp2f(__builtin_fmaf(v[u][e], kLog2e, -lse[u]));
                v[u][e] = own[u] == e ? at_target : v[u][e];
              }
              if (row[u] < M && col < a.piece.ld)
                *reinterpret_cast<s16x8*>(a.piece.g + static_cast<int64_t>(row[u]) * a.piece.ld +
                                          col) = rounded<T>(v[u]);
            }
          } else {
            float most[SIDE], sum[SIDE];
#pragma unroll
            for (int u = 0; u < SIDE; ++u) {
              if (own[u] >= 0 && own[u] < 8 && row[u] < M) {
                float z = v[u][0];
#pragma unroll
                for (int e = 1; e < 8; ++e) z = own[u] == e ? v[u][e] : z;
                r.target_logit[row[u]] = z;
              }
              most[u] = larger(larger(v[u][0], v[u][1], v[u][2]),
                               larger(v[u][3], v[u][4], v[u][5]),
                               larger(v[u][6], v[u][7], v[u][7]));
            }
            over_lanes<LANES, SIDE>(most, [](float x, float y) { return larger(x, y, y); });
#pragma unroll
            for (int u = 0; u < SIDE; ++u) {
              // From here on in powers of two, 14 above the maximum. Nothing in these
              // columns: their exponentials are 0 from any point.
              const float point = most[u] * kLog2e;
              const bool none = point == -__builtin_inff();
              const float from_here = (none ? 0.0f : point) - kLossExponent;
              most[u] = none ? point : from_here + kLossExponent;  // exactly what was taken off
              sum[u] = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                v[u][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[u][e], kLog2e, -from_here));
                sum[u] += v[u][e];
              }
            }
            over_lanes<LANES, SIDE>(sum, [](float x, float y) { return x + y; });
#pragma unroll
            for (int u = 0; u < SIDE; ++u) {
              if (row[u] < M && lane % LANES == 0 && chunk < r.chunks)
                r.sums[static_cast<int64_t>(chunk) * r.tokens + row[u]] =
                    make_float2(most[u], sum[u]);
              if constexpr (WHAT == LossProduct::kKeep) {
                if (row[u] < M && col < a.piece.ld)
                  *reinterpret_cast<s16x8*>(a.piece.g + static_cast<int64_t>(row[u]) * a.piece.ld +
                                            col) = rounded<Fp16>(v[u]);
              }
            }
          }
        }
      }
      wave_fence();
    }
    // LDS is free for the next tile, and no store is counted with its copies; the last
    // tile's stores need nobody to wait for them
    if (w + gridDim.x < total) wait_and_meet<0>();
  }
}

template <typename T, LossProduct WHAT, int MT, int NT, int WM, int WN, int BUFFERS>
hipError_t launch_tile(const LossProductArgs& a, hipStream_t stream, int64_t max_grid) {
  using G = Tile<MT, NT, WM, WN, BUFFERS>;
  constexpr bool INPUT = WHAT == LossProduct::kInput, WEIGHT = WHAT == LossProduct::kWeight;
  // as many as there would be if every token counted
  const int64_t m = WEIGHT ? a.piece.cols : a.r.tokens;
  const int64_t n = INPUT || WEIGHT ? a.r.hidden : a.piece.cols;
  const int64_t total = ((m + G::rows - 1) / G::rows) * ((n + G::cols - 1) / G::cols) *
                        (INPUT || WEIGHT ? a.shape.parts : 1);
  const int64_t grid = std::max<int64_t>(1, std::min({total, kMaxWorkgroups, max_grid}));
  LossProductArgs copy = a;
  void* params[] = {&copy};
  return hipLaunchKernel(
      reinterpret_cast<const void*>(&loss_product_kernel<T, WHAT, MT, NT, WM, WN, BUFFERS>),
      dim3(static_cast<unsigned>(grid)), dim3(G::threads), params, 0, stream);
}

template <typename T, LossProduct WHAT>
hipError_t launch_one(const LossProductArgs& a, hipStream_t stream, int64_t max_grid) {
  if constexpr (WHAT != LossProduct::kWeight) {  // turned rows of g are 128 columns at least
    if (a.shape.tile == LossTile::kSmallest)
      return launch_tile<T, WHAT, 1, 2, 1, 2, 4>(a, stream, max_grid);
    if (a.shape.tile == LossTile::kSmall)
      return launch_tile<T, WHAT, 1, 2, 2, 2, 3>(a, stream, max_grid);
  }
  return a.shape.tile == LossTile::kLarge ? launch_tile<T, WHAT, 4, 4, 2, 2, 5>(a, stream, max_grid)
                                          : launch_tile<T, WHAT, 2, 2, 2, 2, 1>(a, stream, max_grid);
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

namespace {

int64_t tiles_of(LossTile tile, int64_t m, int64_t n) {
  const int64_t rows = tile == LossTile::kLarge ? 256 : tile == LossTile::kMedium ? 128 : 64;
  const int64_t cols = tile == LossTile::kLarge ? 256 : 128;
  return ((m + rows - 1) / rows) * ((n + cols - 1) / cols);
}

// What `tiles` tiles of `stages` stages take, in us, from these measurements (us,
// 256 x 256 | 128 x 128 | 64 x 128):
//   logits of 4096 tokens, 32768 words, hidden 512    212 |  176 |
//                                       hidden 4096   904 | 1082 |
//             256                       hidden 4096   101 |   95 |
//             512 tokens, 8000 words, hidden 4096         |   65 |  62
//            2048                     hidden  512         |   26 |  40
//            2048 tokens, 1000 words, hidden 4096         |   62 |  39
//             512                     hidden 1024         |   19 |  11
//   the weight's gradient, 4096 columns of 32768 words, from
//             256 tokens                              123 |  100 |
//            4096                                     845 | 1037 |
// The medium tile has one buffer, and four workgroups a compute unit that take
// turns (with two or four buffers and fewer workgroups all of these took as long
// or longer), the small one three and two workgroups: it is the one for few tiles,
// which nothing else hides the copies of.
double time_of(LossTile tile, int64_t tiles, int64_t stages) {
  const double s = static_cast<double>(stages);
  const int64_t each = (tiles + 255) / 256;  // of a compute unit
  if (tile == LossTile::kLarge) return static_cast<double>(each) * (14.0 + 1.55 * s);
  if (tile == LossTile::kMedium) {
    const int64_t rest = each % 4;
    return static_cast<double>(each / 4) * (5.4 + 2.04 * s) +
           (rest > 0 ? 2.5 + s * (1.2 + 0.21 * static_cast<double>(rest)) : 0.0);
  }
  return static_cast<double>(each / 2) * (2.5 + 0.95 * s) +
         static_cast<double>(each % 2) * (2.5 + 0.4 * s);
}

// A product's shape and its modelled time, and whether it would take more parts
// than it may.
struct Choice {
  LossShape shape;
  double time;
  bool held_back;
};

// The tile and parts, at most `most` of them, that take least for an m x n product
// over `depth`. `least`: elements of a part at least; 0: one part.
Choice shape_of(int64_t m, int64_t n, int64_t depth, int64_t least, bool small, int64_t most) {
  Choice best = {{LossTile::kMedium, 1}, 0.0, false}, any = best;
  const int64_t sensible =
      least > 0 ? std::max<int64_t>(1, std::min<int64_t>(64, depth / least)) : 1;
  for (LossTile tile : {LossTile::kSmall, LossTile::kMedium, LossTile::kLarge}) {
    if (tile == LossTile::kSmall && !small) continue;
    for (int64_t k = 1; k <= sensible; ++k) {
      const int64_t stages = (depth + kLossDepth * k - 1) / (kLossDepth * k);
      double t = time_of(tile, tiles_of(tile, m, n) * k, stages);
      // parts' binary32 results are written and read, at 5 TB/s, by a launch more
      if (k > 1) t += 4.0 + static_cast<double>(k * m * n) * 8.0 / 5e6;
      const Choice c = {{tile, static_cast<int32_t>(k)}, t, false};
      if (any.time == 0.0 || t < 0.99 * any.time) any = c;
      if (k <= most && (best.time == 0.0 || t < 0.99 * best.time)) best = c;
    }
  }
  if (any.shape.parts <= most) return any;
  best.held_back = true;
  return best;
}

// The same for one to 64 tokens, whose tile is given: two workgroups a compute unit.
Choice few_shape_of(LossTile tile, int64_t hidden, int64_t columns, int64_t most) {
  const int64_t tiles = (hidden + 127) / 128;
  // of at least 512 columns each
  const int64_t wanted = std::max<int64_t>(1, std::min({columns / 512, 512 / tiles, int64_t(64)}));
  const int64_t parts = std::min(wanted, most);
  const int64_t stages = (columns + kLossDepth * parts - 1) / (kLossDepth * parts);
  return {{tile, static_cast<int32_t>(parts)}, time_of(LossTile::kSmall, tiles * parts, stages),
          parts < wanted};
}

}  // namespace

// Up to this many tokens the weight's traffic decides: tiles of 32 or 64 rows by
// 128 columns, whose copies of the weight pass by the caches (24 tokens x 4096 x
// 128000, 1.05 GB: logits 198 us, and 262 us through them).
constexpr int64_t kFewTokens = 64, kFewestTokens = 32;

// What a piece costs beside its products, us: their launches.
constexpr double kPieceTime = 10.0;

LossShapes loss_shapes(const LossSizes& z, int64_t room) {
  LossShapes s = {};
  const int64_t tokens = std::max<int64_t>(1, z.tokens);
  const int64_t columns = std::min(z.columns, z.vocab);
  const int64_t row_bytes = 4 * ((z.hidden + kLossDepth - 1) / kLossDepth * kLossDepth);
  // parts of an output of `rows` rows that there is room for, `kept` of them being there
  // in any case
  auto most_of = [&](int64_t rows, int64_t kept) {
    return std::max<int64_t>(1, kept + room / (rows * row_bytes));
  };
  const int64_t kept = loss_least_parts(z);
  const int64_t most_input = most_of(tokens, kept);
  Choice logits, input;
  if (tokens <= kFewTokens) {
    const LossTile tile = tokens <= kFewestTokens ? LossTile::kSmallest : LossTile::kSmall;
    const int64_t stages = (z.hidden + kLossDepth - 1) / kLossDepth;
    logits = {{tile, 1}, time_of(LossTile::kSmall, (z.vocab + 127) / 128, stages), false};
    input = few_shape_of(tile, z.hidden, columns, most_input);
  } else {
    logits = shape_of(tokens, z.vocab, z.hidden, 0, true, 1);
    input = shape_of(tokens, z.hidden, columns, 512, true, most_input);
  }
  if (z.input && input.shape.parts > 1) room -= (input.shape.parts - kept) * tokens * row_bytes;
  const Choice weight = shape_of(columns, z.hidden, tokens, 512, false,
                                 most_of(std::max<int64_t>(1, columns), 0));
  s.logits = logits.shape;
  s.input = input.shape;
  s.weight = weight.shape;
  s.chunk_shift = s.logits.tile == LossTile::kLarge ? 7 : kLeastChunkShift;
  const double pieces = static_cast<double>(std::max<int64_t>(1, z.pieces));
  s.time = logits.time * (2.0 - 1.0 / pieces) +
           pieces * (kPieceTime + (z.input ? input.time : 0.0) + (z.weight ? weight.time : 0.0));
  s.held_back = (z.input && input.held_back) || (z.weight && weight.held_back);
  return s;
}

hipError_t launch_loss_product(const LossProductArgs& a, LossProduct what, hipStream_t stream,
                               int64_t max_grid) {
  return a.r.bf16 ? launch_type<Bf16>(a, what, stream, max_grid)
                  : launch_type<Fp16>(a, what, stream, max_grid);
}

}  // namespace la
