// la_product.hip -- the matrix products of the orthogonalised update for
// gfx950: C = P Q^T over stacks of matrices, with the iteration's epilogues.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "la_muon.h"

#pragma clang fp contract(off)

namespace la {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Raw buffer resource over a uniform base: no stride, 2 GiB of range, the
// fourth word of a 32-bit-format buffer.
constexpr int kRsrcRange = 0x7fffffff;
constexpr int kRsrcWord3 = 0x00020000;

// 16 bytes per lane from memory to 1 KiB of LDS at `to` (lane order), without
// a register between; done when the wave's vmcnt says so.
__device__ __forceinline__ void copy_to_lds(__amdgpu_buffer_rsrc_t from, _Float16* to, int offset,
                                            int uniform_offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      from, (__attribute__((address_space(3))) void*)to, 16, offset, uniform_offset, 0, 0);
}

// All but the last PENDING of this wave's copies have landed and its reads of
// LDS are done; so are those of every wave of the workgroup after it.
template <int PENDING>
__device__ __forceinline__ void wait_and_meet() {
  static_assert(PENDING >= 0 && PENDING < 64, "six bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(PENDING) : "memory");
}

// Orders the wave's own LDS accesses, which lanes exchange data through.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

struct ProductArgs {
  ProductGroup g[kGroupsPerLaunch];
  int64_t tile_end[kGroupsPerLaunch];  // cumulative tiles
  int32_t tiles_m[kGroupsPerLaunch], tiles_n[kGroupsPerLaunch];
  int32_t tiles[kGroupsPerLaunch];     // tiles of one matrix
  ProductScales s;
  const int32_t* skip;
  int32_t count;
};
static_assert(sizeof(ProductArgs) <= 4096, "kernel arguments");

// BF16, round to nearest even, NaN -> 0x7FC0 (as in the update's kernel).
__device__ __forceinline__ uint16_t bf16_bits(float x) {
  const uint32_t b = __float_as_uint(x);
  const uint32_t r = (b + 0x7FFFu + ((b >> 16) & 1u)) >> 16;
  return static_cast<uint16_t>(__builtin_isnan(x) ? 0x7FC0u : r);
}

__device__ __forceinline__ uint16_t fp16_bits(float x) {
  const uint16_t h = __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
  return __builtin_isnan(x) ? uint16_t(0x7E00) : h;
}

// Workgroups are dealt to the 8 XCDs in turn: give each XCD consecutive tiles
// of every 256 of a stack, so that the tiles its L2 serves share operand
// rows, and each XCD the same share of every stack (sums of one stack are
// equally long).
__device__ __forceinline__ int64_t xcd_order(int64_t w, int64_t n) {
  const int64_t base = w & ~int64_t(255);
  const int part = static_cast<int>(n - base < 256 ? n - base : 256);
  const int l = static_cast<int>(w - base), x = l & 7;
  const int q = part >> 3, r = part & 7;
  return base + x * q + (x < r ? x : r) + (l >> 3);
}

// Tile t of a matrix, in bands of four tile rows taken column by column: 32
// consecutive tiles are about 4 x 8 of them.
__device__ __forceinline__ void rectangle(int t, int tiles_m, int tiles_n, int& i, int& j) {
  const int band = t / (4 * tiles_n), first = 4 * band;
  const int rows = tiles_m - first < 4 ? tiles_m - first : 4;
  const int l = t - band * 4 * tiles_n;
  i = first + l % rows;
  j = l / rows;
}

// The same for the lower triangle: a band's columns up to its first row are
// whole, the last ones shorter by one tile each.
__device__ __forceinline__ void triangle(int t, int tiles_m, int& i, int& j) {
  int r = static_cast<int>((__builtin_sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
  while (static_cast<int64_t>(r) * (r + 1) / 2 > t) --r;
  while (static_cast<int64_t>(r + 1) * (r + 2) / 2 <= t) ++r;
  const int first = r & ~3;
  const int rows = tiles_m - first < 4 ? tiles_m - first : 4;
  int l = t - static_cast<int>(static_cast<int64_t>(first) * (first + 1) / 2);
  if (l < rows * (first + 1)) {
    i = first + l % rows;
    j = l / rows;
    return;
  }
  l -= rows * (first + 1);
  int c = 1;
  while (l >= rows - c) {
    l -= rows - c;
    ++c;
  }
  i = first + c + l;
  j = first + c;
}

// ---- the kernel ----------------------------------------------------------------------
// A workgroup of WM x WN waves forms a tile of (32 MT WM) x (32 NT WN)
// elements of C, each wave MT x NT blocks of 32 x 32. A stage is kDepth elements of the
// summed side: 128 bytes of every row of both operands, copied from memory
// straight into LDS, where a row's 16-byte pieces are stored at piece ^
// (row / 2 % 8): a wave's read of one piece of 32 rows then meets every bank
// group equally often, whichever of its lanes are served together. Two stages
// are held; the copy of one runs under the products of the other. Per stage a
// wave takes four steps of 16 elements, whose fragments it reads one step
// ahead; before the last step's products it waits for its own copies and
// meets the others, so that the next stage's first fragments arrive under
// these products.
//
// In 256 x 256 tiles a wave reads 8 fragments from LDS for 16 products, in 128 x
// 128 ones 4 for 4; the large tile takes all of a compute unit's registers, so
// nothing runs under its epilogue. Measured on 5120 x 17408, in 256 x 256
// tiles: X X^T (210 tiles on 256 compute units) 415 us, 1.15 PFLOP/s of what
// the tiles compute; B X with its update (1360 tiles) 942 us, 0.97 PFLOP/s, the
// epilogue's 8 bytes an element among it; the last step 840 us, 1.09 PFLOP/s.
// The matrix units are busy 50 to 58 % of the time, at 1.9 GHz.

template <int MT, int NT, int WM, int WN, int BUFFERS>
struct Tile {
  static constexpr int waves = WM * WN;
  static constexpr int threads = 64 * waves;
  static constexpr int rows = 32 * MT * WM, cols = 32 * NT * WN;
  static constexpr int stage = (rows + cols) * kDepth;  // elements
  static constexpr int pieces = kDepth / 8;             // of 16 bytes in a row
  static constexpr int copy_rows = 64 / pieces;        // rows that one copy of a wave brings
  static constexpr int p_copies = rows / (copy_rows * waves);
  static constexpr int q_copies = cols / (copy_rows * waves);
  static constexpr int in_flight = (BUFFERS - 2) * (p_copies + q_copies);
  static_assert(BUFFERS * stage * 2 >= waves * 32 * MT * 256, "the epilogue's part of LDS");
  static_assert(rows % (copy_rows * waves) == 0 && cols % (copy_rows * waves) == 0,
                "whole rows per copy");
  static_assert(kDepth == 64, "slot()");
  // Where piece p of row r is kept: 64 banks hold 256 bytes, two rows.
  static __device__ __forceinline__ int slot(int r, int p) { return p ^ ((r >> 1) & 7); }
};

template <int MT, int NT>
struct Fragments {
  half8 p[MT], q[NT];
};

// x y + z in one rounding: where the terms are converted from binary16 it is one
// instruction for both.
__device__ __forceinline__ float fma(float x, float y, float z) {
  return __builtin_fmaf(x, y, z);
}

// `mask` over the bits of eight binary16 numbers.
__device__ __forceinline__ half8 keep(half8 h, u32x4 mask) {
  return __builtin_bit_cast(half8, __builtin_bit_cast(u32x4, h) & mask);
}

// What no later product reads passes by the caches: lo, X's reading in the
// epilogue, the result (5120 x 17408: an update in 975 us instead of 1000). X
// itself, in both layouts, and A and B do not: X X^T after a turned X stored so
// took 13 % longer.
template <typename T>
__device__ __forceinline__ T load_once(const void* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
}

template <typename T>
__device__ __forceinline__ void store_through(T v, void* p) {
  __builtin_nontemporal_store(v, reinterpret_cast<T*>(p));
}

// What the epilogue reads for eight neighbours of one row: loaded ahead of the
// sums' exchange, so that its latency is paid once for four rows of a lane.
template <Product WHAT>
struct Operands {
  half8 hi;          // all but kGram
  u32x2 lo;          // kUpdate
  f32x4 master[2];   // kMuon
  float diag;        // the row's
};

template <Product WHAT>
__device__ __forceinline__ void load_operands(Operands<WHAT>& x, const ProductGroup& g, int z,
                                              int row, int col) {
  if constexpr (WHAT != Product::kGram) {
    const int r = row < g.M ? row : g.M - 1;
    const int c = col < g.ldc ? col : g.ldc - 8;
    const int64_t at = z * g.c_stride + static_cast<int64_t>(r) * g.ldc + c;
    const half_bits* hi = g.hi + at;
    if constexpr (WHAT == Product::kUpdate || WHAT == Product::kOut)
      x.hi = load_once<half8>(hi);
    else
      x.hi = *reinterpret_cast<const half8*>(hi);
    if constexpr (WHAT == Product::kUpdate)
      x.lo = load_once<u32x2>(g.lo + at);
    if (WHAT == Product::kSquare || !g.tall) x.diag = g.diag[z * g.diag_stride + r];
    if constexpr (WHAT == Product::kMuon) {
      if (row < g.M && col < g.N) {
        const float* m = g.master + (static_cast<int64_t>(z) * g.M + row) * g.N + col;
        if (g.vectors) {  // N is a multiple of 8
          x.master[0] = *reinterpret_cast<const f32x4*>(m);
          x.master[1] = *reinterpret_cast<const f32x4*>(m + 4);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x.master[e >> 2][e & 3] = m[col + e < g.N ? e : 0];
        }
      }
    }
  }
}

// Eight results of one row from their sums: what is kept of them in binary16
// (zero outside the matrix), after what the epilogue stores itself. dc: the
// diagonal along the columns (kSquare; the others where g.tall); mask: the
// columns inside the matrix.
template <Product WHAT, int OUT>
__device__ __forceinline__ half8 finish(const ProductGroup& g, const ProductScales& s, int z,
                                        int row, int col, const float (&sum)[8],
                                        const Operands<WHAT>& x, const float (&dc)[8],
                                        u32x4 mask) {
  const bool row_in = row < g.M;
  const int64_t at = z * g.c_stride + static_cast<int64_t>(row) * g.ldc + col;
  half8 h;
  if constexpr (WHAT == Product::kGram || WHAT == Product::kSquare) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (WHAT == Product::kGram)
        h[e] = static_cast<_Float16>(sum[e] * s.acc);
      else
        h[e] = static_cast<_Float16>(fma(fma(s.diag, x.diag + dc[e], s.linear),
                                         static_cast<float>(x.hi[e]), s.acc * sum[e]));
    }
    if (row_in && row >= col && row < col + 8) {  // the lane that holds a diagonal element
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (row == col + e) {
          if constexpr (WHAT == Product::kGram)
            g.diag_out[z * g.diag_stride + row] = sum[e] * s.acc;
          else
            g.diag_out[z * g.diag_stride + row] =
                (s.linear * x.diag + (s.diag * (x.diag * x.diag) + s.acc * sum[e])) * s.out;
          h[e] = static_cast<_Float16>(0.0f);
        }
    }
  } else if constexpr (WHAT == Product::kUpdate) {
    u32x2 l = {};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float hi = static_cast<float>(x.hi[e]);
      const int lo = static_cast<int>(x.lo[e >> 2] << (24 - 8 * (e & 3))) >> 24;
      const float d = s.diag * (g.tall ? dc[e] : x.diag);
      const float v =
          settled(fma(s.linear, with_low_byte(hi, lo), fma(d, hi, s.acc * sum[e])));
      h[e] = static_cast<_Float16>(v);
      l[e >> 2] |= (static_cast<uint32_t>(low_byte(v, h[e])) & 0xFFu) << (8 * (e & 3));
    }
    if (g.c_lo != nullptr && row_in && col < g.ldc)
      store_through(l, g.c_lo + at);
  } else if (row_in && col < g.N) {
    const bool whole = g.vectors && col + 8 <= g.N;
    float v[8];
    u16x8 w;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = s.diag * (g.tall ? dc[e] : x.diag);
      v[e] = fma(s.linear + d, static_cast<float>(x.hi[e]), s.acc * sum[e]);
      if constexpr (WHAT == Product::kMuon)
        v[e] = x.master[e >> 2][e & 3] * s.decay - g.step * v[e];
      w[e] = OUT == kBf16 ? bf16_bits(v[e]) : fp16_bits(v[e]);
    }
    uint16_t* o = static_cast<uint16_t*>(g.out);
    if constexpr (WHAT == Product::kOut) {
      o += z * g.out_stride + row * g.out_ld + col;
    } else {
      const int64_t k = (static_cast<int64_t>(z) * g.M + row) * g.N + col;
      float* m = g.master + k;
      if (whole) {
        *reinterpret_cast<f32x4*>(m) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(m + 4) = f32x4{v[4], v[5], v[6], v[7]};
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < g.N) m[e] = v[e];
      }
      o += k;
    }
    if constexpr (OUT >= 0) {
      if (whole) {
        store_through(w, o);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < g.N) o[e] = w[e];
      }
    }
  }
  if constexpr (WHAT == Product::kGram || WHAT == Product::kSquare || WHAT == Product::kUpdate) {
    const uint32_t r = row_in ? ~0u : 0u;
    h = keep(h, mask & u32x4{r, r, r, r});
    if (row_in && col < g.ldc)
      *reinterpret_cast<half8*>(reinterpret_cast<_Float16*>(g.c) + at) = h;
    return h;
  }
  return half8{};
}

template <Product WHAT, int OUT, int MT, int NT, int WM, int WN, int BUFFERS>
__global__ __launch_bounds__(64 * WM * WN, 1) void product_kernel(ProductArgs a) {
  using T = Tile<MT, NT, WM, WN, BUFFERS>;
  constexpr bool SYM = WHAT == Product::kGram || WHAT == Product::kSquare;
  constexpr bool TURN = SYM || WHAT == Product::kUpdate;
  __shared__ __align__(1024) _Float16 lds[BUFFERS * T::stage];
  if (a.skip != nullptr && *a.skip != 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave / WN) * 32 * MT, wn = (wave % WN) * 32 * NT;
  const int64_t total = a.tile_end[a.count - 1];

  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    int gi = 0;
    while (w >= a.tile_end[gi]) ++gi;
    const ProductGroup& g = a.g[gi];
    const int64_t first = gi ? a.tile_end[gi - 1] : 0;
    const int64_t local = xcd_order(w - first, a.tile_end[gi] - first);
    // in 32 bits where they suffice: a 64-bit division is a routine
    int z, t;
    if (total <= 0x7fffffff) {
      z = static_cast<int>(static_cast<uint32_t>(local) / static_cast<uint32_t>(a.tiles[gi]));
      t = static_cast<int>(local) - z * a.tiles[gi];
    } else {
      z = static_cast<int>(local / a.tiles[gi]);
      t = static_cast<int>(local % a.tiles[gi]);
    }
    int ti, tj;
    if constexpr (SYM) triangle(t, a.tiles_m[gi], ti, tj);
    else rectangle(t, a.tiles_m[gi], a.tiles_n[gi], ti, tj);
    const int row0 = ti * T::rows, col0 = tj * T::cols;

    // A row past the matrix is its last one again: its results are not kept.
    // Offsets are 32 bits from the tile's first row (at most 256 rows of 2
    // MiB).
    const int64_t p_first = static_cast<int64_t>(z) * g.p_stride + static_cast<int64_t>(row0) * g.ldp;
    const int64_t q_first = static_cast<int64_t>(z) * g.q_stride + static_cast<int64_t>(col0) * g.ldq;
    const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<half_bits*>(g.p + p_first), 0, kRsrcRange, kRsrcWord3);
    const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<half_bits*>(g.q + q_first), 0, kRsrcRange, kRsrcWord3);
    int po[T::p_copies], qo[T::q_copies];
    auto offset = [&](int c, int most, int ld) {
      const int r = (c * T::waves + wave) * T::copy_rows + lane / T::pieces;
      return (r < most ? r : most) * ld * 2 + (T::slot(r, lane % T::pieces) << 4);
    };
#pragma unroll
    for (int c = 0; c < T::p_copies; ++c) po[c] = offset(c, g.M - 1 - row0, g.ldp);
#pragma unroll
    for (int c = 0; c < T::q_copies; ++c) qo[c] = offset(c, g.N - 1 - col0, g.ldq);
    // copies [from, to) of stage k
    auto copy = [&](int k, int buffer, int from, int to) {
      _Float16* base = lds + buffer * T::stage + wave * T::copy_rows * kDepth;
#pragma unroll
      for (int c = from; c < to; ++c) {
        const bool p = c < T::p_copies;
        copy_to_lds(p ? rp : rq, base + c * T::waves * T::copy_rows * kDepth,
                    p ? po[p ? c : 0] : qo[p ? 0 : c - T::p_copies], k * kDepth * 2);
      }
    };
    auto read = [&](Fragments<MT, NT>& f, int buffer, int step) {
      const _Float16* from = lds + buffer * T::stage;
      const int piece = 2 * step + (lane >> 5);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int r = wm + 32 * i + (lane & 31);
        f.p[i] = *reinterpret_cast<const half8*>(from + r * kDepth + (T::slot(r, piece) << 3));
      }
      from += T::rows * kDepth;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int r = wn + 32 * j + (lane & 31);
        f.q[j] = *reinterpret_cast<const half8*>(from + r * kDepth + (T::slot(r, piece) << 3));
      }
    };
    f32x16 acc[MT][NT] = {};
    auto multiply = [&](const Fragments<MT, NT>& f) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.p[i], f.q[j], acc[i][j], 0, 0, 0);
    };

    // Deals a step's reads of LDS, and behind them `copies` copies, out among
    // its products: a wave that issues its copies in a row waits for the
    // address unit, and its products behind them (measured: 29 % of the time).
    auto interleave = [&](auto copies) {
      constexpr int reads = MT + NT, products = MT * NT, n = decltype(copies)::value;
      constexpr int each = n > 0 ? 1 : products / reads;
#pragma unroll
      for (int i = 0; i < reads; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // LDS read
        __builtin_amdgcn_sched_group_barrier(0x008, each, 0);  // MFMA
      }
#pragma unroll
      for (int i = 0; i < n; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);  // copy
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
      if constexpr (n > 0 && products > reads + n)
        __builtin_amdgcn_sched_group_barrier(0x008, products - reads - n, 0);
      __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int ALL = T::p_copies + T::q_copies;
    constexpr int A = (ALL + 2) / 3, B = (ALL - A + 1) / 2, C = ALL - A - B;
    using Acopies = std::integral_constant<int, A>;
    using Bcopies = std::integral_constant<int, B>;
    using Ccopies = std::integral_constant<int, C>;
    using None = std::integral_constant<int, 0>;
    const int stages = g.K / kDepth;
    Fragments<MT, NT> f[2];
    if constexpr (BUFFERS == 2) {
      // Stage k + 2 takes stage k's buffer: its copies start behind the meeting
      // after stage k's last reads, under the last products of stage k, and go
      // on under the first half of stage k + 1. The loop has no branch that
      // would part the products: past the end the last stage is copied again,
      // into a buffer that nobody reads.
      auto stage = [&](int k) { return k < stages ? k : stages - 1; };
      copy(0, 0, 0, ALL);
      wait_and_meet<0>();
      read(f[0], 0, 0);
      copy(stage(1), 1, 0, A);
      for (int k = 0; k < stages; ++k) {
        const int b = k & 1;
        read(f[1], b, 1);
        copy(stage(k + 1), b ^ 1, A, A + B);
        multiply(f[0]);
        interleave(Bcopies());
        read(f[0], b, 2);
        copy(stage(k + 1), b ^ 1, A + B, ALL);
        multiply(f[1]);
        interleave(Ccopies());
        read(f[1], b, 3);
        multiply(f[0]);
        interleave(None());
        wait_and_meet<0>();
        read(f[0], b ^ 1, 0);
        copy(stage(k + 2), b, 0, A);
        multiply(f[1]);
        interleave(Acopies());
      }
      wait_and_meet<0>();
    } else {
#pragma unroll
      for (int k = 0; k < BUFFERS - 1; ++k)
        if (k < stages) copy(k, k, 0, ALL);
      if (stages >= BUFFERS - 1) wait_and_meet<T::in_flight>();
      else wait_and_meet<0>();
      read(f[0], 0, 0);
      int buffer = 0;
      for (int k = 0; k < stages; ++k) {
        const int next = buffer + 1 == BUFFERS ? 0 : buffer + 1;
        const int last = buffer == 0 ? BUFFERS - 1 : buffer - 1;
        const bool more = k + BUFFERS - 1 < stages;
        if (more) copy(k + BUFFERS - 1, last, 0, ALL);
#pragma unroll
        for (int step = 1; step < kDepth / 16; ++step) {
          read(f[step & 1], buffer, step);
          multiply(f[(step - 1) & 1]);
          interleave(None());
        }
        if (more) wait_and_meet<T::in_flight>();
        else wait_and_meet<0>();
        if (k + 1 < stages) read(f[0], next, 0);
        multiply(f[1]);
        buffer = next;
      }
    }
    // Every wave is past its last read of LDS. The sums change from the
    // accumulators' layout (lane l: column l % 32; register r: row 8 (r / 4) +
    // 4 (l / 32) + r % 4) to eight neighbours of a row per lane through the
    // wave's own part of LDS, 64 columns at a time: rows of 256 bytes, whose
    // halves are exchanged every four rows. Their binary16 form goes back into
    // the first half of the row it came from, at 16-byte piece ^ (row / 8 % 8),
    // to be stored turned. The loops are not unrolled: a tile's epilogue would
    // be more code than the instruction cache holds.
    float* sums = reinterpret_cast<float*>(lds) + wave * (32 * MT * 64);
    _Float16* turn = reinterpret_cast<_Float16*>(sums);
    const bool mirror = TURN && (!SYM || ti != tj);
    const int k8 = (lane & 7) * 8;
#pragma unroll 1
    for (int cj = 0; cj < NT / 2; ++cj) {
      const int rowc = row0 + wm, colw = col0 + wn + 64 * cj;
      float dc[8] = {};
      if constexpr (WHAT != Product::kGram) {
        if (WHAT == Product::kSquare || g.tall) {
          const int c = colw + k8 < g.ldc ? colw + k8 : g.ldc - 8;
          const f32x4* d = reinterpret_cast<const f32x4*>(g.diag + z * g.diag_stride + c);
          *reinterpret_cast<f32x4*>(dc) = d[0];
          *reinterpret_cast<f32x4*>(dc + 4) = d[1];
        }
      }
      u32x4 mask;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = colw + k8 + 2 * e;
        mask[e] = c + 1 < g.N ? ~0u : c < g.N ? 0xFFFFu : 0u;
      }
      Operands<WHAT> next[4];
      auto load = [&](int i) {
#pragma unroll
        for (int p = 0; p < 4; ++p)
          load_operands(next[p], g, z, rowc + 32 * i + 8 * p + (lane >> 3), colw + k8);
      };
      load(0);
#pragma unroll
      for (int c = 0; c < NT / 2; ++c) {
        if (c != cj) continue;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int r = 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
              sums[r * 64 + ((32 * j + (lane & 31)) ^ ((lane >> 5) << 5))] = acc[i][2 * c + j][e];
            }
      }
      wave_fence();
#pragma unroll 1
      for (int i = 0; i < MT; ++i) {
        Operands<WHAT> x[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) x[p] = next[p];
        if (i + 1 < MT) load(i + 1);
        float v[4][8];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int r = 32 * i + 8 * p + (lane >> 3);
          const float* from = sums + r * 64 + (k8 ^ (((r >> 2) & 1) << 5));
          *reinterpret_cast<f32x4*>(v[p]) = *reinterpret_cast<const f32x4*>(from);
          *reinterpret_cast<f32x4*>(v[p] + 4) = *reinterpret_cast<const f32x4*>(from + 4);
        }
        if constexpr (TURN) wave_fence();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int r = 32 * i + 8 * p + (lane >> 3);
          const half8 h =
              finish<WHAT, OUT>(g, a.s, z, rowc + r, colw + k8, v[p], x[p], dc, mask);
          if constexpr (TURN)
            *reinterpret_cast<half8*>(turn + r * 128 + (((lane & 7) ^ ((r >> 3) & 7)) << 3)) = h;
        }
      }
      if (mirror) {
        wave_fence();
        _Float16* to = reinterpret_cast<_Float16*>(SYM ? g.c : g.turned) +
                       static_cast<int64_t>(z) * (SYM ? g.c_stride : g.turned_stride);
        const int ld = SYM ? g.ldc : g.ld_turned;
        // 64 rows (32 where the wave has no more) and a column per lane
        constexpr int ACROSS = MT > 1 ? 8 : 4;
        const int r = (lane % ACROSS) * 8;
#pragma unroll 2
        for (int p = 0; p < ACROSS; ++p) {
          const int k = (64 / ACROSS) * p + lane / ACROSS;
#pragma unroll
          for (int c = 0; c < (MT + 1) / 2; ++c) {
            half8 h;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              h[e] = turn[(64 * c + r + e) * 128 + (((k >> 3) ^ (lane % ACROSS)) << 3) + (k & 7)];
            const int row = rowc + 64 * c + r;
            if (colw + k < g.N && row < ld)
              *reinterpret_cast<half8*>(to + static_cast<int64_t>(colw + k) * ld + row) = h;
          }
        }
      }
      wave_fence();
    }
    wait_and_meet<0>();  // LDS is free for the next tile, and no store is counted with its copies
  }
}

template <Product WHAT, int OUT, int MT, int NT, int WM, int WN, int BUFFERS>
hipError_t launch_tile(const ProductGroup* groups, int count, const ProductScales& s,
                       const int32_t* skip, hipStream_t stream, int64_t max_grid) {
  using T = Tile<MT, NT, WM, WN, BUFFERS>;
  constexpr bool SYM = WHAT == Product::kGram || WHAT == Product::kSquare;
  // The tiles of the longest sums first: the short ones fill the last round's
  // gaps (the 14B-shaped layer's X X^T: 2.05 -> 1.4 ms).
  int order[kGroupsPerLaunch];
  for (int i = 0; i < count; ++i) order[i] = i;
  std::stable_sort(order, order + count,
                   [&](int x, int y) { return groups[x].K > groups[y].K; });
  ProductArgs a = {};
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    const ProductGroup& g = a.g[i] = groups[order[i]];
    const int64_t tm = (g.M + T::rows - 1) / T::rows;
    const int64_t tn = (g.N + T::cols - 1) / T::cols;
    const int64_t tiles = SYM ? tm * (tm + 1) / 2 : tm * tn;
    a.tiles_m[i] = static_cast<int32_t>(tm);
    a.tiles_n[i] = static_cast<int32_t>(tn);
    a.tiles[i] = static_cast<int32_t>(tiles);
    total += tiles * g.count;
    a.tile_end[i] = total;
  }
  a.s = s;
  a.skip = skip;
  a.count = count;
  int64_t grid = total < kMaxWorkgroups ? total : kMaxWorkgroups;
  if (grid > max_grid) grid = max_grid;
  void* params[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(&product_kernel<WHAT, OUT, MT, NT, WM, WN, BUFFERS>),
                         dim3(static_cast<unsigned>(grid)), dim3(T::threads), params, 0, stream);
}

template <Product WHAT, int OUT>
hipError_t launch_one(const ProductGroup* groups, int count, const ProductScales& s,
                      const int32_t* skip, hipStream_t stream, int64_t max_grid) {
  constexpr bool SYM = WHAT == Product::kGram || WHAT == Product::kSquare;
  // A workgroup has a compute unit to itself, or half of one in the smallest
  // tile. One of 256 x 256 takes 5/3 of the time of one of 128 x 128 (K = 4096:
  // 84 us to 50 us), and that half as much again as one of 64 x 64 (K = 256: 12
  // us to 8 us; 4096 x 2560, where 820 small tiles make two rounds and 210 of
  // 128 one: 49 us to 61 us): the size whose rounds take least.
  auto rounds = [&](int64_t side, int64_t slots) {
    int64_t tiles = 0;
    for (int i = 0; i < count; ++i) {
      const int64_t tm = (groups[i].M + side - 1) / side, tn = (groups[i].N + side - 1) / side;
      tiles += (SYM ? tm * (tm + 1) / 2 : tm * tn) * groups[i].count;
    }
    return (tiles + slots - 1) / slots;
  };
  const int64_t large = 5 * rounds(256, 256), medium = 3 * rounds(128, 256),
                small = 2 * rounds(64, 512);
  if (large < medium && large < small)
    return launch_tile<WHAT, OUT, 4, 4, 2, 2, 2>(groups, count, s, skip, stream, max_grid);
  if (small < medium)
    return launch_tile<WHAT, OUT, 1, 2, 2, 1, 4>(groups, count, s, skip, stream, max_grid);
  return launch_tile<WHAT, OUT, 2, 2, 2, 2, 4>(groups, count, s, skip, stream, max_grid);
}

}  // namespace

hipError_t launch_product(const ProductGroup* groups, int count, Product what, int out_type,
                          const ProductScales& s, const int32_t* skip, hipStream_t stream,
                          int64_t max_grid) {
  switch (what) {
    case Product::kGram: return launch_one<Product::kGram, 0>(groups, count, s, skip, stream, max_grid);
    case Product::kSquare: return launch_one<Product::kSquare, 0>(groups, count, s, skip, stream, max_grid);
    case Product::kUpdate: return launch_one<Product::kUpdate, 0>(groups, count, s, skip, stream, max_grid);
    case Product::kOut:
      return out_type == kFp16 ? launch_one<Product::kOut, kFp16>(groups, count, s, skip, stream, max_grid)
                               : launch_one<Product::kOut, kBf16>(groups, count, s, skip, stream, max_grid);
    default:
      return out_type == kFp16   ? launch_one<Product::kMuon, kFp16>(groups, count, s, skip, stream, max_grid)
             : out_type == kBf16 ? launch_one<Product::kMuon, kBf16>(groups, count, s, skip, stream, max_grid)
                                 : launch_one<Product::kMuon, -1>(groups, count, s, skip, stream, max_grid);
  }
}

}  // namespace la
