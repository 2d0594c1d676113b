// la_narrow.hip -- the orthogonalised update of narrow matrices (short side m
// at most 128) for gfx950.
//
// Every step multiplies X by a polynomial in S = X X^T, and these commute: so
// S and the product Q of the steps' factors are carried along as m x m
// matrices,
//
//   S_0 = X_0 X_0^T;  P = a + b S + c S S;  Q <- P Q;  S <- P S P
//
// and X is read for its norm (in a Muon step the momentum pass has formed it),
// for S_0 and for O = Q X_0, where the step-by-step form reads and writes it in
// every step. What the short form asks for is precision: an error in S grows by
// up to a^2 per step where the singular values are small. Every operand here is
// a pair of binary16 numbers (hi + lo / 2^11, 22 bits) under a power-of-two
// scale from the host's bounds, every product the three hi hi + hi lo + lo hi
// with binary32 sums: measured 1e-6 to 8e-4 of the direction, less than the
// step-by-step form's (few elements that are not zero: up to 3e-3). The long sums
// of S_0 are binary32 over 64 columns and binary64 beyond: in binary32 alone, on
// a matrix with one strong direction, the last bits of its sum would swallow the
// others (520 of 4 x 20000 with a strong column: 49 % off).
//
// m x m matrices of up to 128 x 128 live in the registers of one workgroup, in
// the accumulators' layout, and pass through LDS (two operands of 64 KiB) to be
// multiplied. They are symmetric up to rounding, so the layout's four
// consecutive rows of one column are stored as four consecutive columns of one
// row. 17 products in turn decide there (14 of them a chain): 74 us for five
// steps at 128 x 128, 4.4 us a product; one 64 x 64 matrix, all parts in one
// workgroup, 40 us. The parts over X are bound by its conversion and by LDS: S
// of 40 matrices of 128 x 5120 takes 63 us (58 us from FP32), Q X 79 us (52 MB
// each way).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "la_muon.h"

#pragma clang fp contract(off)

namespace la {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct NarrowArgs {
  NarrowGroup g[kGroupsPerLaunch];
  int64_t end[kGroupsPerLaunch];  // cumulative workgroups
  NarrowPlan plan;
  const int32_t* skip;
  int32_t count;
};
static_assert(sizeof(NarrowArgs) <= 4096, "kernel arguments");

template <int TYPE, typename Raw>
__device__ __forceinline__ float decode(Raw v) {
  if constexpr (TYPE == kFp32) return v;
  else if constexpr (TYPE == kFp16) return static_cast<float>(__builtin_bit_cast(_Float16, v));
  else return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

__device__ __forceinline__ uint16_t bits16(float x, int type) {
  const uint32_t b = __float_as_uint(x);
  const uint32_t r = (b + 0x7FFFu + ((b >> 16) & 1u)) >> 16;
  const uint16_t h = __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
  const bool nan = __builtin_isnan(x);
  return type == kFp16 ? (nan ? uint16_t(0x7E00) : h) : static_cast<uint16_t>(nan ? 0x7FC0u : r);
}

// Where 16-byte piece p of row r of an operand with K elements a row is kept,
// so that 32 rows' reads of one piece meet every bank equally often.
template <int K>
__device__ __forceinline__ int slot(int r, int p) {
  return K == 64 ? p ^ ((r >> 1) & 7) : p ^ (r & 15);
}

template <int MP, int TYPE, NarrowPart PART>
__global__ __launch_bounds__(MP == 128 ? 512 : 256, PART == NarrowPart::kWhole ? 1 : 2)
void narrow_kernel(NarrowArgs a) {
  using Raw = std::conditional_t<TYPE == kFp32, float, uint16_t>;
  constexpr int WAVES = MP == 128 ? 8 : 4, THREADS = 64 * WAVES, BJ = MP / 64;
  constexpr int OPERAND = 2 * MP * MP;  // elements: hi, then lo
  constexpr int LO = MP * MP;           // of an m x m operand
  constexpr int XLO = MP * 64;          // of a block of X
  constexpr int PER = MP * 64 / THREADS;
  static_assert(PER == 16, "sixteen elements of a block per thread");
  // an m x m operand; another, or two blocks of X
  __shared__ __align__(1024) _Float16 lds[OPERAND + (OPERAND > 4 * XLO ? OPERAND : 4 * XLO)];
  __shared__ double sums[WAVES];
  if (a.skip != nullptr && *a.skip != 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32 * BJ;
  _Float16* const first_operand = lds;
  _Float16* const second = lds + OPERAND;
  constexpr bool whole = PART == NarrowPart::kWhole;
  const int64_t total = a.end[a.count - 1];

  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    int gi = 0;
    while (w >= a.end[gi]) ++gi;
    const NarrowGroup& g = a.g[gi];
    const int64_t local = w - (gi ? a.end[gi - 1] : 0);
    const bool tall = g.rows > g.cols;
    const int m = tall ? g.cols : g.rows, n = tall ? g.rows : g.cols;
    const int parts = PART == NarrowPart::kSum || PART == NarrowPart::kApply ? g.splits : 1;
    const int64_t z = local / parts;
    const int split = static_cast<int>(local % parts);
    const int first = whole ? 0 : split * g.chunk;
    const int last = whole || first + g.chunk > n ? n : first + g.chunk;
    const int64_t source = z * g.matrix_stride;

    // Element e of this thread in a block of 64 columns of X (m x n): along the
    // axis on which the matrix is contiguous, a short row's 64 lanes shared by
    // as many columns as fit, and eight neighbours of the other axis in a row.
    // False, for the whole wave, past the block.
    int log = 0;
    while ((1 << log) < m && log < 6) ++log;
    auto place = [&](int e, int& i, int& c) {
      if (!tall) {
        c = lane;
        i = 8 * (wave + WAVES * (e >> 3)) + (e & 7);
        return i < m;
      }
      if (MP == 128) {
        c = 8 * wave + (e & 7);
        i = lane + 64 * (e >> 3);
        return true;
      }
      const int unit = wave + WAVES * e;
      c = (unit << (6 - log)) + (lane >> log);
      i = lane & ((1 << log) - 1);
      return (unit << (6 - log)) < 64;
    };
    // Raw elements, from inside the matrix whatever the place: a load under a
    // condition would be waited for before the next is asked for (measured: two
    // and a half times the time of the whole sum).
    auto fetch = [&](Raw (&v)[PER], int c0) {
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        int i, c;
        place(e, i, c);
        i = i < m ? i : m - 1;
        c = c < 64 ? c : 63;
        c = c0 + c < last ? c0 + c : last - 1;
        const Raw* from = static_cast<const Raw*>(g.in) + source;
        if (tall && MP == 64) {
          v[e] = from[c * g.row_stride + i];
        } else {  // the row is the wave's
          const int row = __builtin_amdgcn_readfirstlane(tall ? c : i);
          v[e] = (from + row * g.row_stride)[static_cast<uint32_t>(tall ? i : c)];
        }
      }
    };
    auto value = [&](Raw v, int i, int c) {
      return i < m && c < last ? decode<TYPE>(v) : 0.0f;
    };

    double factor = 0.0;
    if constexpr (PART != NarrowPart::kFactor) {
      double sum = 0.0;
      if (g.partial != nullptr) {
        for (int k = tid; k < g.partials; k += THREADS) sum += g.partial[z * g.partials + k];
      } else {
        for (int c0 = 0; c0 < n; c0 += 64) {
          Raw v[PER];
          fetch(v, c0);
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            int i, c;
            const bool in = place(e, i, c);
            const double x = in ? value(v[e], i, c0 + c) : 0.0f;
            sum += x * x;
          }
        }
      }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
      if (lane == 0) sums[wave] = sum;
      __syncthreads();
      sum = sums[0];
      for (int k = 1; k < WAVES; ++k) sum += sums[k];
      const double norm = __builtin_sqrt(sum);
      const double denominator = norm < a.plan.eps ? a.plan.eps : norm;  // NaN stays
      if (denominator > 0.0) factor = __builtin_ldexp(1.0, a.plan.x) / denominator;
      if (!(sum < __builtin_inf())) factor = __builtin_nan("");
    }
    // As a power of two and a binary32 number in [1/2, 1): its rounding scales the
    // whole matrix by 1 + 2^-25 at most, and no x is out of range on the way.
    const int factor_exponent = __builtin_amdgcn_frexp_exp(factor);
    const float factor_mantissa = static_cast<float>(__builtin_amdgcn_frexp_mant(factor));

    // A block of X as an operand: rows i, summed over c (turned: rows c, summed
    // over i). Rows i past the last one that place() gives stay as they were.
    // Where a thread's neighbours are a row's, eight go to LDS at once (40 of 128
    // x 5120: Q X in 80 us, 91 us one by one).
    auto put = [&](const Raw (&v)[PER], int c0, _Float16* to, bool turned) {
      auto split = [&](int e, int i, int c, _Float16& hi, _Float16& lo) {
        const float x = settled(
            __builtin_ldexpf(value(v[e], i, c0 + c), factor_exponent) * factor_mantissa);
        hi = static_cast<_Float16>(x);
        lo = static_cast<_Float16>((x - static_cast<float>(hi)) * 0x1p11f);
      };
      if (turned ? !tall : tall && MP == 128) {
#pragma unroll
        for (int h = 0; h < PER / 8; ++h) {
          half8 hi, lo;
          int i, c;
          if (!place(8 * h, i, c)) continue;
          const int at = turned ? c * MP + slot<MP>(c, i >> 3) * 8
                                : i * 64 + slot<64>(i, c >> 3) * 8;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            _Float16 a, b;
            place(8 * h + e, i, c);
            split(8 * h + e, i, c, a, b);
            hi[e] = a;
            lo[e] = b;
          }
          *reinterpret_cast<half8*>(to + at) = hi;
          *reinterpret_cast<half8*>(to + XLO + at) = lo;
        }
        return;
      }
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        int i, c;
        if (!place(e, i, c)) continue;
        const int at = turned ? c * MP + slot<MP>(c, i >> 3) * 8 + (i & 7)
                              : i * 64 + slot<64>(i, c >> 3) * 8 + (c & 7);
        split(e, i, c, to[at], to[XLO + at]);
      }
    };

    // acc += P Q^T over 16 * depth elements for the wave's 32 rows of P and blocks of 32 rows of
    // Q; low parts, hi lo and lo hi, in sums of their own, 2^11 times as large
    // (three chains of matrix instructions that do not wait for each other).
    auto multiply = [&](auto k_const, auto blocks, const _Float16* p, int p_lo, int p_row,
                        const _Float16* q, int q_lo, int q_row, int depth, f32x16* acc,
                        f32x16* low) {
      constexpr int K = decltype(k_const)::value, BLOCKS = decltype(blocks)::value;
      const int r = p_row + (lane & 31);
      constexpr bool APART = BLOCKS == 1;  // two blocks have chains enough
      constexpr int PAIR = BLOCKS == 1 ? 2 : 1;
      f32x16 other[BLOCKS] = {};
#pragma unroll 1
      for (int k0 = 0; k0 < depth; k0 += PAIR)
#pragma unroll
        for (int h = 0; h < PAIR; ++h) {
          const int piece = 2 * (k0 + h) + (lane >> 5);
          const _Float16* pp = p + r * K + slot<K>(r, piece) * 8;
          const half8 ph = *reinterpret_cast<const half8*>(pp);
          const half8 pl = *reinterpret_cast<const half8*>(pp + p_lo);
#pragma unroll
          for (int j = 0; j < BLOCKS; ++j) {
            const int s = q_row + 32 * j + (lane & 31);
            const _Float16* qq = q + s * K + slot<K>(s, piece) * 8;
            const half8 qh = *reinterpret_cast<const half8*>(qq);
            const half8 ql = *reinterpret_cast<const half8*>(qq + q_lo);
            acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph, qh, acc[j], 0, 0, 0);
            low[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ph, ql, low[j], 0, 0, 0);
            f32x16& last_low = APART ? other[j] : low[j];
            last_low = __builtin_amdgcn_mfma_f32_32x32x16_f16(pl, qh, last_low, 0, 0, 0);
          }
        }
      if constexpr (APART)
#pragma unroll
        for (int e = 0; e < 16; ++e) low[0][e] += other[0][e];
    };
    const int deep = ((m + 31) >> 5) * 2;  // past m every operand is zero
    using Side = std::integral_constant<int, MP>;
    using Stage = std::integral_constant<int, 64>;
    using Blocks = std::integral_constant<int, BJ>;
    using One = std::integral_constant<int, 1>;

    // The m x m matrices, in the accumulators' layout.
    f32x16 S[BJ] = {}, Q[BJ] = {};
    // P Q^T of two m x m operands, times 2^-e
    auto product = [&](const _Float16* p, const _Float16* q, int e, f32x16 (&out)[BJ]) {
      f32x16 acc[BJ] = {}, low[BJ] = {};
      multiply(Side(), Blocks(), p, LO, wm, q, LO, wn, deep, acc, low);
      const float f = __builtin_ldexpf(1.0f, -e);
#pragma unroll
      for (int j = 0; j < BJ; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) out[j][k] = (acc[j][k] + low[j][k] * 0x1p-11f) * f;
    };
    auto store = [&](const f32x16 (&v)[BJ], _Float16* to, int e) {
      const float f = __builtin_ldexpf(1.0f, e);
#pragma unroll
      for (int j = 0; j < BJ; ++j) {
        const int row = wn + 32 * j + (lane & 31);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          half4 hi, lo;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float x = v[j][4 * q + k] * f;  // exact
            hi[k] = static_cast<_Float16>(x);
            lo[k] = static_cast<_Float16>((x - static_cast<float>(hi[k])) * 0x1p11f);
          }
          _Float16* at = to + row * MP + slot<MP>(row, (wm >> 3) + q) * 8 + 4 * (lane >> 5);
          *reinterpret_cast<half4*>(at) = hi;
          *reinterpret_cast<half4*>(at + LO) = lo;
        }
      }
    };

    if constexpr (whole || PART == NarrowPart::kSum) {
      // hi hi, block by block: low is 2^11 times finer than what its sums lose
      double total[BJ][16] = {};
      f32x16 low[BJ] = {};
      Raw v[PER];
      fetch(v, first);
      int b = 0;
      for (int c0 = first; c0 < last; c0 += 64, b ^= 1) {
        put(v, c0, lds + b * OPERAND, false);
        __syncthreads();
        if (c0 + 64 < last) fetch(v, c0 + 64);
        f32x16 acc[BJ] = {};
        multiply(Stage(), Blocks(), lds + b * OPERAND, XLO, wm, lds + b * OPERAND, XLO, wn, 4,
                 acc, low);
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k) total[j][k] += acc[j][k];
      }
      __syncthreads();
      const double f = __builtin_ldexp(1.0, -2 * a.plan.x);
#pragma unroll
      for (int j = 0; j < BJ; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int row = wm + 8 * (k >> 2) + 4 * (lane >> 5) + (k & 3);
          const int col = wn + 32 * j + (lane & 31);
          // rows past m were not written: what their sums hold is not used
          const double sum = (total[j][k] + low[j][k] * 0x1p-11f) * f;
          S[j][k] = row < m && col < m ? static_cast<float>(sum) : 0.0f;
        }
      if (!whole) {
        float* to = g.gram + (z * g.splits + split) * (MP * MP) + wave * (BJ * 1024) + lane;
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k) to[(16 * j + k) * 64] = S[j][k];
      }
    }
    if (PART == NarrowPart::kFactor && wm < m && wn < m) {
      // in the parts' order; several of them on their way at once
      constexpr int AHEAD = 4 / BJ;
      double sum[BJ][16] = {};
      const float* from = g.gram + z * g.splits * (MP * MP) + wave * (BJ * 1024) + lane;
      for (int s = 0; s < g.splits; s += AHEAD) {
        f32x16 part[AHEAD][BJ];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const int t = s + u < g.splits ? s + u : g.splits - 1;
#pragma unroll
          for (int j = 0; j < BJ; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k) part[u][j][k] = from[t * (MP * MP) + (16 * j + k) * 64];
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
          if (s + u < g.splits)
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
              for (int k = 0; k < 16; ++k) sum[j][k] += part[u][j][k];
      }
#pragma unroll
      for (int j = 0; j < BJ; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) S[j][k] = static_cast<float>(sum[j][k]);
    }

    if constexpr (whole || PART == NarrowPart::kFactor) {
      store(S, first_operand, a.plan.step[0].s);
      __syncthreads();
#pragma unroll 1
      for (int k = 0; k < a.plan.steps; ++k) {
        const NarrowStep& t = a.plan.step[k];
        const bool more = k + 1 < a.plan.steps;
        f32x16 P[BJ];
        product(first_operand, first_operand, 2 * t.s, P);
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int row = wm + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
            const int col = wn + 32 * j + (lane & 31);
            P[j][e] = (row == col && row < m ? t.a : 0.0f) + (t.b * S[j][e] + t.c * P[j][e]);
          }
        store(P, second, t.p);
        __syncthreads();
        if (more) {
          // An operand stored from V holds V^T: T = S^T P, S <- P^T T; the mean
          // of it and its mirror image, which comes turned through LDS, is
          // symmetric.
          f32x16 T[BJ];
          product(first_operand, second, t.p + t.s, T);
          __syncthreads();
          store(T, first_operand, t.t);
          __syncthreads();
          product(second, first_operand, t.t + t.p, S);
          __syncthreads();
          float* const turn = reinterpret_cast<float*>(first_operand);
          auto at = [&](int row, int col) { return row * MP + (col ^ (row & 31)); };
#pragma unroll
          for (int j = 0; j < BJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              turn[at(wm + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3),
                      wn + 32 * j + (lane & 31))] = S[j][e];
          __syncthreads();
#pragma unroll
          for (int j = 0; j < BJ; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              S[j][e] = 0.5f * (S[j][e] + turn[at(wn + 32 * j + (lane & 31),
                                                  wm + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3))]);
          __syncthreads();
        }
        if (k == 0) {
#pragma unroll
          for (int j = 0; j < BJ; ++j) Q[j] = P[j];
        } else {
          const int before = a.plan.step[k - 1].q;
          store(Q, first_operand, before);
          __syncthreads();
          product(second, first_operand, t.p + before, Q);
          __syncthreads();
        }
        if (more) store(S, first_operand, a.plan.step[k + 1].s);
        __syncthreads();
      }
      store(Q, first_operand, a.plan.step[a.plan.steps - 1].q);
      __syncthreads();
      if (!whole) {
        half8* to = reinterpret_cast<half8*>(g.q + z * OPERAND);
        for (int k = tid; k < OPERAND / 8; k += THREADS)
          to[k] = reinterpret_cast<const half8*>(first_operand)[k];
      }
    }

    if constexpr (whole || PART == NarrowPart::kApply) {
      if (!whole) {
        const half8* from = reinterpret_cast<const half8*>(g.q + z * OPERAND);
        for (int k = tid; k < OPERAND / 8; k += THREADS)
          reinterpret_cast<half8*>(first_operand)[k] = from[k];
      }
      // Tiles of 64 columns, one 32 x 32 block per wave; two blocks of X take
      // turns in the second buffer. Lanes run along the axis on which the
      // result is contiguous.
      const int wi = (wave >> 1) * 32, wj = (wave & 1) * 32;
      const float f =
          __builtin_ldexpf(1.0f, -(a.plan.x + a.plan.step[a.plan.steps - 1].q));
      Raw v[PER];
      fetch(v, first);
      // the rows past m are summed over here, against zeros of Q
      for (int k = tid; k < 4 * XLO / 8; k += THREADS)
        reinterpret_cast<half8*>(second)[k] = half8{};
      __syncthreads();
      int b = 0;
      for (int c0 = first; c0 < last; c0 += 64, b ^= 1) {
        _Float16* x = second + b * 2 * XLO;
        put(v, c0, x, true);
        __syncthreads();
        if (c0 + 64 < last) fetch(v, c0 + 64);
        f32x16 acc[1] = {}, low[1] = {};
        multiply(Side(), One(), tall ? x : first_operand, tall ? XLO : LO, tall ? wj : wi,
                 tall ? first_operand : x, tall ? LO : XLO, tall ? wi : wj, deep, acc, low);
        const int rows = tall ? last : m, cols = tall ? m : last;
        const int row0 = (tall ? c0 + wj : wi) + 4 * (lane >> 5);
        const int col = (tall ? wi : c0 + wj) + (lane & 31);
        // register k holds row row0 + 8 (k / 4) + k % 4
        auto down = [](int k) { return 8 * (k >> 2) + (k & 3); };
        const bool col_in = col < cols;
        float* const master = g.master + ((z * g.rows + row0) * g.cols + col);
        float p[16];
        if (g.master != nullptr) {
#pragma unroll
          for (int k = 0; k < 16; ++k)  // from inside the matrix, as in fetch
            p[k] = *(col_in && row0 + down(k) < rows
                         ? master + static_cast<int64_t>(down(k)) * g.cols
                         : g.master);
        }
        const int64_t stride = g.master != nullptr ? g.cols : g.out_row_stride;
        uint16_t* const out =
            static_cast<uint16_t*>(g.out) +
            (g.master != nullptr ? (z * g.rows + row0) * g.cols
                                 : z * g.out_matrix_stride + row0 * g.out_row_stride) + col;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const bool in = col_in && row0 + down(k) < rows;
          float o = (acc[0][k] + low[0][k] * 0x1p-11f) * f;
          if (g.master != nullptr) {
            o = p[k] * a.plan.decay - g.step * o;
            if (in) master[static_cast<int64_t>(down(k)) * g.cols] = o;
          }
          if (g.out != nullptr && in) out[down(k) * stride] = bits16(o, a.plan.out_type);
        }
      }
    }
    __syncthreads();  // LDS is free for the next matrix
  }
}

// ---- short sides up to 16 ----------------------------------------------------------
// An error in S grows as above whatever the side, but on few directions it does
// not spread: with pairs a 2 x 2 matrix comes out up to 0.4 % off, and the
// step-by-step form's roundings up to 1.4 %. So S, its polynomial and the last
// product are binary64 here, at 16 x 16 x 4 of a matrix instruction: lane l has
// element (l / 16 + 4 r, l % 16) of a result in register r, and gives element (l %
// 16, l / 16) of the left operand and (l / 16, l % 16) of the right one. Register r
// of a symmetric result is therefore an operand as it is, for the four summed
// positions l / 16 + 4 r: a wave multiplies 16 x 16 matrices without LDS, in four
// dependent instructions, and every wave forms the factor for itself. The norm
// is the trace of U U^T, so X is read twice in all. Off by 2e-7 at most over the
// spectra tried. 1 x 1 in 9 us, most of it start and loads; 520 of 8 x 8192 in 280
// us (0.7 TB/s: 16 rows' worth of element-wise loads and matrix instructions for 8),
// 64 of 16 x 4096 in 13 us for S and 21 us for the factor and the result.

typedef double f64x4 __attribute__((ext_vector_type(4)));

// P^T Q
__device__ __forceinline__ f64x4 product16(f64x4 p, f64x4 q) {
  f64x4 s = {};
#pragma unroll
  for (int r = 0; r < 4; ++r) s = __builtin_amdgcn_mfma_f64_16x16x4f64(p[r], q[r], s, 0, 0, 0);
  return s;
}

template <int TYPE, NarrowPart PART>
__global__ __launch_bounds__(256) void tiny_kernel(NarrowArgs a) {
  using Raw = std::conditional_t<TYPE == kFp32, float, uint16_t>;
  constexpr bool whole = PART == NarrowPart::kWhole;
  constexpr int WAVES = 4, STRIP = 32;  // columns that a wave's eight instructions sum over
  __shared__ double share[WAVES][kTiny * kTiny];
  if (a.skip != nullptr && *a.skip != 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int down = lane >> 4, across = lane & 15;
  const int64_t total = a.end[a.count - 1];

  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    int gi = 0;
    while (w >= a.end[gi]) ++gi;
    const NarrowGroup& g = a.g[gi];
    const int64_t local = w - (gi ? a.end[gi - 1] : 0);
    const bool tall = g.rows > g.cols;
    const int m = tall ? g.cols : g.rows, n = tall ? g.rows : g.cols;
    const int parts = whole ? 1 : g.splits;
    const int64_t z = local / parts;
    const int split = static_cast<int>(local % parts);
    const int first = whole ? 0 : split * g.chunk;
    const int last = whole || first + g.chunk > n ? n : first + g.chunk;
    const Raw* const from = static_cast<const Raw*>(g.in) + z * g.matrix_stride;

    // Element (i, c), i along the short side: loaded from inside the matrix
    // whatever the place, so that no load waits for a condition.
    auto fetch = [&](int i, int c) {
      i = i < m ? i : m - 1;
      c = c < last ? c : last - 1;
      return from[tall ? c * g.row_stride + i : i * g.row_stride + c];
    };
    auto value = [&](Raw v, int i, int c) {
      return i < m && c < last ? static_cast<double>(decode<TYPE>(v)) : 0.0;
    };

    f64x4 S = {};
    if constexpr (whole || PART == NarrowPart::kSum) {
      // neighbours along the axis on which the matrix is contiguous
      auto column = [&](int e) { return tall ? 4 * e + down : 8 * down + e; };
      Raw v[8];
      auto load = [&](int c0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fetch(across, c0 + column(e));
      };
      load(first + STRIP * wave);
      for (int c0 = first + STRIP * wave; c0 < last; c0 += STRIP * WAVES) {
        double x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = value(v[e], across, c0 + column(e));
        load(c0 + STRIP * WAVES);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          S = __builtin_amdgcn_mfma_f64_16x16x4f64(x[e], x[e], S, 0, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) share[wave][64 * r + lane] = S[r];
      __syncthreads();
      if constexpr (!whole) {
        double sum = share[0][tid];
#pragma unroll
        for (int k = 1; k < WAVES; ++k) sum += share[k][tid];
        g.sums[(z * g.splits + split) * (kTiny * kTiny) + tid] = sum;
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          S[r] = share[0][64 * r + lane];
#pragma unroll
          for (int k = 1; k < WAVES; ++k) S[r] += share[k][64 * r + lane];
        }
      }
    }
    if constexpr (PART == NarrowPart::kApply) {
      const double* parts_of = g.sums + z * g.splits * (kTiny * kTiny) + lane;
#pragma unroll 4
      for (int t = 0; t < g.splits; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[r] += parts_of[t * (kTiny * kTiny) + 64 * r];
    }

    if constexpr (whole || PART == NarrowPart::kApply) {
      double trace = 0.0;
#pragma unroll
      for (int r = 0; r < 4; ++r) trace += down + 4 * r == across ? S[r] : 0.0;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) trace += __shfl_xor(trace, d, 64);
      const double norm = __builtin_sqrt(trace);
      const double denominator = norm < a.plan.eps ? a.plan.eps : norm;  // NaN stays
      double factor = denominator > 0.0 ? 1.0 / denominator : 0.0;
      if (!(trace < __builtin_inf())) factor = __builtin_nan("");
      S = S * factor * factor;

      f64x4 Q = {};
#pragma unroll 1
      for (int k = 0; k < a.plan.steps; ++k) {
        const double ta = a.plan.step[k].a, tb = a.plan.step[k].b, tc = a.plan.step[k].c;
        f64x4 P = tb * S + tc * product16(S, S);
#pragma unroll
        for (int r = 0; r < 4; ++r) P[r] += down + 4 * r == across && across < m ? ta : 0.0;
        Q = k == 0 ? P : product16(P, Q);
        S = product16(P, product16(S, P));
      }
      Q = Q * factor;

      // 64 columns of X at a time, whose 16 results a lane has at rows (columns
      // where the matrix is tall) down + 4 r and columns (rows) across
      float* const master = g.master;
      uint16_t* const out = static_cast<uint16_t*>(g.out);
      const int64_t base = master != nullptr ? z * g.rows * g.cols : z * g.out_matrix_stride;
      const int64_t stride = master != nullptr ? g.cols : g.out_row_stride;
      const int rows = tall ? last : m, cols = tall ? m : last;
      for (int c0 = first + 64 * wave; c0 < last; c0 += 64 * WAVES) {
        Raw v[4][4];
        float p[4][4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r) v[k][r] = fetch(down + 4 * r, c0 + 16 * k + across);
        auto row = [&](int k, int r) { return (tall ? c0 + 16 * k : 0) + down + 4 * r; };
        auto col = [&](int k) { return (tall ? 0 : c0 + 16 * k) + across; };
        auto inside = [&](int k, int r) { return row(k, r) < rows && col(k) < cols; };
        auto at = [&](int k, int r) { return base + row(k, r) * stride + col(k); };
        if (master != nullptr) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r) p[k][r] = master[inside(k, r) ? at(k, r) : 0];
        }
        float o[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f64x4 O = {};
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const double x = value(v[k][r], down + 4 * r, c0 + 16 * k + across);
            O = __builtin_amdgcn_mfma_f64_16x16x4f64(tall ? x : Q[r], tall ? Q[r] : x, O, 0, 0, 0);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            o[k][r] = static_cast<float>(O[r]);
            if (master != nullptr) o[k][r] = p[k][r] * a.plan.decay - g.step * o[k][r];
          }
        }
        if (master != nullptr) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (inside(k, r)) master[at(k, r)] = o[k][r];
        }
        if (out != nullptr) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (inside(k, r)) out[at(k, r)] = bits16(o[k][r], a.plan.out_type);
        }
      }
    }
    __syncthreads();  // LDS is free for the next matrix
  }
}

template <int MP, int TYPE, NarrowPart PART>
hipError_t launch(NarrowArgs& a, int64_t total, hipStream_t stream, int64_t max_grid) {
  int64_t grid = total < kMaxWorkgroups ? total : kMaxWorkgroups;
  if (grid > max_grid) grid = max_grid;
  void* params[] = {&a};
  const void* kernel;
  if constexpr (MP == kTiny) kernel = reinterpret_cast<const void*>(&tiny_kernel<TYPE, PART>);
  else kernel = reinterpret_cast<const void*>(&narrow_kernel<MP, TYPE, PART>);
  return hipLaunchKernel(kernel, dim3(static_cast<unsigned>(grid)), dim3(MP == 128 ? 512 : 256),
                         params, 0, stream);
}

template <int MP, NarrowPart PART>
hipError_t launch_type(NarrowArgs& a, int64_t total, int type, hipStream_t stream,
                       int64_t max_grid) {
  return type == kFp32   ? launch<MP, kFp32, PART>(a, total, stream, max_grid)
         : type == kFp16 ? launch<MP, kFp16, PART>(a, total, stream, max_grid)
                         : launch<MP, kBf16, PART>(a, total, stream, max_grid);
}

template <int MP>
hipError_t launch_part(NarrowArgs& a, int64_t total, int type, NarrowPart part,
                       hipStream_t stream, int64_t max_grid) {
  switch (part) {
    case NarrowPart::kWhole:
      if constexpr (MP != 128)
        return launch_type<MP, NarrowPart::kWhole>(a, total, type, stream, max_grid);
      else
        return hipErrorInvalidValue;
    case NarrowPart::kSum:
      return launch_type<MP, NarrowPart::kSum>(a, total, type, stream, max_grid);
    case NarrowPart::kFactor:  // reads sums, not directions
      if constexpr (MP != kTiny)
        return launch<MP, kFp32, NarrowPart::kFactor>(a, total, stream, max_grid);
      else
        return hipErrorInvalidValue;
    default:
      return launch_type<MP, NarrowPart::kApply>(a, total, type, stream, max_grid);
  }
}

}  // namespace

hipError_t launch_narrow(const NarrowGroup* groups, int count, int side, int type,
                         NarrowPart part, const NarrowPlan& plan, const int32_t* skip,
                         hipStream_t stream, int64_t max_grid) {
  NarrowArgs a = {};
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    a.g[i] = groups[i];
    const bool split = part == NarrowPart::kSum || part == NarrowPart::kApply;
    total += static_cast<int64_t>(groups[i].count) * (split ? groups[i].splits : 1);
    a.end[i] = total;
  }
  a.plan = plan;
  a.skip = skip;
  a.count = count;
  return side == kTiny ? launch_part<kTiny>(a, total, type, part, stream, max_grid)
         : side == 64  ? launch_part<64>(a, total, type, part, stream, max_grid)
                       : launch_part<128>(a, total, type, part, stream, max_grid);
}

}  // namespace la
