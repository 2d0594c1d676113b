// la_product.hip -- the matrix products of the orthogonalised update for
// gfx950: C = P Q^T over stacks of matrices, with the iteration's epilogues.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "la_muon.h"

#pragma clang fp contract(off)

namespace la {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct ProductArgs {
  ProductGroup g[kGroupsPerLaunch];
  int64_t tile_end[kGroupsPerLaunch];  // cumulative tiles
  int32_t tiles_n[kGroupsPerLaunch];   // tiles along N (square form: along either side)
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

// Tile index within a stack of symmetric results: row i of the lower triangle
// holds the tiles (i, 0) .. (i, i).
__device__ __forceinline__ void triangle(int t, int& i, int& j) {
  int r = static_cast<int>((__builtin_sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
  while (static_cast<int64_t>(r) * (r + 1) / 2 > t) --r;
  while (static_cast<int64_t>(r + 1) * (r + 2) / 2 <= t) ++r;
  i = r;
  j = t - static_cast<int>(static_cast<int64_t>(r) * (r + 1) / 2);
}

// Workgroup w of n runs on XCD w % 8: give each XCD consecutive tiles of
// every 256, so that the tiles its L2 serves share operand rows.
__device__ __forceinline__ int64_t xcd_order(int64_t w, int64_t n) {
  const int64_t base = w & ~int64_t(255);
  const int part = static_cast<int>(n - base < 256 ? n - base : 256);
  const int l = static_cast<int>(w - base), x = l & 7;
  const int q = part >> 3, r = part & 7;
  return base + x * q + (x < r ? x : r) + (l >> 3);
}

template <Product WHAT, int OUT>
__global__ __launch_bounds__(256) void product_kernel(ProductArgs a) {
  constexpr int BM = 128, BN = 128;
  constexpr bool SYM = WHAT == Product::kGram || WHAT == Product::kSquare;
  __shared__ __align__(16) _Float16 sp[2][BM * kDepth];
  __shared__ __align__(16) _Float16 sq[2][BN * kDepth];
  if (a.skip != nullptr && *a.skip != 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  const int64_t total = a.tile_end[a.count - 1];

  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int64_t tile = xcd_order(w, total);
    int gi = 0;
    while (tile >= a.tile_end[gi]) ++gi;
    const ProductGroup& g = a.g[gi];
    const int64_t local = tile - (gi ? a.tile_end[gi - 1] : 0);
    const int z = static_cast<int>(local / a.tiles[gi]);
    const int t = static_cast<int>(local % a.tiles[gi]);
    int ti, tj;
    if constexpr (SYM) {
      triangle(t, ti, tj);
    } else {
      ti = t / a.tiles_n[gi];
      tj = t % a.tiles_n[gi];
    }
    const int row0 = ti * BM, col0 = tj * BN;

    // Thread t loads 16-byte piece (t & 7) of row (t >> 3) + 32 i of each
    // operand's stage; a row past the matrix is its last one, whose results
    // are not stored.
    const _Float16* P = reinterpret_cast<const _Float16*>(g.p) + z * g.p_stride;
    const _Float16* Q = reinterpret_cast<const _Float16*>(g.q) + z * g.q_stride;
    const _Float16* pp[4];
    const _Float16* qq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (tid >> 3) + 32 * i;
      const int piece = (tid & 7) ^ ((r >> 1) & 7);
      const int pr = row0 + r < g.M ? row0 + r : g.M - 1;
      const int qr = col0 + r < g.N ? col0 + r : g.N - 1;
      pp[i] = P + static_cast<int64_t>(pr) * g.ldp + piece * 8;
      qq[i] = Q + static_cast<int64_t>(qr) * g.ldq + piece * 8;
    }

    f32x16 acc[2][2] = {};
    const int stages = g.K / kDepth;
    half8 rp[4], rq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rp[i] = *reinterpret_cast<const half8*>(pp[i]);
      rq[i] = *reinterpret_cast<const half8*>(qq[i]);
    }
    for (int k = 0; k < stages; ++k) {
      const int b = k & 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<half8*>(&sp[b][(tid + 256 * i) * 8]) = rp[i];
        *reinterpret_cast<half8*>(&sq[b][(tid + 256 * i) * 8]) = rq[i];
      }
      __syncthreads();
      if (k + 1 < stages) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          rp[i] = *reinterpret_cast<const half8*>(pp[i] + static_cast<int64_t>(k + 1) * kDepth);
          rq[i] = *reinterpret_cast<const half8*>(qq[i] + static_cast<int64_t>(k + 1) * kDepth);
        }
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        half8 fp[2], fq[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = wm + 32 * i + (lane & 31), c = 2 * kk + (lane >> 5);
          fp[i] = *reinterpret_cast<const half8*>(&sp[b][r * kDepth + ((c ^ ((r >> 1) & 7)) * 8)]);
          const int s = wn + 32 * i + (lane & 31);
          fq[i] = *reinterpret_cast<const half8*>(&sq[b][s * kDepth + ((c ^ ((s >> 1) & 7)) * 8)]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fp[i], fq[j], acc[i][j], 0, 0, 0);
      }
    }

    // Lane l holds column l & 31 and, in register r, row 8 (r / 4) +
    // 4 (l / 32) + r % 4 of each 32 x 32 result.
    const _Float16* HI = reinterpret_cast<const _Float16*>(g.hi) + z * g.c_stride;
    const _Float16* LO = reinterpret_cast<const _Float16*>(g.lo) + z * g.c_stride;
    _Float16* C = reinterpret_cast<_Float16*>(g.c) + z * g.c_stride;
    _Float16* CLO = reinterpret_cast<_Float16*>(g.c_lo) + z * g.c_stride;
    _Float16* T = reinterpret_cast<_Float16*>(g.turned) + z * g.turned_stride;
    const float* D = g.diag + z * g.diag_stride;
    float* DOUT = g.diag_out + z * g.diag_stride;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = col0 + wn + 32 * j + (lane & 31);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int row = row0 + wm + 32 * i + 8 * q + 4 * (lane >> 5);
          _Float16 h[4] = {};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float sum = acc[i][j][4 * q + e];
            const bool in = row + e < g.M && col < g.N;
            const int64_t at = static_cast<int64_t>(row + e) * g.ldc + col;
            if constexpr (WHAT == Product::kGram) {
              if (in) {
                const float v = sum * a.s.acc;
                if (row + e == col) DOUT[col] = v;
                else h[e] = static_cast<_Float16>(v);
              }
            } else if constexpr (WHAT == Product::kSquare) {
              if (in) {
                if (row + e == col) {
                  const float d = D[col];
                  DOUT[col] = (a.s.linear * d + (a.s.diag * (d * d) + a.s.acc * sum)) * a.s.out;
                } else {
                  const float d = a.s.diag * (D[row + e] + D[col]);
                  h[e] = static_cast<_Float16>((a.s.linear + d) * static_cast<float>(HI[at]) +
                                               a.s.acc * sum);
                }
              }
            } else if (in) {
              const float hi = static_cast<float>(HI[at]);
              const float d = a.s.diag * (g.tall ? D[col] : D[row + e]);
              float v;
              if constexpr (WHAT == Product::kUpdate)
                v = a.s.linear * (hi + static_cast<float>(LO[at]) * 0x1p-11f) + (d * hi + a.s.acc * sum);
              else
                v = (a.s.linear + d) * hi + a.s.acc * sum;
              if constexpr (WHAT == Product::kUpdate) {
                h[e] = static_cast<_Float16>(v);
                if (g.c_lo != nullptr)
                  CLO[at] = static_cast<_Float16>((v - static_cast<float>(h[e])) * 0x1p11f);
              } else if constexpr (WHAT == Product::kOut) {
                static_cast<uint16_t*>(g.out)[z * g.out_stride + (row + e) * g.out_ld + col] =
                    OUT == kBf16 ? bf16_bits(v) : fp16_bits(v);
              } else {
                const int64_t k = (static_cast<int64_t>(z) * g.M + row + e) * g.N + col;
                const float p = g.master[k] * a.s.decay - g.step * v;
                g.master[k] = p;
                if constexpr (OUT >= 0)
                  static_cast<uint16_t*>(g.out)[k] = OUT == kBf16 ? bf16_bits(p) : fp16_bits(p);
              }
            }
            if constexpr (SYM || WHAT == Product::kUpdate) {
              if (row + e < g.M && col < g.ldc) C[at] = h[e];
            }
          }
          // four consecutive elements of the turned result (row is a multiple
          // of 4 and the padded side of 64)
          if constexpr (SYM) {
            if (ti != tj && col < g.N && row < g.ldc)
              *reinterpret_cast<half4*>(&C[static_cast<int64_t>(col) * g.ldc + row]) =
                  half4{h[0], h[1], h[2], h[3]};
          } else if constexpr (WHAT == Product::kUpdate) {
            if (col < g.N && row < g.ld_turned)
              *reinterpret_cast<half4*>(&T[static_cast<int64_t>(col) * g.ld_turned + row]) =
                  half4{h[0], h[1], h[2], h[3]};
          }
        }
      }
    __syncthreads();  // the stages are free for the next tile
  }
}

template <Product WHAT, int OUT>
hipError_t launch_one(ProductArgs& a, int64_t total, hipStream_t stream, int64_t max_grid) {
  int64_t grid = total < kMaxWorkgroups ? total : kMaxWorkgroups;
  if (grid > max_grid) grid = max_grid;
  void* params[] = {&a};
  return hipLaunchKernel(reinterpret_cast<const void*>(&product_kernel<WHAT, OUT>),
                         dim3(static_cast<unsigned>(grid)), dim3(256), params, 0, stream);
}

}  // namespace

hipError_t launch_product(const ProductGroup* groups, int count, Product what, int out_type,
                          const ProductScales& s, const int32_t* skip, hipStream_t stream,
                          int64_t max_grid) {
  ProductArgs a = {};
  const bool symmetric = what == Product::kGram || what == Product::kSquare;
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    a.g[i] = groups[i];
    const int64_t tm = (groups[i].M + 127) / 128, tn = (groups[i].N + 127) / 128;
    const int64_t tiles = symmetric ? tm * (tm + 1) / 2 : tm * tn;
    a.tiles_n[i] = static_cast<int32_t>(tn);
    a.tiles[i] = static_cast<int32_t>(tiles);
    total += tiles * groups[i].count;
    a.tile_end[i] = total;
  }
  a.s = s;
  a.skip = skip;
  a.count = count;
  switch (what) {
    case Product::kGram: return launch_one<Product::kGram, 0>(a, total, stream, max_grid);
    case Product::kSquare: return launch_one<Product::kSquare, 0>(a, total, stream, max_grid);
    case Product::kUpdate: return launch_one<Product::kUpdate, 0>(a, total, stream, max_grid);
    case Product::kOut:
      return out_type == kFp16 ? launch_one<Product::kOut, kFp16>(a, total, stream, max_grid)
                               : launch_one<Product::kOut, kBf16>(a, total, stream, max_grid);
    default:
      return out_type == kFp16   ? launch_one<Product::kMuon, kFp16>(a, total, stream, max_grid)
             : out_type == kBf16 ? launch_one<Product::kMuon, kBf16>(a, total, stream, max_grid)
                                 : launch_one<Product::kMuon, -1>(a, total, stream, max_grid);
  }
}

}  // namespace la
