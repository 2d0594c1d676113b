// Internal interface between the C ABI of the orthogonalised update
// (la_muon_api.cpp) and its kernels (la_muon.hip, la_product.hip,
// la_narrow.hip). Not installed; callers use include/layeradam.h.
//
// The iteration, on a matrix U of rows x cols with m = min(rows, cols) and
// n = max(rows, cols): X_0 = U / max(||U||_F, eps), held so that its short
// side comes first, and for each step with coefficients (a, b, c)
//
//   A = X X^T            (m x m, symmetric)          product kernel, kGram
//   B = b A + c A A      (m x m, symmetric)          product kernel, kSquare
//   X <- a X + B X                                   product kernel, kUpdate,
//                                                    kOut or kMuon
//
// All three products are of the form P Q^T with both operands contiguous
// along the summed side, so X is kept twice: as the user's rows x cols
// ("straight") and as cols x rows ("turned").
//
// Number formats. An iterate is a binary16 number hi and a signed byte lo, the
// eight bits that follow: as binary32, bits(x) = bits(hi) + 32 lo, rounded to
// 19 significant bits. A power-of-two scale that the host derives from the
// coefficients keeps every value inside the format. The term a X takes both:
// it is what carries the small singular values through the steps, and a
// rounding of X to 11 bits would grow with them (measured on matrices of low
// rank: 4 % of the direction instead of 0.05 %). The products read hi alone. The last step needs no lo: no
// later one enlarges its rounding. A and B are binary16 but for their
// diagonals, which are the large entries where X is near orthogonal (and all
// there is where m = 1): those are binary32 and enter elementwise, as
// (D + F)^2 = D^2 + D F + F D + F^2. The sums are binary32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace la {

// Stacks of matrices per launch: their descriptions travel in the kernel
// arguments.
constexpr int kGroupsPerLaunch = 16;

// A launch has at most this many workgroups; the kernels stride past it.
constexpr int64_t kMaxWorkgroups = int64_t(1) << 22;

// Partial sums of squares per matrix, at most.
constexpr int kMaxPartials = 1024;

// Sides are padded with zeros to whole multiples of this many elements along
// the contiguous axis: the depth of one stage of the products.
constexpr int kDepth = 64;

// Element types of the directions (la_element_type).
constexpr int kBf16 = 0;
constexpr int kFp16 = 1;
constexpr int kFp32 = 2;

typedef uint16_t half_bits;

// ---- directions and their norms ------------------------------------------------

// One stack of the momentum pass: contiguous rows x cols matrices.
struct MomentumGroup {
  float* momentum;
  float* direction;          // g + mu B, or null without the Nesterov form
  const uint16_t* g[8];
  double* partial;           // count x partials sums of squares
  int64_t numel;             // of one matrix
  int64_t direction_stride;  // between matrices of `direction`
  int64_t chunk;             // elements of one workgroup, a multiple of 2048
  int32_t partials;          // ceil(numel / chunk)
  int32_t count;
  int32_t vectors;           // 1: every 8 elements of a chunk are 16-byte aligned
};

hipError_t launch_momentum(const MomentumGroup* groups, int count, int replicas, bool fp16,
                           float mu, float unscale, int32_t* flag, const int32_t* skip,
                           hipStream_t stream, int64_t max_grid);

// One stack of directions: rows x cols matrices, rows row_stride elements
// apart, matrices matrix_stride apart.
struct DirectionGroup {
  const void* in;
  int64_t row_stride, matrix_stride;
  double* partial;         // count x partials
  half_bits* straight;     // rows x ld_straight: hi
  int8_t* straight_lo;     // rows x ld_straight: lo
  half_bits* turned;       // cols x ld_turned: hi
  int32_t rows, cols, count;
  int32_t ld_straight, ld_turned;
  int32_t partials;        // sums of squares per matrix
  int32_t rows_per_partial;
  int32_t vectors;         // 1: every 8 elements of a row are 16-byte aligned
};

// Sums of squares of the directions (orthogonalize only: the momentum pass
// forms its own).
hipError_t launch_square_sums(const DirectionGroup* groups, int count, int type,
                              hipStream_t stream, int64_t max_grid);

// X_0 scaled by `scale`, in both layouts.
hipError_t launch_normalise(const DirectionGroup* groups, int count, int type, float scale,
                            double eps, const int32_t* skip, hipStream_t stream,
                            int64_t max_grid);

// ---- products ----------------------------------------------------------------------

enum class Product { kGram, kSquare, kUpdate, kOut, kMuon };

// One stack of products C = P Q^T (M x N over K) with their epilogue.
struct ProductGroup {
  const half_bits* p;      // M x ldp
  const half_bits* q;      // N x ldq
  const half_bits* hi;     // linear term: M x ldc (kSquare: A; kUpdate...: X straight)
  const int8_t* lo;        // kUpdate
  const float* diag;       // m padded: diagonal of A (kSquare) or of B (kUpdate, kOut, kMuon)
  float* diag_out;         // m padded: diagonal of A (kGram) or of B (kSquare)
  half_bits* c;            // result, M x ldc (kOut: none)
  int8_t* c_lo;            // kUpdate, or null where nothing reads it
  half_bits* turned;       // kUpdate: N x ld_turned
  void* out;               // kOut: result; kMuon: the compute copy or null
  float* master;           // kMuon
  int64_t p_stride, q_stride, c_stride, turned_stride, diag_stride;
  int64_t out_stride, out_ld;  // kOut
  int32_t M, N, K;         // K: a multiple of kDepth, zero-padded
  int32_t ldp, ldq, ldc, ld_turned;
  int32_t count;
  int32_t tall;            // diag runs along N rather than M
  int32_t vectors;         // kOut, kMuon: every 8 elements of a row are 16-byte aligned
  float step;              // kMuon: lr times the stack's scale
};

// kGram:    A' = acc P Q^T, its diagonal apart in binary32
// kSquare:  B' = (linear + diag (d_i + d_j)) A'_ij + acc P Q^T off the diagonal
//           and (linear d_i + (diag d_i^2 + acc P Q^T)) out on it
// kUpdate:  linear (hi + lo) + (diag d_i hi + acc P Q^T)
// kOut, kMuon: (linear + diag d_i) hi + acc P Q^T
// with A' and B' the stored ones: scaled, with zeros on the diagonal.
struct ProductScales {
  float acc, linear, diag, out;
  float decay;  // kMuon: 1 - lr * weight_decay
};

// out_type: kOut kBf16 or kFp16; kMuon: kBf16, kFp16, or -1 for no copy.
hipError_t launch_product(const ProductGroup* groups, int count, Product what, int out_type,
                          const ProductScales& s, const int32_t* skip, hipStream_t stream,
                          int64_t max_grid);

// ---- narrow matrices ---------------------------------------------------------------

// Matrices whose short side is at most this take the iteration on S = X X^T.
constexpr int kNarrow = 128;

// Up to this side the iteration on S is binary64.
constexpr int kTiny = 16;

// Steps of a polynomial at most (LA_MAX_POLYNOMIAL_STEPS).
constexpr int kMaxSteps = 16;

// One stack of narrow matrices.
struct NarrowGroup {
  const void* in;           // directions, rows x cols
  double* partial;          // count x partials sums of squares, or null: formed here
  float* gram;              // count x splits partial sums of S, in the accumulators' order
  half_bits* q;             // count x (hi, lo) of the polynomial's factor
  double* sums;             // side kTiny: count x splits partial sums of U U^T
  void* out;                // result, or the compute copy or null
  float* master;            // the Muon step; null: the result goes to out
  int64_t row_stride, matrix_stride, out_row_stride, out_matrix_stride;
  int32_t rows, cols, count;
  int32_t partials;
  int32_t splits, chunk;    // columns of one part of the sum, a multiple of 64
  float step;               // lr times the stack's scale
};

struct NarrowStep {
  float a, b, c;
  int32_t s, p, t, q;  // exponents of the scales of S, P = a + b S + c S S, P S and Q = P ... P
};

// kWhole (sides kTiny and 64): all of it, one workgroup per matrix; kSum, kFactor, kApply:
// its three parts, with as many workgroups as there is work for (side kTiny: kApply
// forms the factor too).
enum class NarrowPart { kWhole, kSum, kFactor, kApply };

struct NarrowPlan {
  NarrowStep step[kMaxSteps];
  int32_t steps;
  int32_t x;        // exponent of the scale of X
  double eps;
  float decay;
  int32_t out_type; // kBf16, kFp16, -1: none
};

// side: kTiny, 64 or 128, at least every group's short side.
hipError_t launch_narrow(const NarrowGroup* groups, int count, int side, int type,
                         NarrowPart part, const NarrowPlan& plan, const int32_t* skip,
                         hipStream_t stream, int64_t max_grid);

// x as it is in binary32, before it is split into hi and what follows. Without
// it the compiler may form hi from x's last operation in one rounding, once for
// the store and not for the difference x - hi: where the two roundings to
// binary16 part, one element in some thousands, what follows is that of
// another hi, and X is off by 2^-11 there.
__device__ __forceinline__ float settled(float x) {
  asm("" : "+v"(x));
  return x;
}

// The byte that follows hi = binary16(x). Where hi is below the format's normal
// range the byte saturates: the error stays under half of hi's spacing there,
// 2^-25 of the scaled value.
__device__ __forceinline__ int low_byte(float x, _Float16 hi) {
  const int d = __float_as_int(x) - __float_as_int(static_cast<float>(hi)) + 16;
  const int q = d >> 5;
  return q < -128 ? -128 : q > 127 ? 127 : q;
}

__device__ __forceinline__ float with_low_byte(float hi, int lo) {
  return __int_as_float(__float_as_int(hi) + lo * 32);
}

}  // namespace la
