// la_muon_api.cpp -- the C ABI of the orthogonalised update and the Muon step
// (declared in include/layeradam.h).
//
// Host side only: checks every argument before anything is enqueued, derives
// the scales of the number formats from the coefficients, lays the
// workspace out and enqueues the stages for all matrices of the call, up to
// kGroupsPerLaunch stacks to a launch.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <vector>

#include "la_error.h"
#include "la_muon.h"
#include "layeradam.h"

namespace {

using la::fail;
using la::ok;

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool finite_nonneg(double x) { return std::isfinite(x) && x >= 0.0; }
int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// ---- the polynomial ----------------------------------------------------------------

constexpr double kDefault[3] = {3.4445, -4.7750, 2.0315};
constexpr int kDefaultSteps = 5;
constexpr double kDefaultEps = 1e-7;

struct Step {
  double a, b, c;
  int x, gram, poly;  // exponents of the scales of X, A and B
  // narrow form: of P = a + b S + c S S, of P S and of Q, the product of the P
  int factor, turn, whole;
};

struct Polynomial {
  Step step[LA_MAX_POLYNOMIAL_STEPS];
  int steps;
  double eps;
  double growth;  // bound of Q after the last step
};

// Smallest e with x <= 2^e.
int exponent(double x) {
  int e;
  const double f = std::frexp(x, &e);  // x = f 2^e, 1/2 <= f < 1
  return f == 0.5 ? e - 1 : e;
}

// Bounds of what the iteration can hold, for singular values in [0, s]: the
// entries of X are at most s, those of A = X X^T at most s^2, those of the
// symmetric b A + c A^2 at most the largest |b l + c l^2| over l in [0, s^2].
// Each is scaled to stay below 2^14, a quarter of the format's range, which
// leaves room for the rounding of earlier steps.
la_status derive_polynomial(const la_polynomial* p, Polynomial* out) {
  const int steps = p == nullptr ? kDefaultSteps : p->num_steps;
  if (steps < 1 || steps > LA_MAX_POLYNOMIAL_STEPS)
    return fail(LA_ERR_INVALID_ARGUMENT, "num_steps = %d, need 1..%d", steps,
                LA_MAX_POLYNOMIAL_STEPS);
  if (p != nullptr && p->coefficients == nullptr)
    return fail(LA_ERR_INVALID_ARGUMENT, "coefficients is NULL");
  out->steps = steps;
  out->eps = p == nullptr ? kDefaultEps : p->eps;
  if (!finite_nonneg(out->eps)) return fail(LA_ERR_INVALID_ARGUMENT, "eps = %g", out->eps);
  double s = 1.0;
  out->growth = 1.0;
  for (int k = 0; k < steps; ++k) {
    const double* t = p == nullptr ? kDefault : p->coefficients + 3 * k;
    const double a = t[0], b = t[1], c = t[2];
    if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c))
      return fail(LA_ERR_INVALID_ARGUMENT, "coefficients of step %d: (%g, %g, %g)", k, a, b, c);
    auto value = [&](double q) { return std::fabs((a + (b + c * q) * q) * std::sqrt(q)); };
    auto inner = [&](double q) { return std::fabs((b + c * q) * q); };
    auto whole = [&](double q) { return std::fabs(a + (b + c * q) * q); };
    const double end = s * s;
    double next = value(end), poly = inner(end), factor = std::max(std::fabs(a), whole(end));
    if (c != 0.0) {
      const double q = -b / (2.0 * c);
      if (q > 0.0 && q < end) {
        poly = std::max(poly, inner(q));
        factor = std::max(factor, whole(q));
      }
    }
    // a + 3 b q + 5 c q^2 = 0 at the inner extremes. Both roots come from the sum
    // that does not cancel: with a c far below b the other one would be lost.
    auto extreme = [&](double q) {
      if (q > 0.0 && q < end) next = std::max(next, value(q));
    };
    const double d = 9.0 * b * b - 20.0 * a * c;
    if (d >= 0.0) {
      const double t = -0.5 * (3.0 * b + std::copysign(std::sqrt(d), b));
      if (c != 0.0) extreme(t / (5.0 * c));
      if (t != 0.0) extreme(a / t);
    }
    if (!(next <= 0x1p20) || !(next >= 0x1p-20) || !(poly <= 0x1p40))
      return fail(LA_ERR_INVALID_ARGUMENT,
                  "step %d: the polynomial reaches %g (its inner part %g) on [0, %g]", k, next,
                  poly, s);
    out->growth *= factor * 1.01;
    out->step[k] = {a,
                    b,
                    c,
                    14 - exponent(s),
                    14 - exponent(end),
                    14 - exponent(std::max(poly, 0x1p-20)),
                    14 - exponent(factor * 1.01),
                    14 - exponent(factor * end * 1.01),
                    14 - exponent(out->growth)};
    s = next * 1.01;
  }
  return LA_OK;
}

// ---- the plan ------------------------------------------------------------------------

// One stack of the call, and where its parts lie in the workspace (bytes from
// its start).
struct Stack {
  int64_t rows, cols, count;
  int64_t ld_straight, ld_turned;
  int64_t numel_straight, numel_turned;  // of one matrix, padded
  int64_t m, n, ldm;
  int64_t numel_direction;               // FP32 direction of one matrix, padded
  int64_t straight[2], straight_lo[2], turned[2], gram, poly, gram_diag, poly_diag, partial,
      direction;
  int32_t partials;
  int64_t chunk, rows_per_partial;
  int index;  // in the caller's list
  // the narrow form
  bool narrow, whole;  // whole: one workgroup per matrix does everything
  int side;
  int64_t splits, columns;  // parts of the long side, and columns in each
  int64_t sums, factors;
};

// A factor Q that reaches past this leaves its 22 bits too coarse beside the
// singular values near 1, whose factor is about 1 (the default polynomial
// reaches 490): such polynomials take the step-by-step form everywhere.
constexpr double kMostGrowth = 512.0;

// Up to this many columns one workgroup does a narrow matrix alone, from its
// norm to its result, and so it does where there are matrices enough to fill
// the GPU. Beyond, the sum over the columns and the last product are cut into
// about kParts parts.
constexpr int64_t kWholeColumns = 512;
constexpr int64_t kWholeCount = 512;
constexpr int64_t kParts = 512;
constexpr int64_t kMostParts = 32;  // of one matrix: one workgroup adds them up

// Beside wide stacks, whose launches it can share, a small narrow stack does
// not get its own: with sides up to kWholeColumns and up to this many elements as
// the step-by-step form pads them. Shared and in launches of its own, us: 8 of 64 x
// 256 beside one of 256 x 256 116 and 180, beside 8 of 2048 x 2048 2103 and 2117; on
// the other side of the borders, 4 of 64 x 4096 beside one of 256 x 256 218 and 181
// (a longer side makes the few tiles of X X^T long; at 1024 it is still 134 and
// 177), 128 of 64 x 256 beside one of
// 4096 x 2560 878 and 823. Sides up to kTiny do not share: the step-by-step form's
// roundings do not average there (4 of 16 x 300 beside one of 300 x 300: 123 and
// 139).
constexpr int64_t kSharedElements = int64_t(1) << 20;

void choose_form(Stack& s, const Polynomial& p, bool beside_wide) {
  s.m = std::min(s.rows, s.cols);
  s.n = std::max(s.rows, s.cols);
  const bool shares = beside_wide && s.m > la::kTiny && s.n <= kWholeColumns &&
                      s.count * s.n * round_up(s.m, la::kDepth) <= kSharedElements;
  s.narrow = s.m <= la::kNarrow && p.growth <= kMostGrowth && !shares;
  if (!s.narrow) return;
  s.side = s.m <= la::kTiny ? la::kTiny : s.m <= 64 ? 64 : 128;
  // 128 x 128 operands leave the whole form no registers
  s.whole = s.side <= 64 && (s.n <= kWholeColumns || s.count >= kWholeCount);
  s.splits = std::min({(kParts + s.count - 1) / s.count, (s.n + 255) / 256, kMostParts});
  s.columns = round_up((s.n + s.splits - 1) / s.splits, 64);
  s.splits = (s.n + s.columns - 1) / s.columns;
}

la_status check_sides(int i, int64_t rows, int64_t cols, int64_t count) {
  if (rows < 0 || cols < 0 || count < 0 || rows > LA_MAX_SIDE || cols > LA_MAX_SIDE ||
      count > LA_MAX_SIDE)
    return fail(LA_ERR_INVALID_ARGUMENT,
                "tensor %d: %lld matrices of %lld x %lld, need 0..%d of each", i,
                static_cast<long long>(count), static_cast<long long>(rows),
                static_cast<long long>(cols), LA_MAX_SIDE);
  if (static_cast<double>(rows) * static_cast<double>(cols) * static_cast<double>(count) > 0x1p44)
    return fail(LA_ERR_INVALID_ARGUMENT, "tensor %d: %lld x %lld x %lld elements", i,
                static_cast<long long>(count), static_cast<long long>(rows),
                static_cast<long long>(cols));
  return LA_OK;
}

// Lays the stacks out; returns the bytes of the whole. `direction`: an FP32
// direction is kept (Muon with the Nesterov form). It shares the second
// iterate's place, which is first written after the direction's last use.
int64_t lay_out(std::vector<Stack>& stacks, const Polynomial& p, bool direction, bool contiguous) {
  const int steps = p.steps;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, LA_WORKSPACE_ALIGNMENT);
    return here;
  };
  bool wide = false;
  for (const Stack& s : stacks) wide |= std::min(s.rows, s.cols) > la::kNarrow;
  for (Stack& s : stacks) {
    choose_form(s, p, wide);
    s.ld_straight = round_up(s.cols, la::kDepth);
    s.ld_turned = round_up(s.rows, la::kDepth);
    s.numel_straight = s.rows * s.ld_straight;
    s.numel_turned = s.cols * s.ld_turned;
    s.ldm = round_up(s.m, la::kDepth);
    const int64_t numel = s.rows * s.cols;
    s.numel_direction = round_up(numel, 8);
    if (contiguous) {  // the momentum pass cuts a matrix by elements
      s.chunk = round_up(std::max<int64_t>(4096, (numel + la::kMaxPartials - 1) / la::kMaxPartials),
                         2048);
      s.partials = static_cast<int32_t>((numel + s.chunk - 1) / s.chunk);
      s.rows_per_partial = 0;
    } else {  // the sums of squares by rows
      s.chunk = 0;
      s.rows_per_partial = std::max<int64_t>(
          (s.rows + la::kMaxPartials - 1) / la::kMaxPartials,
          std::min<int64_t>(s.rows, (4096 + s.cols - 1) / s.cols));
      s.partials =
          static_cast<int32_t>((s.rows + s.rows_per_partial - 1) / s.rows_per_partial);
    }
    const int64_t k = s.count;
    if (s.narrow) {
      if (direction) s.direction = take(4 * k * s.numel_direction);
      if (!s.whole) {
        const int64_t square = static_cast<int64_t>(s.side) * s.side;
        s.sums = take((s.side == la::kTiny ? 8 : 4) * k * s.splits * square);
        if (s.side != la::kTiny) s.factors = take(2 * 2 * k * square);
      }
      s.partial = take(8 * k * s.partials);
      continue;
    }
    s.straight[0] = take(2 * k * s.numel_straight);
    s.straight_lo[0] = take(k * s.numel_straight);
    s.turned[0] = take(2 * k * s.numel_turned);
    const int64_t second = at;
    if (steps > 1) {
      s.straight[1] = take(2 * k * s.numel_straight);
      if (steps > 2) s.straight_lo[1] = take(k * s.numel_straight);
      s.turned[1] = take(2 * k * s.numel_turned);
    }
    s.direction = second;
    if (direction)
      at = std::max(at, second + round_up(4 * k * s.numel_direction, LA_WORKSPACE_ALIGNMENT));
    s.gram = take(2 * k * s.m * s.ldm);
    s.poly = take(2 * k * s.m * s.ldm);
    s.gram_diag = take(4 * k * s.ldm);
    s.poly_diag = take(4 * k * s.ldm);
    s.partial = take(8 * k * s.partials);
  }
  return at;
}

template <typename T>
T* place(void* workspace, int64_t at) {
  return reinterpret_cast<T*>(static_cast<char*>(workspace) + at);
}

// ---- the stages ----------------------------------------------------------------------

// The products of all steps. `last` fills in the output of the last one.
template <typename Last>
la_status enqueue_products(const std::vector<Stack>& stacks, const Polynomial& p,
                           la::Product last_product, int out_type, float decay, Last last,
                           void* ws, const int32_t* skip, hipStream_t stream) {
  auto launch = [&](la::Product what, const la::ProductScales& scales, int k) -> hipError_t {
    for (size_t first = 0; first < stacks.size(); first += la::kGroupsPerLaunch) {
      la::ProductGroup g[la::kGroupsPerLaunch] = {};
      const int count =
          static_cast<int>(std::min<size_t>(la::kGroupsPerLaunch, stacks.size() - first));
      for (int i = 0; i < count; ++i) {
        const Stack& s = stacks[first + i];
        la::ProductGroup& x = g[i];
        const int now = k & 1, then = now ^ 1;
        const bool tall = s.rows > s.cols;
        const uint16_t* straight = place<uint16_t>(ws, s.straight[now]);
        const uint16_t* turned = place<uint16_t>(ws, s.turned[now]);
        uint16_t* gram = place<uint16_t>(ws, s.gram);
        uint16_t* poly = place<uint16_t>(ws, s.poly);
        x.diag = place<float>(
            ws, what == la::Product::kSquare ? s.gram_diag : s.poly_diag);
        x.diag_out = place<float>(
            ws, what == la::Product::kGram ? s.gram_diag : s.poly_diag);
        x.diag_stride = s.ldm;
        x.count = static_cast<int32_t>(s.count);
        x.tall = tall;
        if (what == la::Product::kGram || what == la::Product::kSquare) {
          const bool first_of = what == la::Product::kGram;
          x.p = x.q = first_of ? (tall ? turned : straight) : gram;
          x.p_stride = x.q_stride =
              first_of ? (tall ? s.numel_turned : s.numel_straight) : s.m * s.ldm;
          x.ldp = x.ldq = static_cast<int32_t>(first_of ? (tall ? s.ld_turned : s.ld_straight)
                                                        : s.ldm);
          x.K = x.ldp;
          x.M = x.N = static_cast<int32_t>(s.m);
          x.hi = gram;
          x.c = first_of ? gram : poly;
          x.ldc = static_cast<int32_t>(s.ldm);
          x.c_stride = s.m * s.ldm;
        } else {
          // wide: B X = B (X^T)^T; tall: the same on the transpose, X^T B = X^T B^T
          x.p = tall ? straight : poly;
          x.q = tall ? poly : turned;
          x.p_stride = tall ? s.numel_straight : s.m * s.ldm;
          x.q_stride = tall ? s.m * s.ldm : s.numel_turned;
          x.ldp = static_cast<int32_t>(tall ? s.ld_straight : s.ldm);
          x.ldq = static_cast<int32_t>(tall ? s.ldm : s.ld_turned);
          x.K = static_cast<int32_t>(s.ldm);
          x.M = static_cast<int32_t>(s.rows);
          x.N = static_cast<int32_t>(s.cols);
          x.hi = straight;
          x.lo = place<int8_t>(ws, s.straight_lo[now]);
          x.ldc = static_cast<int32_t>(s.ld_straight);
          x.c_stride = s.numel_straight;
          if (what == la::Product::kUpdate) {
            x.c = place<uint16_t>(ws, s.straight[then]);
            // the last step reads hi alone
            x.c_lo = k + 2 < p.steps ? place<int8_t>(ws, s.straight_lo[then]) : nullptr;
            x.turned = place<uint16_t>(ws, s.turned[then]);
            x.ld_turned = static_cast<int32_t>(s.ld_turned);
            x.turned_stride = s.numel_turned;
          } else {
            last(s, x);
          }
        }
      }
      const hipError_t e =
          la::launch_product(g, count, what, out_type, scales, skip, stream, la::max_grid());
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  };
  for (int k = 0; k < p.steps; ++k) {
    const Step& t = p.step[k];
    const bool end = k + 1 == p.steps;
    const int next = end ? 0 : p.step[k + 1].x;
    auto power = [](double f, int e) { return static_cast<float>(std::ldexp(f, e)); };
    const la::ProductScales gram = {power(1.0, t.gram - 2 * t.x), 0.0f, 0.0f, 0.0f, 0.0f};
    // stored A' = A 2^gram, B' = B 2^poly: B' = (b A' + c A' A' 2^-gram) 2^(poly - gram)
    const la::ProductScales square = {power(t.c, t.poly - 2 * t.gram), power(t.b, t.poly - t.gram),
                                      power(t.c, t.poly - 2 * t.gram), power(1.0, -t.poly), 0.0f};
    const la::ProductScales update = {power(1.0, next - t.poly - t.x), power(t.a, next - t.x),
                                      power(1.0, next - t.x), 0.0f, decay};
    hipError_t e = launch(la::Product::kGram, gram, k);
    if (e == hipSuccess) e = launch(la::Product::kSquare, square, k);
    if (e == hipSuccess) e = launch(end ? last_product : la::Product::kUpdate, update, k);
    if (e != hipSuccess)
      return fail(LA_ERR_HIP, "kernel launch of step %d failed: %s", k, hipGetErrorString(e));
  }
  return ok();
}

// The narrow stacks, from their directions to the results. `fill` gives a
// group its source and its output.
template <typename Fill>
la_status enqueue_narrow(const std::vector<Stack>& stacks, const Polynomial& p, int type,
                         int out_type, float decay, Fill fill, void* ws, const int32_t* skip,
                         hipStream_t stream) {
  la::NarrowPlan plan = {};
  plan.steps = p.steps;
  plan.x = p.step[0].x;
  plan.eps = p.eps;
  plan.decay = decay;
  plan.out_type = out_type;
  for (int k = 0; k < p.steps; ++k) {
    const Step& t = p.step[k];
    plan.step[k] = {static_cast<float>(t.a), static_cast<float>(t.b), static_cast<float>(t.c),
                    t.gram, t.factor, t.turn, t.whole};
  }
  for (const int side : {la::kTiny, 64, 128})
    for (const bool whole : {true, false}) {
      la::NarrowGroup g[la::kGroupsPerLaunch];
      int count = 0;
      auto flush = [&]() -> hipError_t {
        hipError_t e = hipSuccess;
        auto launch = [&](la::NarrowPart part) {
          if (e == hipSuccess)
            e = la::launch_narrow(g, count, side, type, part, plan, skip, stream, la::max_grid());
        };
        if (count > 0) {
          if (whole) {
            launch(la::NarrowPart::kWhole);
          } else {
            launch(la::NarrowPart::kSum);
            if (side != la::kTiny) launch(la::NarrowPart::kFactor);
            launch(la::NarrowPart::kApply);
          }
        }
        count = 0;
        return e;
      };
      hipError_t e = hipSuccess;
      for (const Stack& s : stacks) {
        if (!s.narrow || s.side != side || s.whole != whole) continue;
        la::NarrowGroup& x = g[count++] = {};
        x.rows = static_cast<int32_t>(s.rows);
        x.cols = static_cast<int32_t>(s.cols);
        x.count = static_cast<int32_t>(s.count);
        x.partial = place<double>(ws, s.partial);
        x.partials = s.partials;
        x.gram = place<float>(ws, s.sums);
        x.sums = place<double>(ws, s.sums);
        x.q = place<uint16_t>(ws, s.factors);
        x.splits = static_cast<int32_t>(s.splits);
        x.chunk = static_cast<int32_t>(s.columns);
        fill(s, x);
        if (count == la::kGroupsPerLaunch && (e = flush()) != hipSuccess) break;
      }
      if (e == hipSuccess) e = flush();
      if (e != hipSuccess)
        return fail(LA_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    }
  return ok();
}

// The direction's fields that a stack gives by itself.
la::DirectionGroup direction_group(const Stack& s, void* ws) {
  la::DirectionGroup d = {};
  d.partial = place<double>(ws, s.partial);
  d.straight = place<uint16_t>(ws, s.straight[0]);
  d.straight_lo = place<int8_t>(ws, s.straight_lo[0]);
  d.turned = place<uint16_t>(ws, s.turned[0]);
  d.rows = static_cast<int32_t>(s.rows);
  d.cols = static_cast<int32_t>(s.cols);
  d.count = static_cast<int32_t>(s.count);
  d.ld_straight = static_cast<int32_t>(s.ld_straight);
  d.ld_turned = static_cast<int32_t>(s.ld_turned);
  d.partials = s.partials;
  d.rows_per_partial = static_cast<int32_t>(s.rows_per_partial);
  return d;
}

la_status check_workspace(const void* ws, int64_t given, int64_t needed) {
  if (needed == 0) return LA_OK;
  if (ws == nullptr) return fail(LA_ERR_INVALID_ARGUMENT, "workspace is NULL");
  if (!aligned(ws, LA_WORKSPACE_ALIGNMENT))
    return fail(LA_ERR_MISALIGNED, "workspace is not %d-byte aligned", LA_WORKSPACE_ALIGNMENT);
  if (given < needed)
    return fail(LA_ERR_INVALID_ARGUMENT, "workspace_bytes = %lld, need %lld",
                static_cast<long long>(given), static_cast<long long>(needed));
  return LA_OK;
}

// ---- aliasing --------------------------------------------------------------------------

struct Range {
  uintptr_t begin, end;  // [begin, end)
  const char* what;
  int tensor;
};

Range range(const void* p, int64_t bytes, const char* what, int tensor) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, b + static_cast<uintptr_t>(bytes), what, tensor};
}

// Written ranges must be pairwise disjoint and disjoint from every range that
// is only read.
la_status check_disjoint(std::vector<Range>& written, const std::vector<Range>& read) {
  auto meet = [](const Range& a, const Range& b) { return a.begin < b.end && b.begin < a.end; };
  auto refuse = [](const Range& a, const Range& b) {
    return fail(LA_ERR_ALIASING, "%s of tensor %d overlaps %s of tensor %d", a.what, a.tensor,
                b.what, b.tensor);
  };
  std::sort(written.begin(), written.end(),
            [](const Range& a, const Range& b) { return a.begin < b.begin; });
  for (size_t k = 1; k < written.size(); ++k)
    if (meet(written[k - 1], written[k])) return refuse(written[k - 1], written[k]);
  for (const Range& r : read) {
    // the first written range that ends after r begins: the ranges are
    // disjoint and sorted, so their ends are sorted too
    auto it = std::lower_bound(written.begin(), written.end(), r.begin,
                               [](const Range& w, uintptr_t x) { return w.end <= x; });
    if (it != written.end() && meet(*it, r)) return refuse(r, *it);
  }
  return LA_OK;
}

// ---- orthogonalize -----------------------------------------------------------------

int64_t type_bytes(int type) { return type == LA_TYPE_FP32 ? 4 : 2; }

la_status plan_matrices(const la_matrices_desc* d, const la_polynomial* polynomial,
                        Polynomial* p, std::vector<Stack>* stacks, int64_t* bytes) {
  if (d == nullptr) return fail(LA_ERR_INVALID_ARGUMENT, "matrices descriptor is NULL");
  if (d->num_matrices < 0 || d->num_matrices > LA_MAX_TENSORS)
    return fail(LA_ERR_INVALID_ARGUMENT, "num_matrices = %d, need 0..%d", d->num_matrices,
                LA_MAX_TENSORS);
  if (d->num_matrices > 0 && d->matrices == nullptr)
    return fail(LA_ERR_INVALID_ARGUMENT, "matrices is NULL with num_matrices = %d",
                d->num_matrices);
  if (d->in_type != LA_TYPE_BF16 && d->in_type != LA_TYPE_FP16 && d->in_type != LA_TYPE_FP32)
    return fail(LA_ERR_UNSUPPORTED, "in_type = %d, need a la_element_type", d->in_type);
  if (d->out_type != LA_TYPE_BF16 && d->out_type != LA_TYPE_FP16)
    return fail(LA_ERR_UNSUPPORTED, "out_type = %d, need LA_TYPE_BF16 or LA_TYPE_FP16",
                d->out_type);
  la_status st = derive_polynomial(polynomial, p);
  if (st != LA_OK) return st;
  for (int i = 0; i < d->num_matrices; ++i) {
    const la_matrix_desc& x = d->matrices[i];
    if ((st = check_sides(i, x.rows, x.cols, x.count)) != LA_OK) return st;
    if (x.rows == 0 || x.cols == 0 || x.count == 0) continue;
    auto strides = [&](int64_t row, int64_t matrix, const char* what) -> la_status {
      constexpr int64_t kMost = int64_t(1) << 40;  // keeps every offset far from 64 bits
      if (x.rows == 1) row = x.cols;
      if (x.count == 1) matrix = x.rows > 1 ? (x.rows - 1) * std::min(row, kMost) + x.cols : x.cols;
      const bool fits = row >= 0 && row <= kMost && matrix >= 0 &&
                        (x.count == 1 || matrix <= kMost);
      const bool stacked = fits && row >= x.cols && matrix >= (x.rows - 1) * row + x.cols;
      const bool beside = fits && matrix >= x.cols && row >= (x.count - 1) * matrix + x.cols;
      if (!stacked && !beside)
        return fail(LA_ERR_INVALID_ARGUMENT,
                    "tensor %d: strides of %s (row %lld, matrix %lld) make %lld matrices of "
                    "%lld x %lld overlap",
                    i, what, static_cast<long long>(row), static_cast<long long>(matrix),
                    static_cast<long long>(x.count), static_cast<long long>(x.rows),
                    static_cast<long long>(x.cols));
      return LA_OK;
    };
    if ((st = strides(x.in_row_stride, x.in_matrix_stride, "in")) != LA_OK) return st;
    if ((st = strides(x.out_row_stride, x.out_matrix_stride, "out")) != LA_OK) return st;
    Stack s = {};
    s.rows = x.rows;
    s.cols = x.cols;
    s.count = x.count;
    s.index = i;
    stacks->push_back(s);
  }
  *bytes = lay_out(*stacks, *p, false, false);
  return LA_OK;
}

la_status orthogonalize(const la_matrices_desc* d, const la_polynomial* polynomial, void* ws,
                        int64_t ws_bytes, void* hip_stream) {
  Polynomial p;
  std::vector<Stack> stacks;
  int64_t bytes = 0;
  la_status st = plan_matrices(d, polynomial, &p, &stacks, &bytes);
  if (st != LA_OK) return st;
  if (stacks.empty()) return ok();
  const int64_t in_bytes = type_bytes(d->in_type), out_bytes = 2;
  std::vector<Range> written, read;
  for (const Stack& s : stacks) {
    const la_matrix_desc& x = d->matrices[s.index];
    if (x.in == nullptr || x.out == nullptr)
      return fail(LA_ERR_INVALID_ARGUMENT, "tensor %d: %s is NULL", s.index,
                  x.in == nullptr ? "in" : "out");
    if (!aligned(x.in, in_bytes) || !aligned(x.out, out_bytes))
      return fail(LA_ERR_MISALIGNED, "tensor %d: %s is not aligned to its element", s.index,
                  aligned(x.in, in_bytes) ? "out" : "in");
    auto extent = [&](int64_t row, int64_t matrix) {
      return (s.rows > 1 ? (s.rows - 1) * row : 0) + (s.count > 1 ? (s.count - 1) * matrix : 0) +
             s.cols;
    };
    const Range in = range(x.in, in_bytes * extent(x.in_row_stride, x.in_matrix_stride), "in",
                           s.index);
    const Range out = range(x.out, out_bytes * extent(x.out_row_stride, x.out_matrix_stride),
                            "out", s.index);
    const bool in_place = x.in == x.out && d->in_type == d->out_type &&
                          (s.rows == 1 || x.in_row_stride == x.out_row_stride) &&
                          (s.count == 1 || x.in_matrix_stride == x.out_matrix_stride);
    written.push_back(out);
    if (!in_place) read.push_back(in);
  }
  if ((st = check_workspace(ws, ws_bytes, bytes)) != LA_OK) return st;
  written.push_back(range(ws, bytes, "the workspace", -1));
  if ((st = check_disjoint(written, read)) != LA_OK) return st;

  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  // the whole narrow form sums its squares itself, and so does that of side kTiny
  std::vector<Stack> wide, summed;
  for (const Stack& x : stacks) {
    if (!x.narrow) wide.push_back(x);
    if (!x.narrow || !(x.whole || x.side == la::kTiny)) summed.push_back(x);
  }
  auto directions = [&](const std::vector<Stack>& list, auto launch) -> la_status {
    for (size_t first = 0; first < list.size(); first += la::kGroupsPerLaunch) {
      la::DirectionGroup g[la::kGroupsPerLaunch];
      const int count =
          static_cast<int>(std::min<size_t>(la::kGroupsPerLaunch, list.size() - first));
      for (int i = 0; i < count; ++i) {
        const Stack& s = list[first + i];
        g[i] = direction_group(s, ws);
        g[i].in = d->matrices[s.index].in;
        g[i].row_stride = d->matrices[s.index].in_row_stride;
        g[i].matrix_stride = d->matrices[s.index].in_matrix_stride;
        g[i].vectors = aligned(g[i].in, 16) && s.cols % 8 == 0 &&
                       (s.rows == 1 || g[i].row_stride % 8 == 0) &&
                       (s.count == 1 || g[i].matrix_stride % 8 == 0);
      }
      const hipError_t e = launch(g, count);
      if (e != hipSuccess)
        return fail(LA_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
    }
    return LA_OK;
  };
  st = directions(summed, [&](const la::DirectionGroup* g, int count) {
    return la::launch_square_sums(g, count, d->in_type, stream, la::max_grid());
  });
  if (st != LA_OK) return st;
  st = enqueue_narrow(
      stacks, p, d->in_type, d->out_type, 0.0f,
      [&](const Stack& s, la::NarrowGroup& x) {
        const la_matrix_desc& t = d->matrices[s.index];
        x.in = t.in;
        x.row_stride = t.in_row_stride;
        x.matrix_stride = t.in_matrix_stride;
        x.out = t.out;
        x.out_row_stride = t.out_row_stride;
        x.out_matrix_stride = t.out_matrix_stride;
        if (s.whole) x.partial = nullptr;
      },
      ws, nullptr, stream);
  if (st != LA_OK) return st;
  st = directions(wide, [&](const la::DirectionGroup* g, int count) {
    return la::launch_normalise(g, count, d->in_type,
                                static_cast<float>(std::ldexp(1.0, p.step[0].x)), p.eps, nullptr,
                                stream, la::max_grid());
  });
  if (st != LA_OK) return st;
  return enqueue_products(
      wide, p, la::Product::kOut, d->out_type, 0.0f,
      [&](const Stack& s, la::ProductGroup& x) {
        x.out = d->matrices[s.index].out;
        x.out_ld = d->matrices[s.index].out_row_stride;
        x.out_stride = d->matrices[s.index].out_matrix_stride;
        x.vectors = aligned(x.out, 16) && (s.rows == 1 || x.out_ld % 8 == 0) &&
                    (s.count == 1 || x.out_stride % 8 == 0);
      },
      ws, nullptr, stream);
}

// ---- the Muon step ---------------------------------------------------------------------

la_status plan_layer(const la_muon_layer_desc* layer, const la_muon_params* hp, Polynomial* p,
                     std::vector<Stack>* stacks, int64_t* bytes) {
  if (layer == nullptr) return fail(LA_ERR_INVALID_ARGUMENT, "layer descriptor is NULL");
  if (layer->num_tensors < 0 || layer->num_tensors > LA_MAX_TENSORS)
    return fail(LA_ERR_INVALID_ARGUMENT, "num_tensors = %d, need 0..%d", layer->num_tensors,
                LA_MAX_TENSORS);
  if (layer->num_tensors > 0 && layer->tensors == nullptr)
    return fail(LA_ERR_INVALID_ARGUMENT, "tensors is NULL with num_tensors = %d",
                layer->num_tensors);
  if (layer->num_replicas < 1 || layer->num_replicas > LA_MAX_REPLICAS)
    return fail(LA_ERR_INVALID_ARGUMENT, "num_replicas = %d, need 1..%d", layer->num_replicas,
                LA_MAX_REPLICAS);
  if (layer->grad_dtype != LA_GRAD_BF16 && layer->grad_dtype != LA_GRAD_FP16)
    return fail(LA_ERR_UNSUPPORTED, "grad_dtype = %d, need LA_GRAD_BF16 or LA_GRAD_FP16",
                layer->grad_dtype);
  if (layer->out_dtype != LA_OUT_BF16 && layer->out_dtype != LA_OUT_FP16 &&
      layer->out_dtype != LA_OUT_NONE)
    return fail(LA_ERR_UNSUPPORTED, "out_dtype = %d, need LA_OUT_BF16, LA_OUT_FP16 or LA_OUT_NONE",
                layer->out_dtype);
  if (hp == nullptr) return fail(LA_ERR_INVALID_ARGUMENT, "hyperparameters are NULL");
  if (!(hp->momentum >= 0.0 && hp->momentum < 1.0))
    return fail(LA_ERR_INVALID_ARGUMENT, "momentum = %g, need 0 <= momentum < 1", hp->momentum);
  if (!finite_nonneg(hp->lr)) return fail(LA_ERR_INVALID_ARGUMENT, "lr = %g", hp->lr);
  if (!finite_nonneg(hp->weight_decay))
    return fail(LA_ERR_INVALID_ARGUMENT, "weight_decay = %g", hp->weight_decay);
  if (!(std::isfinite(hp->grad_unscale) && hp->grad_unscale > 0.0))
    return fail(LA_ERR_INVALID_ARGUMENT, "grad_unscale = %g, need finite > 0", hp->grad_unscale);
  if (hp->nesterov != 0 && hp->nesterov != 1)
    return fail(LA_ERR_INVALID_ARGUMENT, "nesterov = %d, need 0 or 1", hp->nesterov);
  if (hp->lr_scale != LA_LR_SCALE_NONE && hp->lr_scale != LA_LR_SCALE_ORIGINAL &&
      hp->lr_scale != LA_LR_SCALE_MATCH_RMS_ADAMW)
    return fail(LA_ERR_UNSUPPORTED, "lr_scale = %d, need a la_lr_scale", hp->lr_scale);
  la_status st = derive_polynomial(hp->polynomial, p);
  if (st != LA_OK) return st;
  for (int i = 0; i < layer->num_tensors; ++i) {
    const la_muon_tensor_desc& t = layer->tensors[i];
    if ((st = check_sides(i, t.rows, t.cols, t.count)) != LA_OK) return st;
    if (t.rows == 0 || t.cols == 0 || t.count == 0) continue;
    Stack s = {};
    s.rows = t.rows;
    s.cols = t.cols;
    s.count = t.count;
    s.index = i;
    stacks->push_back(s);
  }
  *bytes = lay_out(*stacks, *p, hp->nesterov != 0, true);
  return LA_OK;
}

double lr_scale(int kind, int64_t rows, int64_t cols) {
  const double r = static_cast<double>(rows), c = static_cast<double>(cols);
  return kind == LA_LR_SCALE_ORIGINAL           ? std::sqrt(std::max(1.0, r / c))
         : kind == LA_LR_SCALE_MATCH_RMS_ADAMW ? 0.2 * std::sqrt(std::max(r, c))
                                                : 1.0;
}

la_status muon_step(const la_muon_layer_desc* layer, const la_muon_params* hp, int32_t* flag,
                    const int32_t* skip, void* ws, int64_t ws_bytes, void* hip_stream) {
  Polynomial p;
  std::vector<Stack> stacks;
  int64_t bytes = 0;
  la_status st = plan_layer(layer, hp, &p, &stacks, &bytes);
  if (st != LA_OK) return st;
  if (flag != nullptr && !aligned(flag, 4))
    return fail(LA_ERR_MISALIGNED, "overflow_flag is not 4-byte aligned");
  if (skip != nullptr && !aligned(skip, 4))
    return fail(LA_ERR_MISALIGNED, "skip_if_nonzero is not 4-byte aligned");
  if (stacks.empty()) return ok();
  const bool copy = layer->out_dtype != LA_OUT_NONE;
  std::vector<Range> written, read;
  for (const Stack& s : stacks) {
    const la_muon_tensor_desc& t = layer->tensors[s.index];
    const int64_t n = s.rows * s.cols * s.count;
    la_status bad = LA_OK;
    auto buffer = [&](const void* q, int64_t b, const char* what, bool writes) {
      if (bad != LA_OK) return;
      if (q == nullptr)
        bad = fail(LA_ERR_INVALID_ARGUMENT, "tensor %d: %s is NULL", s.index, what);
      else if (!aligned(q, LA_ALIGNMENT))
        bad = fail(LA_ERR_MISALIGNED, "tensor %d: %s is not %d-byte aligned", s.index, what,
                   LA_ALIGNMENT);
      else
        (writes ? written : read).push_back(range(q, b * n, what, s.index));
    };
    buffer(t.master, 4, "master", true);
    buffer(t.momentum, 4, "momentum", true);
    if (copy) buffer(t.weight_out, 2, "weight_out", true);
    for (int r = 0; r < layer->num_replicas; ++r) buffer(t.grads[r], 2, "grads[r]", false);
    if (bad != LA_OK) return bad;
  }
  if ((st = check_workspace(ws, ws_bytes, bytes)) != LA_OK) return st;
  written.push_back(range(ws, bytes, "the workspace", -1));
  if (flag != nullptr) written.push_back(range(flag, 4, "the flag", -1));
  if (skip != nullptr) read.push_back(range(skip, 4, "skip_if_nonzero", -1));
  if ((st = check_disjoint(written, read)) != LA_OK) return st;

  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  // the direction of a stack: u = g + mu B in the workspace, or B itself
  auto direction = [&](const Stack& s) -> const float* {
    return hp->nesterov ? place<float>(ws, s.direction) : layer->tensors[s.index].momentum;
  };
  auto direction_stride = [&](const Stack& s) {
    return hp->nesterov ? s.numel_direction : s.rows * s.cols;
  };
  for (size_t first = 0; first < stacks.size(); first += la::kGroupsPerLaunch) {
    la::MomentumGroup g[la::kGroupsPerLaunch] = {};
    const int count =
        static_cast<int>(std::min<size_t>(la::kGroupsPerLaunch, stacks.size() - first));
    for (int i = 0; i < count; ++i) {
      const Stack& s = stacks[first + i];
      const la_muon_tensor_desc& t = layer->tensors[s.index];
      g[i].momentum = t.momentum;
      g[i].direction = hp->nesterov ? place<float>(ws, s.direction) : nullptr;
      for (int r = 0; r < layer->num_replicas; ++r)
        g[i].g[r] = static_cast<const uint16_t*>(t.grads[r]);
      g[i].partial = place<double>(ws, s.partial);
      g[i].numel = s.rows * s.cols;
      g[i].direction_stride = s.numel_direction;
      g[i].chunk = s.chunk;
      g[i].partials = s.partials;
      g[i].count = static_cast<int32_t>(s.count);
      g[i].vectors = s.count == 1 || g[i].numel % 8 == 0;
    }
    const hipError_t e = la::launch_momentum(
        g, count, layer->num_replicas, layer->grad_dtype == LA_GRAD_FP16,
        static_cast<float>(hp->momentum), static_cast<float>(hp->grad_unscale), flag, skip, stream,
        la::max_grid());
    if (e != hipSuccess)
      return fail(LA_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  }
  const int out = layer->out_dtype == LA_OUT_BF16   ? la::kBf16
                  : layer->out_dtype == LA_OUT_FP16 ? la::kFp16
                                                    : -1;
  const float decay = static_cast<float>(1.0 - hp->lr * hp->weight_decay);
  auto step = [&](const Stack& s) {
    return static_cast<float>(hp->lr * lr_scale(hp->lr_scale, s.rows, s.cols));
  };
  st = enqueue_narrow(
      stacks, p, la::kFp32, out, decay,
      [&](const Stack& s, la::NarrowGroup& x) {
        x.in = direction(s);
        x.row_stride = s.cols;
        x.matrix_stride = direction_stride(s);
        x.master = layer->tensors[s.index].master;
        x.out = copy ? layer->tensors[s.index].weight_out : nullptr;
        x.step = step(s);
      },
      ws, skip, stream);
  if (st != LA_OK) return st;
  std::vector<Stack> wide;
  for (const Stack& s : stacks)
    if (!s.narrow) wide.push_back(s);
  for (size_t first = 0; first < wide.size(); first += la::kGroupsPerLaunch) {
    la::DirectionGroup g[la::kGroupsPerLaunch];
    const int count =
        static_cast<int>(std::min<size_t>(la::kGroupsPerLaunch, wide.size() - first));
    for (int i = 0; i < count; ++i) {
      const Stack& s = wide[first + i];
      g[i] = direction_group(s, ws);
      g[i].in = direction(s);
      g[i].row_stride = s.cols;
      g[i].matrix_stride = direction_stride(s);
      g[i].vectors = s.cols % 8 == 0;
    }
    const hipError_t e = la::launch_normalise(
        g, count, la::kFp32, static_cast<float>(std::ldexp(1.0, p.step[0].x)), p.eps, skip, stream,
        la::max_grid());
    if (e != hipSuccess)
      return fail(LA_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  }
  return enqueue_products(
      wide, p, la::Product::kMuon, out, decay,
      [&](const Stack& s, la::ProductGroup& x) {
        x.master = layer->tensors[s.index].master;
        x.out = copy ? layer->tensors[s.index].weight_out : nullptr;
        x.vectors = s.cols % 8 == 0;
        x.step = step(s);
      },
      ws, skip, stream);
}

// No exception leaves the C ABI (a host allocation may fail).
template <typename F>
auto guarded(F f, decltype(f()) on_failure) -> decltype(f()) {
  try {
    return f();
  } catch (const std::exception& e) {
    fail(LA_ERR_INVALID_ARGUMENT, "%s", e.what());
    return on_failure;
  }
}

}  // namespace

extern "C" {

LA_API int64_t la_orthogonalize_workspace_bytes(const la_matrices_desc* matrices,
                                                const la_polynomial* polynomial) {
  return guarded(
      [&]() -> int64_t {
        Polynomial p;
        std::vector<Stack> stacks;
        int64_t bytes = 0;
        if (plan_matrices(matrices, polynomial, &p, &stacks, &bytes) != LA_OK) return -1;
        ok();
        return bytes;
      },
      -1);
}

LA_API la_status la_orthogonalize(const la_matrices_desc* matrices,
                                  const la_polynomial* polynomial, void* workspace,
                                  int64_t workspace_bytes, void* hip_stream) {
  return guarded(
      [&] { return orthogonalize(matrices, polynomial, workspace, workspace_bytes, hip_stream); },
      LA_ERR_INVALID_ARGUMENT);
}

LA_API int64_t layer_muon_workspace_bytes(const la_muon_layer_desc* layer,
                                          const la_muon_params* hp) {
  return guarded(
      [&]() -> int64_t {
        Polynomial p;
        std::vector<Stack> stacks;
        int64_t bytes = 0;
        if (plan_layer(layer, hp, &p, &stacks, &bytes) != LA_OK) return -1;
        ok();
        return bytes;
      },
      -1);
}

LA_API la_status layer_muon_step(const la_muon_layer_desc* layer, const la_muon_params* hp,
                                 int32_t* overflow_flag, const int32_t* skip_if_nonzero,
                                 void* workspace, int64_t workspace_bytes, void* hip_stream) {
  return guarded(
      [&] {
        return muon_step(layer, hp, overflow_flag, skip_if_nonzero, workspace, workspace_bytes,
                         hip_stream);
      },
      LA_ERR_INVALID_ARGUMENT);
}

}  // extern "C"
