// la_norm_api.cpp -- the C ABI of layer norm and RMS norm (declared in
// include/layeradam.h). Host side only: checks every argument before anything
// is enqueued and lays the backward pass' workspace out.

#include <hip/hip_runtime.h>

#include <cmath>

#include "la_checks.h"
#include "la_norm.h"

namespace {

using la::aligned;
using la::fail;
using la::NormArgs;
using la::ok;
using la::Range;
using la::range;
using la::type_bytes;

// Elements between rows, and of a whole tensor: keep every offset far from 64 bits.
constexpr int64_t kMostStride = int64_t(1) << 40;
constexpr double kMostExtent = 0x1p56;
constexpr int64_t kMostRows = (int64_t(1) << 30);  // row counts and steps past them fit 32 bits

bool is_type(int t) { return t == LA_TYPE_BF16 || t == LA_TYPE_FP16 || t == LA_TYPE_FP32; }

la_status check_norm(const la_norm_desc* n) {
  if (n == nullptr) return fail(LA_ERR_INVALID_ARGUMENT, "norm descriptor is NULL");
  if (n->kind != LA_NORM_LAYER && n->kind != LA_NORM_RMS)
    return fail(LA_ERR_UNSUPPORTED, "kind = %d, need a la_norm_kind", n->kind);
  if (!is_type(n->type))
    return fail(LA_ERR_UNSUPPORTED, "type = %d, need a la_element_type", n->type);
  if (!is_type(n->weight_type))
    return fail(LA_ERR_UNSUPPORTED, "weight_type = %d, need a la_element_type", n->weight_type);
  if (n->outer < 0 || n->inner < 0 || n->cols < 0 || n->outer > kMostRows ||
      n->inner > kMostRows || n->outer * n->inner > kMostRows || n->cols > LA_MAX_SIDE ||
      static_cast<double>(n->outer * n->inner) * static_cast<double>(n->cols) > 0x1p44)
    return fail(LA_ERR_INVALID_ARGUMENT,
                "%lld x %lld rows of %lld elements: at most 2^30 rows of %d, 2^44 elements",
                static_cast<long long>(n->outer), static_cast<long long>(n->inner),
                static_cast<long long>(n->cols), LA_MAX_SIDE);
  if (!(std::isfinite(static_cast<float>(n->eps)) && n->eps >= 0.0))
    return fail(LA_ERR_INVALID_ARGUMENT, "eps = %g", n->eps);
  return LA_OK;
}

// The buffers of one call: checked one by one, then against each other.
struct Buffers {
  const la_norm_desc& n;
  std::vector<Range> written, read;
  bool merged = true;  // rows of every tensor are one stride apart
  la_status st = LA_OK;

  void rows(const la_rows& t, const char* what, bool writes, la::NormRows* to) {
    if (st != LA_OK) return;
    if (t.data == nullptr) {
      st = fail(LA_ERR_INVALID_ARGUMENT, "%s is NULL", what);
      return;
    }
    const int64_t bytes = type_bytes(n.type);
    if (!aligned(t.data, bytes)) {
      st = fail(LA_ERR_MISALIGNED, "%s is not aligned to its element", what);
      return;
    }
    const int64_t outer = n.outer > 1 ? t.outer_stride : 0;
    const int64_t inner = n.inner > 1 ? t.inner_stride : 0;
    const bool fits = outer >= 0 && inner >= 0 && outer <= kMostStride && inner <= kMostStride &&
                      static_cast<double>(n.outer) * static_cast<double>(outer) +
                              static_cast<double>(n.inner) * static_cast<double>(inner) <=
                          kMostExtent;
    // rows that are written may not touch: one of the two strides passes over the other's
    // rows (looked at where `fits`, which keeps these sums far from 64 bits)
    auto passes = [&](int64_t over, int64_t rows_over, int64_t within, int64_t rows_within) {
      return (rows_within < 2 || within >= n.cols) &&
             (rows_over < 2 || over >= (rows_within - 1) * within + n.cols);
    };
    if (!fits || (writes && !passes(outer, n.outer, inner, n.inner) &&
                  !passes(inner, n.inner, outer, n.outer))) {
      st = fail(LA_ERR_INVALID_ARGUMENT,
                "strides of %s (outer %lld, inner %lld) for %lld x %lld rows of %lld elements", what,
                static_cast<long long>(t.outer_stride), static_cast<long long>(t.inner_stride),
                static_cast<long long>(n.outer), static_cast<long long>(n.inner),
                static_cast<long long>(n.cols));
      return;
    }
    merged = merged && (n.inner < 2 || n.outer < 2 || outer == n.inner * inner);
    *to = {t.data, outer, inner};
    const int64_t extent = (n.outer - 1) * outer + (n.inner - 1) * inner + n.cols;
    (writes ? written : read).push_back(range(t.data, bytes * extent, what));
  }

  // `count` elements; null where `optional`
  void flat(const void* p, int type, int64_t count, const char* what, bool writes, bool optional) {
    if (st != LA_OK || (p == nullptr && optional)) return;
    if (p == nullptr) st = fail(LA_ERR_INVALID_ARGUMENT, "%s is NULL", what);
    else if (!aligned(p, type_bytes(type)))
      st = fail(LA_ERR_MISALIGNED, "%s is not aligned to its element", what);
    else if (count > 0)
      (writes ? written : read).push_back(range(p, type_bytes(type) * count, what));
  }
};

NormArgs arguments(const la_norm_desc& n) {
  NormArgs a = {};
  a.weight = n.weight;
  a.bias = n.bias;
  a.rows = static_cast<int32_t>(n.outer * n.inner);
  a.cols = static_cast<int32_t>(n.cols);
  a.layer = n.kind == LA_NORM_LAYER;
  a.type = n.type;
  a.weight_type = n.weight_type;
  a.eps = static_cast<float>(n.eps);
  a.inverse_cols = static_cast<float>(1.0 / static_cast<double>(n.cols));
  return a;
}

// One stride where it serves every tensor: no division per row.
void merge(NormArgs& a, const la_norm_desc& n, bool merged) {
  a.inner = static_cast<int32_t>(n.inner);
  if (n.inner > 1 && !merged) return;
  a.inner = 1;
  if (n.inner > 1)
    for (la::NormRows* t : {&a.x, &a.residual, &a.y, &a.sum, &a.dy, &a.dsum, &a.dx})
      t->outer_stride = t->inner_stride;
}

la_status forward(const la_norm_desc* n, const la_norm_forward_io* io, void* stream) {
  la_status st = check_norm(n);
  if (st != LA_OK) return st;
  if (io == nullptr) return fail(LA_ERR_INVALID_ARGUMENT, "io is NULL");
  NormArgs a = arguments(*n);
  if (a.rows == 0 || n->cols == 0) return ok();
  Buffers b{*n};
  const bool added = io->residual.data != nullptr;
  if (added != (io->sum.data != nullptr))
    return fail(LA_ERR_INVALID_ARGUMENT, "a residual and its sum are given together");
  b.rows(io->x, "x", false, &a.x);
  if (added) {
    b.rows(io->residual, "residual", false, &a.residual);
    b.rows(io->sum, "sum", true, &a.sum);
  }
  b.rows(io->y, "y", true, &a.y);
  b.flat(n->weight, n->weight_type, n->cols, "weight", false, true);
  b.flat(n->bias, n->weight_type, n->cols, "bias", false, true);
  if (a.layer) b.flat(io->mean, LA_TYPE_FP32, a.rows, "mean", true, true);
  b.flat(io->rstd, LA_TYPE_FP32, a.rows, "rstd", true, true);
  if (b.st != LA_OK) return b.st;
  if ((st = la::check_disjoint(b.written, b.read)) != LA_OK) return st;
  a.mean = a.layer ? io->mean : nullptr;
  a.rstd = io->rstd;
  merge(a, *n, b.merged);
  const hipError_t e =
      la::launch_norm_forward(a, static_cast<hipStream_t>(stream), la::max_grid());
  if (e != hipSuccess) return fail(LA_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

// Places of the backward pass' workspace; returns its bytes.
int64_t plan_backward(const la_norm_desc& n, int32_t* parts, int32_t* rows_per_part,
                      int64_t* partial, int64_t* coefficients) {
  *parts = 0;
  *rows_per_part = 1;
  const int64_t rows = n.outer * n.inner;
  if (n.cols == 0 || rows == 0) return 0;
  const la::NormParts p = la::norm_parts(rows, n.cols, n.type);
  *parts = p.parts;
  *rows_per_part = p.rows_per_part;
  la::Taker take;
  // places for the parts of every smaller number of rows too, some of which have more
  *partial = take(2 * 4 * int64_t(p.most) * n.cols);
  *coefficients = take(n.cols > la::kNormWideCols ? 8 * rows : 0);
  return take.at;
}

la_status backward(const la_norm_desc* n, const la_norm_backward_io* io, void* ws,
                   int64_t ws_bytes, void* stream) {
  la_status st = check_norm(n);
  if (st != LA_OK) return st;
  if (io == nullptr) return fail(LA_ERR_INVALID_ARGUMENT, "io is NULL");
  if (!is_type(io->grad_type))
    return fail(LA_ERR_UNSUPPORTED, "grad_type = %d, need a la_element_type", io->grad_type);
  NormArgs a = arguments(*n);
  if (n->cols == 0) return ok();
  Buffers b{*n};
  if (a.rows > 0) {
    b.rows(io->dy, "dy", false, &a.dy);
    b.rows(io->x, "x", false, &a.x);
    if (io->residual_grad.data != nullptr)
      b.rows(io->residual_grad, "residual_grad", false, &a.dsum);
    if (io->dx.data != nullptr) b.rows(io->dx, "dx", true, &a.dx);
    if (a.layer) b.flat(io->mean, LA_TYPE_FP32, a.rows, "mean", false, false);
    b.flat(io->rstd, LA_TYPE_FP32, a.rows, "rstd", false, false);
  }
  b.flat(n->weight, n->weight_type, n->cols, "weight", false, true);
  b.flat(io->dweight, io->grad_type, n->cols, "dweight", true, true);
  b.flat(io->dbias, io->grad_type, n->cols, "dbias", true, true);
  if (b.st != LA_OK) return b.st;
  int64_t partial = 0, coefficients = 0;
  const int64_t needed = plan_backward(*n, &a.parts, &a.rows_per_part, &partial, &coefficients);
  if ((st = la::check_workspace(ws, ws_bytes, needed)) != LA_OK) return st;
  if (needed > 0) b.written.push_back(range(ws, needed, "the workspace"));
  if ((st = la::check_disjoint(b.written, b.read)) != LA_OK) return st;
  a.mean = const_cast<float*>(io->mean);
  a.rstd = const_cast<float*>(io->rstd);
  a.partial = la::place<float>(ws, partial);
  a.coefficients = la::place<float>(ws, coefficients);
  a.dweight = io->dweight;
  a.dbias = io->dbias;
  a.grad_type = io->grad_type;
  merge(a, *n, b.merged);
  const hipError_t e =
      la::launch_norm_backward(a, static_cast<hipStream_t>(stream), la::max_grid());
  if (e != hipSuccess) return fail(LA_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

LA_API la_status la_norm_forward(const la_norm_desc* norm, const la_norm_forward_io* io,
                                 void* hip_stream) {
  return la::guarded([&] { return forward(norm, io, hip_stream); }, LA_ERR_INVALID_ARGUMENT);
}

LA_API int64_t la_norm_backward_workspace_bytes(const la_norm_desc* norm) {
  return la::guarded(
      [&]() -> int64_t {
        if (check_norm(norm) != LA_OK) return -1;
        int32_t parts, rows_per_part;
        int64_t partial, coefficients;
        const int64_t bytes =
            plan_backward(*norm, &parts, &rows_per_part, &partial, &coefficients);
        ok();
        return bytes;
      },
      -1);
}

LA_API la_status la_norm_backward(const la_norm_desc* norm, const la_norm_backward_io* io,
                                  void* workspace, int64_t workspace_bytes, void* hip_stream) {
  return la::guarded(
      [&] { return backward(norm, io, workspace, workspace_bytes, hip_stream); },
      LA_ERR_INVALID_ARGUMENT);
}

}  // extern "C"
