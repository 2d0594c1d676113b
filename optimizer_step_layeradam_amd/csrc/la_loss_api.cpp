// la_loss_api.cpp -- the C ABI of the linear cross entropy (declared in
// include/layeradam.h). Host side only: checks every argument before anything
// is enqueued, lays the workspace out and enqueues the passes.

#include <hip/hip_runtime.h>

#include <cmath>

#include "la_checks.h"
#include "la_loss.h"

namespace {

using la::aligned;
using la::fail;
using la::LossProduct;
using la::ok;
using la::place;
using la::Range;
using la::range;
using la::round_up;

constexpr int64_t kMostStride = int64_t(1) << 40;  // keeps every offset far from 64 bits

// What a piece takes at most where the caller does not say: with 16 bits an
// element 16384 tokens of a vocabulary of 131072 in one piece.
constexpr int64_t kDefaultPieceBytes = int64_t(4) << 30;

constexpr int64_t kUnlimited = int64_t(1) << 62;  // room for parts

struct Plan {
  bool gradients, pack;
  int64_t rows, width;        // padded to whole depths
  int64_t chunks;
  int64_t columns, pieces;    // of a piece; 0 without gradients
  la::LossSizes sizes;
  la::LossShapes shapes;
  bool direct;                // dx comes straight from its product
  // places in the workspace
  int64_t count, index, target, xc, wc, sums, target_logit, lse, losses, piece, input_parts,
      weight_parts;
  int64_t bytes;
};

la_status check(const la_cross_entropy_desc* d) {
  if (d == nullptr) return fail(LA_ERR_INVALID_ARGUMENT, "descriptor is NULL");
  if (d->type != LA_TYPE_BF16 && d->type != LA_TYPE_FP16)
    return fail(LA_ERR_UNSUPPORTED, "type = %d, need LA_TYPE_BF16 or LA_TYPE_FP16", d->type);
  if (d->target_type != LA_INDEX_INT32 && d->target_type != LA_INDEX_INT64)
    return fail(LA_ERR_UNSUPPORTED, "target_type = %d, need a la_index_type", d->target_type);
  if (d->reduction != LA_REDUCE_SUM && d->reduction != LA_REDUCE_MEAN)
    return fail(LA_ERR_UNSUPPORTED, "reduction = %d, need a la_reduction", d->reduction);
  if (d->tokens < 0 || d->hidden < 1 || d->vocab < 1 || d->tokens > LA_MAX_SIDE ||
      d->hidden > LA_MAX_SIDE || d->vocab > LA_MAX_SIDE)
    return fail(LA_ERR_INVALID_ARGUMENT,
                "%lld tokens, hidden %lld, vocab %lld: need 0, 1 and 1 to %d of each",
                static_cast<long long>(d->tokens), static_cast<long long>(d->hidden),
                static_cast<long long>(d->vocab), LA_MAX_SIDE);
  if (!std::isfinite(static_cast<float>(d->grad_scale)))
    return fail(LA_ERR_INVALID_ARGUMENT, "grad_scale = %g", d->grad_scale);
  auto stride = [&](int64_t s, int64_t rows, int64_t cols, const char* what) -> la_status {
    if (rows > 1 && (s < cols || s > kMostStride))
      return fail(LA_ERR_INVALID_ARGUMENT, "%s = %lld for rows of %lld elements", what,
                  static_cast<long long>(s), static_cast<long long>(cols));
    return LA_OK;
  };
  la_status st;
  // rows of x that are one row are fine to read
  if (d->tokens > 1 && (d->x_row_stride < 0 || d->x_row_stride > kMostStride))
    return fail(LA_ERR_INVALID_ARGUMENT, "x_row_stride = %lld",
                static_cast<long long>(d->x_row_stride));
  if ((st = stride(d->weight_row_stride, d->vocab, d->hidden, "weight_row_stride")) != LA_OK)
    return st;
  if (d->dx != nullptr &&
      (st = stride(d->dx_row_stride, d->tokens, d->hidden, "dx_row_stride")) != LA_OK)
    return st;
  if (d->dweight != nullptr &&
      (st = stride(d->dweight_row_stride, d->vocab, d->hidden, "dweight_row_stride")) != LA_OK)
    return st;
  return LA_OK;
}

// The layout in `pieces` pieces (or fewer, of the same columns), without its shapes
// and what depends on them.
void divide(const la_cross_entropy_desc& d, int64_t pieces, Plan* p) {
  p->gradients = d.dx != nullptr || d.dweight != nullptr;
  p->rows = round_up(d.tokens, la::kLossDepth);
  p->width = round_up(d.hidden, la::kLossDepth);
  // the products read the weight as it lies where its rows are whole depths of
  // aligned pieces, and a padded copy otherwise
  const int64_t ldw = d.vocab > 1 ? d.weight_row_stride : d.hidden;
  p->pack = p->width != d.hidden || ldw % 8 != 0 || ldw > LA_MAX_SIDE || !aligned(d.weight, 16);
  p->columns = p->gradients ? round_up((d.vocab + pieces - 1) / pieces, la::kPieceUnit) : 0;
  p->pieces = p->gradients ? (d.vocab + p->columns - 1) / p->columns : 0;
  p->sizes = {d.tokens, d.hidden, d.vocab, p->columns, p->pieces, d.dx != nullptr,
              d.dweight != nullptr};
}

// Places for so many parts of dx and dw. (A part's bytes are a multiple of the
// workspace's alignment, and take nothing else with them.)
void place_all(const la_cross_entropy_desc& d, int64_t input_parts, int64_t weight_parts, Plan* p) {
  static_assert(4 * la::kLossDepth % LA_WORKSPACE_ALIGNMENT == 0, "");
  la::Taker take;
  p->count = take(4);
  p->index = take(4 * d.tokens);
  p->target = take(4 * d.tokens);
  p->xc = take(2 * p->rows * p->width);
  p->wc = take(p->pack ? 2 * d.vocab * p->width : 0);
  constexpr int64_t chunk = int64_t(1) << la::kLeastChunkShift;
  p->sums = take(8 * d.tokens * ((d.vocab + chunk - 1) / chunk));
  p->target_logit = take(4 * d.tokens);
  p->lse = take(4 * d.tokens);
  p->losses = take(4 * d.tokens);
  p->piece = take(2 * p->rows * p->columns);
  p->input_parts = take(4 * input_parts * d.tokens * p->width);
  p->weight_parts = take(4 * weight_parts * std::min(p->columns, d.vocab) * p->width);
  p->bytes = take.at;
}

// What a call in `pieces` pieces cannot do without.
int64_t least_bytes(const la_cross_entropy_desc& d, int64_t pieces) {
  Plan p;
  divide(d, pieces, &p);
  place_all(d, la::loss_least_parts(p.sizes), 0, &p);
  return p.bytes;
}

// The layout whose parts take `room` bytes at most beside that.
void lay_out(const la_cross_entropy_desc& d, int64_t pieces, int64_t room, Plan* p) {
  divide(d, pieces, p);
  p->shapes = la::loss_shapes(p->sizes, room);
  const int shift = p->shapes.chunk_shift;
  p->chunks = (d.vocab + (int64_t(1) << shift) - 1) >> shift;
  p->direct = p->pieces == 1 && p->shapes.input.parts == 1;
  place_all(d, d.dx != nullptr && !p->direct ? p->shapes.input.parts : 0,
            d.dweight != nullptr && p->shapes.weight.parts > 1 ? p->shapes.weight.parts : 0, p);
}

// The fewest pieces whose columns are at most `columns`, in whole units.
int64_t pieces_of(const la_cross_entropy_desc& d, int64_t columns) {
  columns = round_up(std::max<int64_t>(1, columns), la::kPieceUnit);
  return (d.vocab + columns - 1) / columns;
}

// The smallest workspace that serves: dx over several pieces is summed in it, so that
// one piece may need less than many.
int64_t least_of_all(const la_cross_entropy_desc& d) {
  return std::min(least_bytes(d, 1), least_bytes(d, pieces_of(d, la::kPieceUnit)));
}

// What a call in up to `pieces` pieces asks for, parts of every size included. Fewer
// pieces may need less: one takes no sum of dx over pieces, and larger ones fewer parts.
int64_t wanted_bytes(const la_cross_entropy_desc& d, int64_t pieces) {
  Plan p;
  lay_out(d, 1, kUnlimited, &p);
  int64_t bytes = p.bytes;
  while (pieces > 1 && least_bytes(d, pieces) < bytes) {  // which grows with fewer pieces
    lay_out(d, pieces, kUnlimited, &p);
    bytes = std::min(bytes, p.bytes);
    pieces = p.pieces - 1;  // the next longer columns
  }
  return bytes;
}

// The fewest pieces that the workspace holds, their parts in what is left of it.
// Where that is less than they would take, more and smaller pieces may be the
// faster ones (24 tokens' dx in one part leaves most compute units idle): the least
// modelled time of all up to the first that is not held back, past 16 of every
// sixteenth. False where the workspace holds none.
bool plan_for(const la_cross_entropy_desc& d, int64_t given, Plan* p) {
  if (given < least_of_all(d)) return false;
  const int64_t most = pieces_of(d, la::kPieceUnit);
  int64_t fewest = 1;
  if (least_bytes(d, 1) > given) {  // from two pieces on each more needs less
    int64_t held = most;
    for (fewest = 2; fewest < held;) {
      const int64_t middle = (fewest + held) / 2;
      if (least_bytes(d, middle) <= given) held = middle;
      else fewest = middle + 1;
    }
  }
  lay_out(d, fewest, given - least_bytes(d, fewest), p);
  if (!p->gradients) return true;
  Plan next = *p;
  while (next.shapes.held_back && next.pieces < most) {
    const int64_t pieces = std::max(next.pieces + 1 + next.pieces / 16,
                                    pieces_of(d, next.columns - la::kPieceUnit));
    const int64_t least = least_bytes(d, std::min(pieces, most));
    if (least > given) {  // one piece may need less than two
      divide(d, std::min(pieces, most), &next);
      continue;
    }
    lay_out(d, std::min(pieces, most), given - least, &next);
    if (next.shapes.time < p->shapes.time) *p = next;
  }
  return true;
}

la_status launch_failed(hipError_t e) {
  return fail(LA_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
}

la_status cross_entropy(const la_cross_entropy_desc* d, void* ws, int64_t ws_bytes,
                        void* hip_stream) {
  la_status st = check(d);
  if (st != LA_OK) return st;
  std::vector<Range> written, read;
  auto buffer = [&](const void* p, int64_t element, int64_t count, const char* what,
                    std::vector<Range>& list) {
    if (st != LA_OK) return;
    if (p == nullptr && count > 0) st = fail(LA_ERR_INVALID_ARGUMENT, "%s is NULL", what);
    else if (!aligned(p, element))
      st = fail(LA_ERR_MISALIGNED, "%s is not aligned to its element", what);
    else if (count > 0) list.push_back(range(p, element * count, what));
  };
  auto extent = [&](int64_t rows, int64_t stride) {
    return rows > 0 ? (rows > 1 ? (rows - 1) * stride : 0) + d->hidden : 0;
  };
  const int index_bytes = d->target_type == LA_INDEX_INT64 ? 8 : 4;
  buffer(d->x, 2, extent(d->tokens, d->x_row_stride), "x", read);
  buffer(d->weight, 2, extent(d->vocab, d->weight_row_stride), "weight", read);
  buffer(d->targets, index_bytes, d->tokens, "targets", read);
  buffer(d->loss, 4, 1, "loss", written);
  if (d->losses != nullptr) buffer(d->losses, 4, d->tokens, "losses", written);
  if (d->dx != nullptr) buffer(d->dx, 2, extent(d->tokens, d->dx_row_stride), "dx", written);
  if (d->dweight != nullptr)
    buffer(d->dweight, 2, extent(d->vocab, d->dweight_row_stride), "dweight", written);
  if (st != LA_OK) return st;
  Plan p;
  if (!plan_for(*d, ws_bytes, &p)) return la::check_workspace(ws, ws_bytes, least_of_all(*d));
  if ((st = la::check_workspace(ws, ws_bytes, p.bytes)) != LA_OK) return st;
  written.push_back(range(ws, p.bytes, "the workspace"));
  if ((st = la::check_disjoint(written, read)) != LA_OK) return st;

  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const int64_t max_grid = la::max_grid();
  la::LossProductArgs a = {};
  la::LossRows& r = a.r;
  r.x = static_cast<const uint16_t*>(d->x);
  r.targets = d->targets;
  r.x_stride = d->tokens > 1 ? d->x_row_stride : 0;
  r.ignore_index = d->ignore_index;
  r.tokens = static_cast<int32_t>(d->tokens);
  r.hidden = static_cast<int32_t>(d->hidden);
  r.vocab = static_cast<int32_t>(d->vocab);
  r.wide_targets = d->target_type == LA_INDEX_INT64;
  r.bf16 = d->type == LA_TYPE_BF16;
  r.mean = d->reduction == LA_REDUCE_MEAN;
  r.scale = static_cast<float>(d->grad_scale);
  r.count = place<int32_t>(ws, p.count);
  r.index = place<int32_t>(ws, p.index);
  r.target = place<int32_t>(ws, p.target);
  r.xc = place<uint16_t>(ws, p.xc);
  r.width = static_cast<int32_t>(p.width);
  r.sums = place<float2>(ws, p.sums);
  r.chunks = static_cast<int32_t>(p.chunks);
  r.chunk_shift = p.shapes.chunk_shift;
  r.target_logit = place<float>(ws, p.target_logit);
  r.lse = place<float>(ws, p.lse);
  r.losses = d->losses;
  r.compact_losses = place<float>(ws, p.losses);
  r.loss = d->loss;
  r.dx = static_cast<uint16_t*>(d->dx);
  r.dx_stride = d->tokens > 1 ? d->dx_row_stride : 0;
  a.w = static_cast<const uint16_t*>(d->weight);
  a.ldw = d->vocab > 1 ? d->weight_row_stride : d->hidden;
  a.direct = p.direct;
  a.dw = static_cast<uint16_t*>(d->dweight);
  a.dw_stride = d->vocab > 1 ? d->dweight_row_stride : 0;

  hipError_t e = la::launch_loss_gather(r, stream, max_grid);
  if (e != hipSuccess) return launch_failed(e);
  if (p.pack) {
    uint16_t* wc = place<uint16_t>(ws, p.wc);
    e = la::launch_pack(a.w, a.ldw, d->vocab, r.hidden, wc, r.width, stream, max_grid);
    if (e != hipSuccess) return launch_failed(e);
    a.w = wc;
    a.ldw = p.width;
  }
  auto product = [&](LossProduct what, int64_t first, int64_t columns) {
    a.piece.g = place<uint16_t>(ws, p.piece);
    a.piece.ld = static_cast<int32_t>(p.columns);
    a.piece.first = static_cast<int32_t>(first);
    a.piece.cols = static_cast<int32_t>(std::min(columns, d->vocab - first));
    const bool input = what == LossProduct::kInput, weight = what == LossProduct::kWeight;
    a.shape = input ? p.shapes.input : weight ? p.shapes.weight : p.shapes.logits;
    a.partial = place<float>(ws, input ? p.input_parts : p.weight_parts);
    const int64_t sum = input ? a.piece.cols : d->tokens;
    a.depth = static_cast<int32_t>(
        round_up(std::max<int64_t>(1, (sum + a.shape.parts - 1) / a.shape.parts), la::kLossDepth));
    return la::launch_loss_product(a, what, stream, max_grid);
  };
  if (!p.gradients) {
    if ((e = product(LossProduct::kSums, 0, d->vocab)) != hipSuccess) return launch_failed(e);
    e = la::launch_loss_lse(r, true, stream, max_grid);
    return e == hipSuccess ? ok() : launch_failed(e);
  }
  if (p.pieces > 1 &&
      (e = product(LossProduct::kSums, p.columns, d->vocab)) != hipSuccess)
    return launch_failed(e);
  if ((e = product(LossProduct::kKeep, 0, p.columns)) != hipSuccess) return launch_failed(e);
  if ((e = la::launch_loss_lse(r, false, stream, max_grid)) != hipSuccess) return launch_failed(e);
  e = la::launch_loss_softmax(r, a.piece, stream, max_grid);
  if (e != hipSuccess) return launch_failed(e);
  for (int64_t k = 0; k < p.pieces; ++k) {
    const int64_t first = k * p.columns;
    if (k > 0 && (e = product(LossProduct::kAgain, first, p.columns)) != hipSuccess)
      return launch_failed(e);
    a.add = k > 0;
    if (d->dx != nullptr && (e = product(LossProduct::kInput, first, p.columns)) != hipSuccess)
      return launch_failed(e);
    if (d->dweight != nullptr) {
      if ((e = product(LossProduct::kWeight, first, p.columns)) != hipSuccess)
        return launch_failed(e);
      if (a.shape.parts > 1 && (e = la::launch_loss_weight(a, stream, max_grid)) != hipSuccess)
        return launch_failed(e);
    }
  }
  if (d->dx != nullptr && !p.direct) {
    e = la::launch_loss_input(r, place<float>(ws, p.input_parts), p.shapes.input.parts, stream,
                              max_grid);
    if (e != hipSuccess) return launch_failed(e);
  }
  return ok();
}

}  // namespace

extern "C" {

LA_API int64_t la_linear_cross_entropy_workspace_bytes(const la_cross_entropy_desc* loss,
                                                       int64_t piece_columns) {
  return la::guarded(
      [&]() -> int64_t {
        if (check(loss) != LA_OK) return -1;
        if (piece_columns < 0) {
          fail(LA_ERR_INVALID_ARGUMENT, "piece_columns = %lld",
               static_cast<long long>(piece_columns));
          return -1;
        }
        const int64_t rows = std::max<int64_t>(1, round_up(loss->tokens, la::kLossDepth));
        const int64_t held = kDefaultPieceBytes / (2 * rows) / la::kPieceUnit * la::kPieceUnit;
        const int64_t columns =
            std::min<int64_t>(piece_columns > 0 ? piece_columns : held, LA_MAX_SIDE);
        const int64_t bytes = wanted_bytes(*loss, pieces_of(*loss, columns));
        ok();
        return bytes;
      },
      -1);
}

LA_API la_status la_linear_cross_entropy(const la_cross_entropy_desc* loss, void* workspace,
                                         int64_t workspace_bytes, void* hip_stream) {
  return la::guarded([&] { return cross_entropy(loss, workspace, workspace_bytes, hip_stream); },
                     LA_ERR_INVALID_ARGUMENT);
}

}  // extern "C"
