// Internal interface between the C ABI of the linear cross entropy
// (la_loss_api.cpp) and its kernels (la_loss.hip, la_loss_product.hip). Not
// installed; callers use include/layeradam.h.
//
// With tokens t that count (n of them, known on the device alone), hidden
// states x_t, weight rows w_v and targets y_t:
//
//   z_tv = x_t . w_v;  lse_t = log sum_v exp z_tv;  loss_t = lse_t - z_t,y
//   g_tv = exp(z_tv - lse_t) - [v = y_t]
//   dx_t = c sum_v g_tv w_v;  dw_v = c sum_t g_tv x_t
//
// The tokens that count are gathered first: what is ignored costs nothing and
// nothing of it (a NaN, say) can reach a sum. The vocabulary is taken in
// pieces, and one piece of a T x V matrix is held at a time:
//
//   logits of the first piece -> e = exp(z - max of some columns) with the
//       maxima and the sums beside them            product, kKeep
//   logits of the other pieces -> their maxima and sums alone        kSums
//   lse and losses from those; e -> g in place                       softmax
//   for each piece: dx += g W, dw = g^T x              products, kInput, kWeight
//       (other pieces first form g from their logits and lse again   kAgain)
//
// so a piece that holds the whole vocabulary costs three products, and every
// piece after the first one more.
//
// Number formats. Products multiply 16-bit elements with binary32 sums. e is
// binary16 times 2^14, in (0, 2^14]: 11 bits down to 2^-28 of the largest of
// its columns. g is of the tensors' type, for binary16 times 2^14, so that
// probabilities down to 2^-28 keep 11 bits; the entry of the target, the
// difference of nearly equal numbers where a token is predicted well, comes from
// binary32. c, with the mean's 1 / n, multiplies the binary32 sums.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace la {

// Columns of the held piece are a multiple of this; its rows, and the depth of
// every sum, of 64.
constexpr int kPieceUnit = 256;
constexpr int kLossDepth = 64;

// Scale of e, and of g in binary16.
constexpr float kLossExponent = 14.0f, kLossScale = 16384.0f;

// Exponentials are powers of two: of z log2 e, which one multiply-add forms to
// the last bit or so of z. log2 e itself is 1.3e-8 off in binary32, a fifth of
// what rounding z costs.
constexpr float kLog2e = 1.44269504088896341f;
constexpr double kLn2 = 0.693147180559945309;

// What the passes over tokens need.
struct LossRows {
  const uint16_t* x;        // tokens x hidden
  const void* targets;      // int64 or int32
  int64_t x_stride;
  int64_t ignore_index;
  int32_t tokens, hidden, vocab;
  int32_t wide_targets;     // 1: int64
  int32_t bf16;             // 1: BF16, 0: FP16
  int32_t mean;             // 1: the loss and c are divided by n
  float scale;              // c without that
  // in the workspace
  int32_t* count;           // n
  int32_t* index;           // of the gathered tokens: where they come from
  int32_t* target;          // their targets, -1 where out of range
  uint16_t* xc;             // gathered, rows x width, zeros behind hidden
  int32_t width;            // hidden, up to whole depths
  float2* sums;             // chunks x tokens: maximum m of z log2 e, sum of e = 2^(z log2 e - m + 14)
  int32_t chunks;           // of vocab columns
  int32_t chunk_shift;      // log2 of a chunk's columns
  float* target_logit;
  float* lse;               // times log2 e
  // outputs
  float* losses;            // per token, or null
  float* compact_losses;    // workspace
  float* loss;
  uint16_t* dx;             // or null
  int64_t dx_stride;
};

// The held piece of e, later g: rows x ld.
struct LossPiece {
  uint16_t* g;
  int32_t first, cols;      // columns of the vocabulary
  int32_t ld;
};

enum class LossProduct { kKeep, kSums, kAgain, kInput, kWeight };

// Tiles of the products: 32 x 128, 64 x 128, 128 x 128 and 256 x 256.
enum class LossTile { kSmallest, kSmall, kMedium, kLarge };

// A product's tiles, and the parts that its sum is cut into.
struct LossShape {
  LossTile tile;
  int32_t parts;
};

// What a call's shapes depend on.
struct LossSizes {
  int64_t tokens, hidden, vocab;
  int64_t columns, pieces;  // of a piece; 0: no gradients
  bool input, weight;       // which of the two
};

struct LossShapes {
  LossShape logits, input, weight;
  int32_t chunk_shift;      // log2 of the columns of one of `sums`, by the logits' tile
  double time;              // of the call's products, modelled, us
  bool held_back;           // some product would take more parts than there is room for
};

// `room`: bytes that binary32 results may take beside those that no call does
// without (kLeastChunkShift, loss_least_parts).
LossShapes loss_shapes(const LossSizes& s, int64_t room);

// The shortest chunk of columns that a tile forms has 2^6: `sums` has places for these
// whatever the tile, so that fewer tokens never need more of a workspace.
constexpr int kLeastChunkShift = 6;

// Parts of dx that lie in the workspace in any case: its sum over several pieces.
constexpr int64_t loss_least_parts(const LossSizes& s) { return s.input && s.pieces > 1 ? 1 : 0; }

struct LossProductArgs {
  LossRows r;
  LossPiece piece;
  LossShape shape;          // of this product
  const uint16_t* w;        // weight, rows ldw elements apart, zeros behind hidden up to width
  int64_t ldw;
  float* partial;           // results in binary32, parts x rows x width: always of kInput, unless
                            // `direct`; of kWeight where its sum has parts
  int32_t depth;            // elements of one part, a multiple of 64
  int32_t add;              // kInput: to what is there
  int32_t direct;           // kInput: the results are dx
  uint16_t* dw;             // kWeight
  int64_t dw_stride;
};

hipError_t launch_loss_gather(const LossRows& r, hipStream_t stream, int64_t max_grid);
hipError_t launch_pack(const uint16_t* from, int64_t stride, int64_t rows, int cols, uint16_t* to,
                       int width, hipStream_t stream, int64_t max_grid);
// lse and losses from the chunks; with `sum`, the loss from those.
hipError_t launch_loss_lse(const LossRows& r, bool sum, hipStream_t stream, int64_t max_grid);
// e becomes g in the first piece; the loss.
hipError_t launch_loss_softmax(const LossRows& r, const LossPiece& piece, hipStream_t stream,
                               int64_t max_grid);
// dx, or dw of a piece, from the parts.
hipError_t launch_loss_input(const LossRows& r, const float* partial, int parts,
                             hipStream_t stream, int64_t max_grid);
hipError_t launch_loss_weight(const LossProductArgs& a, hipStream_t stream, int64_t max_grid);

hipError_t launch_loss_product(const LossProductArgs& a, LossProduct what, hipStream_t stream,
                               int64_t max_grid);

}  // namespace la
