// Internal interface between the C ABI of the norms (la_norm_api.cpp) and
// their kernels (la_norm.hip). Not installed; callers use
// include/layeradam.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace la {

// Rows of a tensor: row i * inner + j at p + i * outer_stride + j * inner_stride.
struct NormRows {
  void* p;
  int64_t outer_stride, inner_stride;
};

struct NormArgs {
  NormRows x, residual, y, sum;              // forward; backward: x alone
  NormRows dy, dsum, dx;                     // backward
  const void* weight;                        // null: ones
  const void* bias;                          // null: none
  float* mean;                               // layer norm
  float* rstd;                               // 1 / spread
  float* partial;                            // backward: parts x (1 or 2) x cols
  float* coefficients;                       // backward of long rows: two per row
  void *dweight, *dbias;                     // null: not wanted
  int32_t rows, inner;
  int32_t parts;                             // backward: partial sums of the parameters' gradients
  int32_t rows_per_part;
  int32_t cols;
  int32_t layer;                             // 1: layer norm, 0: RMS norm
  int32_t type, weight_type, grad_type;      // la_element_type
  float eps, inverse_cols;
};

// Rows up to this many bytes are held in registers beside what their columns
// need, up to this many elements alone in those of 1024 lanes.
constexpr int kNormRegisterBytes = 32768;
constexpr int kNormWideCols = 32768;

// The backward pass' parts: how many sums over rows are formed side by side,
// and of how many rows each; and the most that any call of up to these rows has.
struct NormParts {
  int32_t parts, rows_per_part, most;
};
NormParts norm_parts(int64_t rows, int64_t cols, int type);

hipError_t launch_norm_forward(const NormArgs& a, hipStream_t stream, int64_t max_grid);
// The backward pass over rows of up to kNormWideCols elements, by their type.
hipError_t norm_backward_bf16(const NormArgs& a, hipStream_t stream, int64_t max_grid);
hipError_t norm_backward_fp16(const NormArgs& a, hipStream_t stream, int64_t max_grid);
hipError_t norm_backward_fp32(const NormArgs& a, hipStream_t stream, int64_t max_grid);

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t stream, int64_t max_grid);

}  // namespace la
