// la_norm_backward_fp32.hip -- the norms' backward pass over FP32 rows.

#include "la_norm_backward.h"

namespace la {

hipError_t norm_backward_fp32(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  return backward_rows<Fp32>(a, stream, max_grid);
}

}  // namespace la
