// la_norm_backward_fp16.hip -- the norms' backward pass over FP16 rows.

#include "la_norm_backward.h"

namespace la {

hipError_t norm_backward_fp16(const NormArgs& a, hipStream_t stream, int64_t max_grid) {
  return backward_rows<Fp16>(a, stream, max_grid);
}

}  // namespace la
