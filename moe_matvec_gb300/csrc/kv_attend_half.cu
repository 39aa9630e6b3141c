// Attention over the paged 8-bit cache: f16 and bfloat16 queries, 16 rows a fragment.
#include "kv_attend.cuh"

namespace qmv {

cudaError_t launch_attend_half(AttendParams& p, int D, cudaStream_t stream) {
  return launch_attend_as<true, false>(p, D, stream);
}

}  // namespace qmv
