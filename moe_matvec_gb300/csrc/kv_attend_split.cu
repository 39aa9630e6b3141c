// Attention over the paged 8-bit cache: queries in two f16 parts, 8 rows a fragment.
#include "kv_attend.cuh"

namespace qmv {

cudaError_t launch_attend_split(AttendParams& p, int D, cudaStream_t stream) {
  return launch_attend_as<false, false>(p, D, stream);
}

}  // namespace qmv
