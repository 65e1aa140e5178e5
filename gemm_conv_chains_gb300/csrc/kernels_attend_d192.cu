// kernels_attend_d192.cu -- the split cache attention for head size 192.
#include "cache_attention.cuh"

namespace b2b {

cudaError_t launch_attend_192(int nt, const AttendParams& p, cudaStream_t s) {
  return launch_attend_d<192, false>(nt, p, s);
}

}  // namespace b2b
