// kernels_attend_d256.cu -- the split cache attention for head size 256.
#include "cache_attention.cuh"

namespace b2b {

cudaError_t launch_attend_256(int nt, const AttendParams& p, cudaStream_t s) {
  return launch_attend_d<256>(nt, p, s);
}

}  // namespace b2b
