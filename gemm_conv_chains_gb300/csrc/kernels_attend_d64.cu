// kernels_attend_d64.cu -- the split cache attention for head size 64.
#include "cache_attention.cuh"

namespace b2b {

cudaError_t launch_attend_64(int nt, const AttendParams& p, cudaStream_t s) {
  return launch_attend_d<64, false>(nt, p, s);
}

}  // namespace b2b
