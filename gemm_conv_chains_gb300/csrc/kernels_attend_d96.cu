// kernels_attend_d96.cu -- the split cache attention for head size 96.
#include "cache_attention.cuh"

namespace b2b {

cudaError_t launch_attend_96(int nt, const AttendParams& p, cudaStream_t s) {
  return launch_attend_d<96>(nt, p, s);
}

}  // namespace b2b
