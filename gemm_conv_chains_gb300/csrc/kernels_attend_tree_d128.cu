// kernels_attend_tree_d128.cu -- the split cache attention of drafted trees for head size 128.
#include "cache_attention.cuh"

namespace b2b {

cudaError_t launch_attend_tree_128(int nt, const AttendParams& p, cudaStream_t s) {
  return launch_attend_d<128, true>(nt, p, s);
}

}  // namespace b2b
