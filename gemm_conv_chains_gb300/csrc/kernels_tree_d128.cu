// kernels_tree_d128.cu -- the tcgen05 cache attention for wide drafted trees of head size 128.
#include "cache_prompt.cuh"

namespace b2b {

cudaError_t launch_tree_units_128(bool cut, const AttendParams& p, int row_tiles, int64_t ctas, cudaStream_t s) {
  return launch_tree_d<128>(cut, p, row_tiles, ctas, s);
}

}  // namespace b2b
