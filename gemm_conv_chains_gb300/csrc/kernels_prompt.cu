// kernels_prompt.cu -- the tcgen05 cache attention for prompts, head sizes 64, 96 and 128, and the
// order in which its CTAs take ragged sequences.
#include "cache_prompt.cuh"

namespace b2b {

// order[r] = the pair (numbered as plain_pair does) with the r-th most key tiles.
__global__ void __launch_bounds__(kRankedPairs) prompt_order_kernel(const AttendParams p, int row_tiles,
                                                                    int* order) {
  __shared__ int key_tiles[kRankedPairs];
  grid_launch_dependents();
  grid_dependency_wait();
  const int mine = threadIdx.x, pairs = row_tiles * p.c.B;
  if (mine < pairs) {
    PromptUnit u;
    int b, rt;
    plain_pair(p, row_tiles, mine, b, rt);
    (void)prompt_unit(p, b, 0, rt, u);
    key_tiles[mine] = u.tiles;
  }
  __syncthreads();
  if (mine >= pairs) return;
  int rank = 0;
  for (int i = 0; i < pairs; ++i)
    rank += key_tiles[i] > key_tiles[mine] || (key_tiles[i] == key_tiles[mine] && i < mine) ? 1 : 0;
  order[rank] = mine;
}

int64_t prompt_workspace(int64_t rows, int32_t B) {
  const int64_t row_tiles = (rows + kPromptRows - 1) / kPromptRows;
  return B > 1 && row_tiles > 1 && row_tiles * B <= kRankedPairs ? 4 * kRankedPairs : 0;
}

int64_t prompt_order_bytes(int64_t pairs) { return pairs <= kRankedPairs ? 4 * kRankedPairs : 0; }
cudaError_t launch_prompt_order(const AttendParams& p, int row_tiles, cudaStream_t s) {
  return launch_early(prompt_order_kernel, 1, kRankedPairs, 0, s, p, row_tiles, reinterpret_cast<int*>(p.meta));
}

cudaError_t launch_prompt(const AttendParams& p, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.c.max_new) * p.group;
  const int64_t row_tiles = (rows + kPromptRows - 1) / kPromptRows;
  const int64_t ctas = row_tiles * p.c.heads * p.c.B;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if (p.meta != nullptr) {
    if (cudaError_t e = launch_prompt_order(p, static_cast<int>(row_tiles), s); e != cudaSuccess) return e;
  }
  switch (p.c.D) {
    case 64: return launch_prompt_d<64, kCausal>(p, static_cast<int>(row_tiles), ctas, s);
    case 96: return launch_prompt_d<96, kCausal>(p, static_cast<int>(row_tiles), ctas, s);
    case 128: return launch_prompt_d<128, kCausal>(p, static_cast<int>(row_tiles), ctas, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace b2b
