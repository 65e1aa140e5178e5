// kernels_prompt.cu -- the tcgen05 cache attention for prompts, head sizes 64, 96 and 128.
#include "cache_prompt.cuh"

namespace b2b {

cudaError_t launch_prompt(const AttendParams& p, cudaStream_t s) {
  switch (p.c.D) {
    case 64: return launch_prompt_d<64>(p, s);
    case 96: return launch_prompt_d<96>(p, s);
    case 128: return launch_prompt_d<128>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace b2b
