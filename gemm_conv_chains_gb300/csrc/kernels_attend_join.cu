// kernels_attend_join.cu -- joins the partial results of the row tiles that the split cache
// attention cut between CTAs, and chooses its row tiles.
#include "cache_attention.cuh"

namespace b2b {

// One block per query row.  A row tile of `tiles` numbered tiles from number a on lies in the
// runs a / per .. (a + tiles - 1) / per; one run: the row is already written.  The weights
// 2^(lse_i - max) are computed once per row in shared memory, so that the sums over the parts
// are independent loads; groups of D / 4 threads take every so-many-th part.
__global__ void attend_join_kernel(const AttendParams p, int RT) {
  extern __shared__ float sh[];
  const CacheView& c = p.c;
  const int D = c.D;
  const int64_t x = blockIdx.x;
  const int head = static_cast<int>(x % p.q_heads);
  const int tq = static_cast<int>(x / p.q_heads % c.max_new);
  const int b = static_cast<int>(x / p.q_heads / c.max_new);
  const Sequence s = load_sequence(c, b, DK_ATTEND);
  grid_dependency_wait();
  if (tq >= s.n) return;
  const int h = head / p.group;
  const int r = tq * p.group + head % p.group;
  const int row_tiles = (s.n * p.group + RT - 1) / RT;
  const int64_t tiles = (s.len + kTileTokens - 1) / kTileTokens;
  const int64_t per = p.meta[0];
  const int64_t a = p.meta[1 + b] + (static_cast<int64_t>(h) * row_tiles + r / RT) * tiles;
  const int64_t c0 = a / per, c1 = (a + tiles - 1) / per;
  if (c0 == c1) return;
  const int parts = static_cast<int>(c1 - c0) + 1;
  const int64_t part_floats = static_cast<int64_t>(RT) * (D + 1);
  const float* first = p.part + (2 * c0 + (c0 * per < a ? 1 : 0)) * part_floats;
  const float* rest = p.part + 2 * (c0 + 1) * part_floats;   // slot 0 of the later runs
  const int rr = r % RT;
  auto part_of = [&](int i) { return i == 0 ? first : rest + 2 * (i - 1) * part_floats; };

  float* weight = sh;
  float* scratch = sh + p.grid;
  float top = kNoMax;
  for (int i = threadIdx.x; i < parts; i += blockDim.x) {
    const float v = __ldg(part_of(i) + RT * D + rr);
    weight[i] = v;
    top = fmaxf(top, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) top = fmaxf(top, scratch[w]);
  __syncthreads();

  const int lanes = D / 4, groups = blockDim.x / lanes;
  const int grp = threadIdx.x / lanes, d = 4 * (threadIdx.x % lanes);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  if (grp < groups) {
#pragma unroll 4
    for (int i = grp; i < parts; i += groups) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(part_of(i) + rr * D + d));
      const float f = weight[i] <= kNoMax ? 0.f : exp2_fast(weight[i] - top);
      sum += f;
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
    float4* put = reinterpret_cast<float4*>(scratch);
    put[grp * lanes + d / 4] = acc;
    if (d == 0) weight[p.grid + 4 * groups * lanes + grp] = sum;
  }
  __syncthreads();
  if (threadIdx.x < lanes) {
    const float4* get = reinterpret_cast<const float4*>(scratch);
    for (int k = 1; k < groups; ++k) {
      const float4 v = get[k * lanes + threadIdx.x];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
      sum += weight[p.grid + 4 * groups * lanes + k];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* dst = p.out + ((s.row + static_cast<int64_t>(tq)) * p.q_heads + head) * D + d;
    *reinterpret_cast<uint2*>(dst) =
        p.is_bf16
            ? make_uint2(narrow2<true>(acc.x * inv, acc.y * inv), narrow2<true>(acc.z * inv, acc.w * inv))
            : make_uint2(narrow2<false>(acc.x * inv, acc.y * inv),
                         narrow2<false>(acc.z * inv, acc.w * inv));
  }
}

cudaError_t launch_attend_combine(const AttendParams& p, int nt, int threads, cudaStream_t s) {
  const int64_t blocks = static_cast<int64_t>(p.c.B) * p.c.max_new * p.q_heads;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const int lanes = p.c.D / 4, groups = threads / lanes;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = sizeof(float) * (p.grid + 4 * groups * lanes + groups + 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel, p, nt * 8);
}

}  // namespace b2b
