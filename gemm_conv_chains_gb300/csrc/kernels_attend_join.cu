// kernels_attend_join.cu -- joins the partial results of the row tiles that the cache attention cut
// between CTAs.
#include "cache_attention.cuh"
#include "cache_prompt.cuh"

namespace b2b {

// One block per query row and share of its channels.  A part is RT rows of D normalised sums and RT
// log2 sums of weights.  Groups of `lanes` threads (four channels each) take every so-many-th part with
// a running maximum of their own, four loads in flight, and are joined in shared memory: latency bound,
// a few KB per block.  part_of(i): where part i begins; rr: the row's number in it; d0: the block's first
// channel; out: the row.
template <class PartOf>
__device__ __forceinline__ void join_row(int parts, PartOf part_of, int rr, int RT, int D, int lanes, int d0,
                                         bool bf16, uint16_t* out) {
  extern __shared__ float sh[];
  const int groups = blockDim.x / lanes;
  const int grp = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int d = d0 + 4 * lane;
  constexpr int kFlight = 4;
  float m = kNoMax, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = grp; i < parts; i += kFlight * groups) {
    float lse[kFlight];
    float4 v[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int at = i + k * groups;
      lse[k] = kNoMax;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (at < parts) {
        const float* part = part_of(at);
        lse[k] = part[RT * D + rr];
        v[k] = *reinterpret_cast<const float4*>(part + rr * D + d);
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) top = fmaxf(top, lse[k]);
    const float f = exp2_fast(m - top);
    m = top;
    l *= f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const float w = lse[k] <= kNoMax ? 0.f : exp2_fast(lse[k] - top);   // a NaN stays one
      l += w;
      acc.x += w * v[k].x;
      acc.y += w * v[k].y;
      acc.z += w * v[k].z;
      acc.w += w * v[k].w;
    }
  }
  float* stat = sh;                                  // [groups][2], then [groups][lanes] float4
  float4* put = reinterpret_cast<float4*>(sh + ((2 * groups + 3) & ~3));
  if (grp < groups) {
    put[grp * lanes + lane] = acc;
    if (lane == 0) {
      stat[2 * grp] = m;
      stat[2 * grp + 1] = l;
    }
  }
  __syncthreads();
  if (threadIdx.x >= lanes) return;
  float top = kNoMax;
  for (int k = 0; k < groups; ++k) top = fmaxf(top, stat[2 * k]);
  float sum = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < groups; ++k) {
    const float w = exp2_fast(stat[2 * k] - top);
    const float4 v = put[k * lanes + lane];
    sum += w * stat[2 * k + 1];
    acc.x += w * v.x;
    acc.y += w * v.y;
    acc.z += w * v.z;
    acc.w += w * v.w;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2*>(out + d) =
      bf16 ? make_uint2(narrow2<true>(acc.x * inv, acc.y * inv), narrow2<true>(acc.z * inv, acc.w * inv))
           : make_uint2(narrow2<false>(acc.x * inv, acc.y * inv), narrow2<false>(acc.z * inv, acc.w * inv));
}

// The row that a block of either kernel below joins.
struct JoinRow {
  int share, head, tq, b;
};
__device__ __forceinline__ JoinRow join_row_of(const AttendParams& p, int shares) {
  JoinRow j;
  int64_t x = blockIdx.x;
  j.share = static_cast<int>(x % shares);
  x /= shares;
  j.head = static_cast<int>(x % p.q_heads);
  j.tq = static_cast<int>(x / p.q_heads % p.c.max_new);
  j.b = static_cast<int>(x / p.q_heads / p.c.max_new);
  return j;
}

// Of the split kernel: a row tile of `tiles` numbered tiles from number a on lies in the runs a / per ..
// (a + tiles - 1) / per; one run: the row is already written.
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams p, int RT, int lanes,
                                                          int shares) {
  const CacheView& c = p.c;
  const int D = c.D;
  const JoinRow j = join_row_of(p, shares);
  grid_launch_dependents();
  // (also for the lengths: the kernel before the split one may have written them)
  grid_dependency_wait();
  const Sequence s = load_sequence(c, j.b, DK_ATTEND);
  if (j.tq >= s.n) return;
  const int h = j.head / p.group;
  const int r = j.tq * p.group + j.head % p.group;
  const int row_tiles = (s.n * p.group + RT - 1) / RT;
  const uint32_t tiles = (s.len + kTileTokens - 1) / kTileTokens;
  const uint32_t per = p.meta[0];
  const uint32_t a = p.meta[1 + j.b] + (static_cast<uint32_t>(h) * row_tiles + r / RT) * tiles;
  const uint32_t c0 = a / per, c1 = (a + tiles - 1) / per;
  if (c0 == c1) return;
  const int64_t part_floats = static_cast<int64_t>(RT) * (D + 1);
  const float* first = p.part + (2 * static_cast<int64_t>(c0) + (c0 * per < a ? 1 : 0)) * part_floats;
  const float* rest = p.part + 2 * (static_cast<int64_t>(c0) + 1) * part_floats;   // slot 0 of the later runs
  join_row(static_cast<int>(c1 - c0) + 1,
           [&](int i) { return i == 0 ? first : rest + 2 * (i - 1) * part_floats; }, r % RT, RT, D, lanes,
           4 * j.share * lanes, p.is_bf16 != 0, p.out + ((s.row + static_cast<int64_t>(j.tq)) * p.q_heads + j.head) * D);
}

// Of the tcgen05 kernel over drafted trees: the pieces of a unit have neighbouring slots.
__global__ void __launch_bounds__(256) tree_join_kernel(const AttendParams p, int64_t pieces, int lanes,
                                                        int shares) {
  const CacheView& c = p.c;
  const JoinRow j = join_row_of(p, shares);
  grid_launch_dependents();
  grid_dependency_wait();
  const TreePlan plan = tree_plan(p.meta, pieces, c.B);
  const int2 cut = plan.cuts[j.b];                   // {first slot, pieces of a unit}
  const Sequence s = load_sequence(c, j.b, DK_PROMPT);
  if (j.tq >= s.n || cut.y <= 1) return;
  const int h = j.head / p.group;
  const int r = j.tq * p.group + j.head % p.group;
  const int row_tiles = (s.n * p.group + kPromptRows - 1) / kPromptRows;
  const int64_t part_floats = static_cast<int64_t>(kPromptRows) * (c.D + 1);
  const float* first =
      plan.parts + (cut.x + (static_cast<int64_t>(h) * row_tiles + r / kPromptRows) * cut.y) * part_floats;
  join_row(cut.y, [&](int i) { return first + i * part_floats; }, r % kPromptRows, kPromptRows, c.D, lanes,
           4 * j.share * lanes, p.is_bf16 != 0, p.out + ((s.row + static_cast<int64_t>(j.tq)) * p.q_heads + j.head) * c.D);
}

namespace {
// Few rows may have many parts each (a long context): more blocks and more groups per row.
struct JoinShape {
  int shares, lanes, threads, smem;
  int64_t blocks;
};
JoinShape join_shape(const AttendParams& p, int num_sms) {
  JoinShape j;
  const int64_t rows = static_cast<int64_t>(p.c.B) * p.c.max_new * p.q_heads;
  j.shares = 1;
  while (rows * j.shares < num_sms && p.c.D / 4 / (2 * j.shares) >= 4 && p.c.D / 4 % (2 * j.shares) == 0)
    j.shares *= 2;
  j.lanes = p.c.D / 4 / j.shares;
  j.threads = rows < 4 * num_sms ? 256 : 128;
  const int groups = j.threads / j.lanes;
  j.smem = 4 * (((2 * groups + 3) & ~3) + 4 * groups * j.lanes);
  j.blocks = rows * j.shares;
  return j;
}
}  // namespace

cudaError_t launch_attend_combine(const AttendParams& p, int nt, int num_sms, cudaStream_t s) {
  const JoinShape j = join_shape(p, num_sms);
  if (j.blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_early(attend_join_kernel, j.blocks, j.threads, j.smem, s, p, nt * 8, j.lanes, j.shares);
}

cudaError_t launch_tree_join(const AttendParams& p, int64_t pieces, int num_sms, cudaStream_t s) {
  const JoinShape j = join_shape(p, num_sms);
  if (j.blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_early(tree_join_kernel, j.blocks, j.threads, j.smem, s, p, pieces, j.lanes, j.shares);
}

}  // namespace b2b
