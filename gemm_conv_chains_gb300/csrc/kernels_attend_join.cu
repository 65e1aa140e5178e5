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

// Of the tcgen05 kernel over drafted trees: the pieces of a unit have neighbouring slots.  `each` warps
// per row take every so-many-th piece, four on their way, and are joined in shared memory.  (16 sequences
// of 60 nodes, each row of 2 or 3 pieces: 36 us with a block of four warps per row, as above.)
constexpr int kTreeJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kTreeJoinWarps) tree_join_kernel(const AttendParams p, int64_t pieces,
                                                                        int each) {
  constexpr int kOwn = D / 32;                       // channels of a lane
  __shared__ float sums[kTreeJoinWarps][D], stat[kTreeJoinWarps][2];
  const CacheView& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t x = (static_cast<int64_t>(blockIdx.x) * kTreeJoinWarps + warp) / each;
  const int share = warp % each;
  const int head = static_cast<int>(x % p.q_heads);
  const int tq = static_cast<int>(x / p.q_heads % c.max_new);
  const int b = static_cast<int>(x / p.q_heads / c.max_new);
  const TreePlan plan = tree_plan(p.meta, pieces, c.B);
  int2 cut = make_int2(0, 0);                        // {first slot, pieces of a unit}
  Sequence s{0, 0, 0};
  if (b < c.B) {
    cut = plan.cuts[b];
    s = load_sequence(c, b, DK_PROMPT);
  }
  const bool here = tq < s.n && cut.y > 1;
  const int h = head / p.group, r = tq * p.group + head % p.group;
  const int row_tiles = (s.n * p.group + kPromptRows - 1) / kPromptRows;
  constexpr int64_t kPart = static_cast<int64_t>(kPromptRows) * (D + 1);
  const int rr = r % kPromptRows;
  const float* first =
      plan.parts + (cut.x + (static_cast<int64_t>(h) * row_tiles + r / kPromptRows) * cut.y) * kPart;
  float m = kNoMax, l = 0.f, acc[kOwn];
#pragma unroll
  for (int e = 0; e < kOwn; ++e) acc[e] = 0.f;
  constexpr int kFlight = 4;
  for (int i = share; here && i < cut.y; i += kFlight * each) {
    float lse[kFlight], v[kFlight][kOwn];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int at = i + k * each;
      const float* part = first + at * kPart;
      lse[k] = kNoMax;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) v[k][e] = 0.f;
      if (at < cut.y) {
        lse[k] = part[kPromptRows * D + rr];
#pragma unroll
        for (int e = 0; e < kOwn; ++e) v[k][e] = part[rr * D + kOwn * lane + e];
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) top = fmaxf(top, lse[k]);
    const float f = exp2_fast(m - top);
    m = top;
    l *= f;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) acc[e] *= f;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const float w = lse[k] <= kNoMax ? 0.f : exp2_fast(lse[k] - top);   // a NaN stays one
      l += w;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) acc[e] += w * v[k][e];
    }
  }
  if (each > 1) {
#pragma unroll
    for (int e = 0; e < kOwn; ++e) sums[warp][kOwn * lane + e] = acc[e];
    if (lane == 0) {
      stat[warp][0] = m;
      stat[warp][1] = l;
    }
    __syncthreads();
    if (share != 0) return;
    float top = kNoMax;
    for (int k = 0; k < each; ++k) top = fmaxf(top, stat[warp + k][0]);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) acc[e] = 0.f;
    for (int k = 0; k < each; ++k) {
      const float w = exp2_fast(stat[warp + k][0] - top);
      l += w * stat[warp + k][1];
#pragma unroll
      for (int e = 0; e < kOwn; ++e) acc[e] += w * sums[warp + k][kOwn * lane + e];
    }
  }
  if (!here) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* dst = p.out + ((s.row + static_cast<int64_t>(tq)) * p.q_heads + head) * D + kOwn * lane;
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    const float o = acc[e] * inv;
    dst[e] = static_cast<uint16_t>((p.is_bf16 ? narrow2<true>(o, 0.f) : narrow2<false>(o, 0.f)) & 0xFFFFu);
  }
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
  const int64_t rows = static_cast<int64_t>(p.c.B) * p.c.max_new * p.q_heads;
  int each = 1;                                      // few rows have many pieces each
  while (each < kTreeJoinWarps && rows * each < 16 * num_sms) each *= 2;
  const int64_t blocks = (rows * each + kTreeJoinWarps - 1) / kTreeJoinWarps;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  switch (p.c.D) {
    case 64: return launch_early(tree_join_kernel<64>, blocks, 32 * kTreeJoinWarps, 0, s, p, pieces, each);
    case 96: return launch_early(tree_join_kernel<96>, blocks, 32 * kTreeJoinWarps, 0, s, p, pieces, each);
    case 128: return launch_early(tree_join_kernel<128>, blocks, 32 * kTreeJoinWarps, 0, s, p, pieces, each);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace b2b
