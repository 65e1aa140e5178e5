// kernels_tree.cu -- the tcgen05 cache attention for wide drafted trees: the plan of its pieces and its
// launches.
#include "cache_prompt.cuh"

namespace b2b {
namespace {

constexpr int kPlanThreads = 256;

struct TreeWork {
  int units, tiles;                    // units of the sequence, and the key tiles of each
};
__device__ __forceinline__ TreeWork tree_work(const AttendParams& p, int b, int& row_tiles) {
  const Sequence s = load_sequence(p.c, b, DK_PROMPT);
  row_tiles = (s.n * p.group + kPromptRows - 1) / kPromptRows;
  return TreeWork{p.c.heads * row_tiles, (s.len + kPromptKeys - 1) / kPromptKeys};
}

// How many key tiles a CTA's own start and end cost.
constexpr int kPieceStart = 8;

// Every block sums all sequences up, one per thread (tree_shape), and writes down its share of the pieces.
// Their longest is between one and three even shares: eight warps compare two lengths each by the waves that
// they take, since a few pieces more than SMs take twice as long as a few less.
__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const AttendParams p, int64_t most, int num_sms) {
  constexpr int kWarps = kPlanThreads / 32, kLengths = 2 * kWarps;
  __shared__ unsigned long long sums[kWarps];
  __shared__ int units_of[kPlanThreads], tiles_of[kPlanThreads], piece_at[kPlanThreads + 1], slot_at[kPlanThreads],
      count_of[kPlanThreads];
  __shared__ long long cost_of[kLengths];
  grid_launch_dependents();
  grid_dependency_wait();
  const TreePlan plan = tree_plan(p.meta, most, p.c.B);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  TreeWork w{0, 0};
  int row_tiles = 0;
  if (t < p.c.B) w = tree_work(p, t, row_tiles);
  units_of[t] = w.units;
  tiles_of[t] = w.tiles;
  // ---- an even share ----
  unsigned long long total = static_cast<unsigned long long>(w.units) * w.tiles;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) sums[warp] = total;
  __syncthreads();
  total = 0;
  for (int i = 0; i < kWarps; ++i) total += sums[i];
  const long long share = static_cast<long long>((total + num_sms - 1) / num_sms);
  auto length_of = [&](int k) -> int {
    const long long l = share + share * k / 8;
    return l < kMinPieceTiles ? kMinPieceTiles : l > 0x7FFFFFFF ? 0x7FFFFFFF : static_cast<int>(l);
  };
  // ---- the longest piece ----
  for (int k = warp; k < kLengths; k += kWarps) {
    const int l = length_of(k);
    int pieces = 0;
    for (int b = lane; b < p.c.B; b += 32)
      if (units_of[b] > 0) pieces += units_of[b] * ((tiles_of[b] - 1) / l + 1);
    pieces = __reduce_add_sync(0xffffffffu, pieces);
    if (lane == 0)
      cost_of[k] = static_cast<long long>((pieces + num_sms - 1) / num_sms) * (static_cast<long long>(l) + kPieceStart);
  }
  __syncthreads();
  int best = 0;
  for (int k = 1; k < kLengths; ++k)
    if (cost_of[k] < cost_of[best]) best = k;
  const int length = length_of(best);
  // ---- where the sequences' pieces and slots begin ----
  const int per_unit = w.units > 0 ? (w.tiles - 1) / length + 1 : 0;
  const int mine = w.units * per_unit, cut_here = per_unit > 1 ? mine : 0;
  unsigned long long upto = static_cast<unsigned long long>(mine) | static_cast<unsigned long long>(cut_here) << 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  unsigned long long ahead = 0, all = 0;
  for (int i = 0; i < kWarps; ++i) {
    ahead += i < warp ? sums[i] : 0ull;
    all += sums[i];
  }
  upto += ahead;
  const int first_slot = static_cast<int>(upto >> 32) - cut_here;
  piece_at[t] = static_cast<int>(upto & 0xFFFFFFFFu) - mine;
  slot_at[t] = per_unit > 1 ? first_slot : -1;
  count_of[t] = per_unit;
  if (t == 0) piece_at[kPlanThreads] = static_cast<int>(all & 0xFFFFFFFFu);
  if (blockIdx.x == 0 && t < p.c.B) plan.cuts[t] = make_int2(first_slot, per_unit);
  __syncthreads();
  // ---- the pieces ----
  const int pieces = piece_at[kPlanThreads];
  for (int i = static_cast<int>(blockIdx.x) * kPlanThreads + t; i < pieces;
       i += static_cast<int>(gridDim.x) * kPlanThreads) {
    int a = 0, z = kPlanThreads - 1;                 // the last sequence whose first piece is at most i
    while (a < z) {
      const int mid = (a + z + 1) / 2;
      if (piece_at[mid] <= i) a = mid;
      else z = mid - 1;
    }
    const int n = count_of[a], k = i - piece_at[a], unit = k / n, at = k - unit * n;
    TreePiece piece;
    piece.b = a;
    piece.h = unit % p.c.heads;
    piece.rt = unit / p.c.heads;
    piece.slot = -1;
    if (slot_at[a] >= 0) piece.slot = slot_at[a] + (piece.h * (units_of[a] / p.c.heads) + piece.rt) * n + at;
    piece.t0 = static_cast<int>(static_cast<int64_t>(tiles_of[a]) * at / n);
    piece.t1 = static_cast<int>(static_cast<int64_t>(tiles_of[a]) * (at + 1) / n);
    piece.pad[0] = piece.pad[1] = 0;
    if (i < most) plan.pieces[i] = piece;
  }
  if (blockIdx.x == 0 && t == 0) *plan.count = pieces < most ? pieces : static_cast<int>(most);
}

struct TreeShape {
  int64_t pieces, slots;               // at most
  bool cut;
};
TreeShape tree_shape(int64_t rows, const CacheView& c, int num_sms) {
  TreeShape s;
  const int64_t units = (rows + kPromptRows - 1) / kPromptRows * c.heads * c.B;
  const int64_t tiles = ((static_cast<int64_t>(c.max_pages) << c.page_shift) + kPromptKeys - 1) / kPromptKeys;
  s.cut = tree_cuts(units, tiles, num_sms) && c.B <= kPlanThreads;
  // pieces of at most L tiles, L >= all tiles / SMs: fewer than SMs besides one per unit, and fewer
  // than 2 SMs in units that are cut
  s.pieces = units + (s.cut ? num_sms : 0);
  s.slots = s.cut ? 2 * static_cast<int64_t>(num_sms) : 0;
  return s;
}

}  // namespace

int64_t tree_workspace(int64_t rows, const CacheView& c, int num_sms) {
  const TreeShape s = tree_shape(rows, c, num_sms);
  // uncut, of ragged sequences in more than one wave: the longest first
  if (!s.cut) return c.B > 1 && s.pieces > num_sms ? prompt_order_bytes(s.pieces / c.heads) : 0;
  return tree_plan_bytes(s.pieces, c.B) + s.slots * kPromptRows * (c.D + 1) * 4;
}
bool tree_fits(const CacheView& c) { return c.D <= 128 && c.max_new <= kMostTreeTokens; }

cudaError_t launch_tree(const AttendParams& p, int num_sms, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.c.max_new) * p.group;
  const TreeShape shape = tree_shape(rows, p.c, num_sms);
  if (shape.pieces > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const int row_tiles = static_cast<int>((rows + kPromptRows - 1) / kPromptRows);
  cudaError_t e = cudaSuccess;
  if (shape.cut) {
    const int64_t plan_blocks = (shape.pieces + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
    e = launch_early(tree_plan_kernel, plan_blocks, kPlanThreads, 0, s, p, shape.pieces, num_sms);
  } else if (p.meta != nullptr) {
    e = launch_prompt_order(p, row_tiles, s);
  }
  if (e != cudaSuccess) return e;
  switch (p.c.D) {
    case 64: e = launch_tree_units_64(shape.cut, p, row_tiles, shape.pieces, s); break;
    case 96: e = launch_tree_units_96(shape.cut, p, row_tiles, shape.pieces, s); break;
    case 128: e = launch_tree_units_128(shape.cut, p, row_tiles, shape.pieces, s); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess || !shape.cut) return e;
  return launch_tree_join(p, shape.pieces, num_sms, s);
}

}  // namespace b2b
