// decoder.h -- internal interface of the decoder-block operators (rotary positions, the
// append to a paged e4m3 cache, the attention over it, the cache's pages): launch parameters and
// launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace b2b {

// Error word of these operators: {code, kernel, what, index}; the first error wins.
enum DecoderError : uint32_t {
  DEC_ERR_POSITION = 1,   // a position outside the rotary table
  DEC_ERR_PAGE = 2,       // a page number outside the pool
  DEC_ERR_LENGTH = 3,     // a length that is below its new tokens or above its page table
  DEC_ERR_STARTS = 4,     // starts that decrease, leave the rows or exceed max_new
  DEC_ERR_PARENT = 5,     // a parent that is no row of the page table
  DEC_ERR_TOKEN = 6       // a kept token outside its sequence or out of order
};
enum DecoderKernel : uint32_t {
  DK_ROTARY = 32, DK_APPEND = 33, DK_ATTEND = 34, DK_PROMPT = 35, DK_PAGES = 36, DK_COPY = 37,
  DK_COMPACT = 38
};
constexpr uint32_t kCodeIndex = 2;   // B2B_ERR_SHAPE: a length, page number or position out of range

constexpr float kE4m3Max = 448.f;
constexpr float kScaleMin = 5.421010862427522e-20f;   // 2^-64

struct RotaryParams {
  const uint16_t* x;
  uint16_t* out;
  const float2* table;        // (cos, sin) of [positions][rot / 2]
  const int32_t* positions;
  int64_t T, ldx, ldo, table_len;
  int32_t H, D, rot;
  int32_t interleaved, inverse;
  uint32_t* err;
};

// The cache and how the sequences of a call lie in it.
struct CacheView {
  uint8_t* k;                 // [pages][heads][page][D]
  uint8_t* v;
  float* k_scale;             // [pages][heads]
  float* v_scale;
  const int32_t* page_table;  // [B][max_pages]
  const int32_t* lens;        // [B], new tokens included
  const int32_t* starts;      // [B + 1] or null: T / B rows each
  int64_t T;
  int32_t pages, heads, page_shift, D;
  int32_t B, max_pages, max_new;
  uint32_t* err;
};

struct AppendParams {
  CacheView c;
  const uint16_t* k;          // [T] rows of heads x D
  const uint16_t* v;
  const uint16_t* q;          // [T] rows of q_heads x D, or null
  uint16_t* q_out;
  const float2* table;        // or null: no rotation
  int64_t ldk, ldv, ldq, ldqo, table_len;
  int32_t q_heads, rot, interleaved;
};

struct AttendParams {
  CacheView c;
  const uint16_t* q;
  uint16_t* out;              // [T][q_heads][D]
  const float* slopes;        // [q_heads] or null
  const uint32_t* masks;      // drafted trees: [T][mask_words] bits, else null
  const int32_t* positions;   // of the new tokens [T], or null: their slots
  int32_t mask_words;
  int64_t ldq;
  int32_t q_heads, group, is_bf16;
  float scale, softcap;       // softcap 0: none
  float inv_softcap;
  int32_t grid, min_tiles, whole;
  float* part;                // split workspace: see cache_attention.cuh
  uint32_t* meta;             // [0]: tiles per run, [1 + b]: sequence b's first tile
  uint64_t wait_limit_ns;
};

// The page table of a step's sequences from the last step's.
struct PagesParams {
  const int32_t* table;       // [B][width]
  const int32_t* lens;        // [B]
  const int32_t* parents;     // [rows], or null: row r follows r
  const int32_t* kept;        // [rows], or null: all of the parent's tokens
  const int32_t* fresh;       // [rows], or null: no new tokens
  int32_t* table_out;         // [rows][width]
  int32_t* lens_out;          // [rows]
  int32_t* copies;            // [rows][3]
  int32_t* left;              // [1]
  uint32_t* owners;           // [pages] in the workspace
  void* kept_rows;            // [rows] of 16 bytes there
  int64_t pages;
  int32_t B, width, rows, page_shift;
  uint32_t* err;
};

struct CopyParams {
  CacheView c;
  const int32_t* copies;      // [n][3]: from, to, tokens
  int64_t n;
};

struct CompactParams {
  CacheView c;
  const int32_t* first;       // [B]
  const int32_t* tokens;      // [B][max_tokens]
  const int32_t* counts;      // [B]
  int32_t max_tokens;
};

// Launches with programmatic stream serialisation, as the chain kernels: the kernel may be scheduled
// while the one before it in the stream finishes, and waits for that (griddepcontrol.wait) before
// it touches global memory.
// `cluster`: consecutive CTAs of one thread-block cluster.
template <class... P, class... A>
cudaError_t launch_early_clusters(void (*fn)(P...), int64_t grid, int cluster, int block, int smem,
                                  cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}
template <class... P, class... A>
cudaError_t launch_early(void (*fn)(P...), int64_t grid, int block, int smem, cudaStream_t s, A... args) {
  return launch_early_clusters(fn, grid, 1, block, smem, s, args...);
}

cudaError_t launch_rotary(bool bf16, const RotaryParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_rotary_table(float2* table, int64_t n, int32_t half, const double* params,
                                cudaStream_t s);
cudaError_t launch_append(bool bf16, const AppendParams& p, int num_sms, cudaStream_t s);

// CTAs of the split kernel that an SM holds at once: its registers decide (one row tile of 8 at
// head sizes up to 128: 168 per thread).  More warps hide more of each strip's latencies.
__host__ __device__ constexpr int attend_ctas_per_sm(int D, int nt) {
  return nt == 1 && D <= 128 ? 3 : 2;
}
// The split kernel with row tiles of 8 nt query rows, per head size; tree: of drafted trees.
cudaError_t launch_attend_64(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_96(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_128(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_192(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_256(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_tree_64(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_tree_96(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_tree_128(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_tree_192(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_tree_256(int nt, const AttendParams& p, cudaStream_t s);
// The tcgen05 kernel for prompts (head sizes 64, 96, 128).
cudaError_t launch_prompt(const AttendParams& p, cudaStream_t s);
// Bytes of workspace that it takes for `rows` query rows per sequence and kv head (p.meta).
int64_t prompt_workspace(int64_t rows, int32_t B);
// Ranks its (sequence, row tile) pairs by their key tiles, the most first, into p.meta; its bytes, 0 for
// too many pairs.
cudaError_t launch_prompt_order(const AttendParams& p, int row_tiles, cudaStream_t s);
int64_t prompt_order_bytes(int64_t pairs);
// The same over drafted trees, contexts cut between CTAs where that fills the SMs (p.meta).
cudaError_t launch_tree(const AttendParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_tree_units_64(bool cut, const AttendParams& p, int row_tiles, int64_t ctas, cudaStream_t s);
cudaError_t launch_tree_units_96(bool cut, const AttendParams& p, int row_tiles, int64_t ctas, cudaStream_t s);
cudaError_t launch_tree_units_128(bool cut, const AttendParams& p, int row_tiles, int64_t ctas, cudaStream_t s);
int64_t tree_workspace(int64_t rows, const CacheView& c, int num_sms);
bool tree_fits(const CacheView& c);
// Whether contexts are cut: the units leave SMs idle, and an even share of all key tiles is shorter than
// a unit's by more than the 8 tiles that the plan and the joining kernel cost.
inline bool tree_cuts(int64_t units, int64_t tiles, int num_sms) {
  return 4 * units < 3 * num_sms && tiles - units * tiles / num_sms > 8;
}
cudaError_t launch_tree_join(const AttendParams& p, int64_t pieces, int num_sms, cudaStream_t s);
// Joins what the split kernel left in parts.
cudaError_t launch_attend_combine(const AttendParams& p, int nt, int num_sms, cudaStream_t s);

// Bytes of workspace that the page table's kernel takes, and the most rows that it does.
int64_t pages_workspace(int64_t pages, int64_t rows);
constexpr int32_t kMostPageRows = 4096;
cudaError_t launch_pages(PagesParams p, void* workspace, int num_sms, cudaStream_t s);
cudaError_t launch_copy(const CopyParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_compact(const CompactParams& p, int num_sms, cudaStream_t s);
constexpr int kMostCompactCluster = 16;
// CTAs per (sequence, kv head, pool) of the compaction, a power of two of at most `most`, what the device
// holds in one cluster: more than one where the items leave SMs idle and a wave of each has tokens.
inline int compact_ctas(int64_t items, int wave, int max_tokens, int num_sms, int most) {
  int ctas = 1;
  while (2 * ctas <= most && items * ctas < num_sms && static_cast<int64_t>(ctas) * wave < max_tokens) ctas *= 2;
  return ctas;
}

}  // namespace b2b
