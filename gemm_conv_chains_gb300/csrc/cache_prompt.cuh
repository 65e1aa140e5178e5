// cache_prompt.cuh -- attention over the paged e4m3 cache for many query rows per sequence and
// kv head (prompts, long chunks): tcgen05 products over 128-row tiles.
//
// The same function as cache_attention.cuh.  4 D operations per (query row, key) against one
// byte per key channel and 256 rows: bound by the tensor cores, and next to them by the
// exponentials (one per 4 D operations) and the softmax's instructions.  A CTA takes 256 query
// rows of one (sequence, kv head), all query heads of the group side by side so that a key is
// turned into fp16 once for all of them, and walks the keys in tiles of 128:
//
//   warps 0-3, 4-7   softmax of row tile A, B (one row per thread); stage Q, write the output
//   warps 8-11       keys:   e4m3 pages -> fp16 tiles, 128B-swizzled, two of them; the scales
//   warps 12-15      values: the same
//   warp 16          TMEM, MMA issue:  S = Q K^T,  O += P V   (17-19 only complete its warpgroup)
//
// TMEM: S and O of both row tiles (4 x 128 columns); P (fp16 pairs) lies over the first half of
// its S.  The two row tiles alternate: while one is in its softmax the tensor core works on the
// other (P V of this key tile, then Q K^T of the next; MMAs of one thread run in issue order,
// so S of the next tile follows the products that read the P it covers).
//
// Precision as in cache_attention.cuh.  The scales of the value pages enter the exponent (as log2)
// and are divided out of the row sum, so that a probability costs one multiply-add, one exponential
// and one addition.  A row's reference, of z + log2 scale, only moves when a product would be above
// 2^15, and O, in TMEM, is rescaled only then.
//
// Measured: prompts of 451 to 2048 tokens behind 1192 to 4096 cached ones (4 sequences, 32 query
// heads on 8 of 128 channels): 228 us, 1.07 PFLOP/s, 0.56 of the library's dense bf16 rate.  The
// split kernel took 1480 us on them.  The tensor pipe is busy for 44 % of the time: a key tile's
// chain (S ready, 128 columns read, exponentials, P written, P V and the next Q K^T issued) takes
// ~3700 clocks, of which the products are ~1100 and a softmax warp's work ~1500; the rest are
// hand-offs.  64 channels take nearly as long per key tile as 128 (187 us for the same prompts), so
// the bound is this latency; the tensor memory that they leave free is not used.  Capped or biased
// scores take two passes over every tile (with a cap, up to 1024 tokens behind up to 2048: 417 us for 116).  Tried on an earlier form of
// 236 us, and slower: one issuing warp per row tile (353 us: the softmaxes fall into step and the
// tensor core idles; 264 when the two take turns), waits that spin (238), rolled MMA loops (246), the
// operand waits hidden behind the other row tile's products (239 to 252).
#pragma once

#include <type_traits>

#include "decoder_device.cuh"

namespace b2b {

constexpr int kPromptRows = 256;       // query rows of a CTA: two M = 128 tiles
constexpr int kPromptKeys = 128;       // keys per tile
constexpr int kPromptThreads = 640;
// Registers per thread of the softmax, producer and MMA warpgroups: 2 x 136 + 2 x 72 + 64 <= 5 x 96,
// what 640 threads are launched with.
constexpr int kSoftmaxRegs = 136, kProducerRegs = 72, kIssueRegs = 64;
constexpr int kGranule = 16;           // tokens that surely share a page
constexpr int kGranules = kPromptKeys / kGranule;
// The region in which some rows of a CTA see a token and others do not: at most 256 tokens,
// from the start of a key tile on.
constexpr int kEdgeTokens = 512;

enum PromptSite : uint32_t {
  PS_QFULL = 48, PS_KFULL, PS_KEMPTY, PS_VFULL, PS_VEMPTY, PS_SFULL, PS_PREADY, PS_OFULL, PS_DRAIN, PS_MERGE
};

template <int D>
struct PromptSmem {
  static constexpr int kBlocks = (D + 63) / 64;                 // 128-byte-wide blocks of a row
  static constexpr int kTile = kBlocks * 128 * 128;             // 128 rows, bytes
  static constexpr int kQ = 0;                                  // two row tiles
  static constexpr int kK = kQ + 2 * kTile;                     // two key tiles
  static constexpr int kV = kK + 2 * kTile;
  static constexpr int kScales = kV + 2 * kTile;                // [4][granules] (k scale, log2 v scale)
  static constexpr int kNan = kScales + 4 * kGranules * 8;      // [kEdgeTokens][D / 32] bits
  static constexpr int kBar = kNan + kEdgeTokens * (D / 32) * 4;
  static constexpr int kBytes = kBar + 256;
  static constexpr int kAlloc = kBytes + 1024;                  // the tiles start 1 KB aligned
  static constexpr int kMasks = kBytes;                         // trees: [words][256 rows]
  static constexpr int kTreeAlloc = kAlloc + (kEdgeTokens - kPromptKeys) / 32 * kPromptRows * 4;
};

struct PromptBars {
  uint64_t qfull[2], kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pready[2], ofull[2], drain, merge;
  uint32_t tmem, abort_flag, nan_any;
};
static_assert(sizeof(PromptBars) <= 256, "barrier block");

// 32 columns of this warp's lanes; the registers pass through the wait.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                 "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 lanes per instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// A page's value scale as the exponent that it adds.  A scale of zero stands for 2^-96: that page
// takes its weight in the row sum, and what comes out of it is less than any other's by so much that
// fp16 has nothing of it; a row that sees no other pages is told by its sum (kNoValues).  A NaN
// stays one.
constexpr float kNoValues = 5.0706024e30f;          // 2^102: 2^-64, the least scale of an append, over 2^23 tokens
__device__ __forceinline__ float exponent_of(float scale) {
  const float lv = log2f(scale);
  return lv < -96.f ? -96.f : lv;
}

// What a CTA works on: up to 256 query rows of one sequence and kv head.
struct PromptUnit {
  Sequence s;
  int b, h, row0, rows, start, kv_end, tiles, row_tiles;
  int t0;                              // trees: the piece's first key tile (tiles: how many),
  int slot;                            // and where its part goes, -1: the unit is not cut
};

// Row tile rt of sequence b, for kv head h; false where the sequence has no such rows.
__device__ __forceinline__ bool prompt_unit(const AttendParams& p, int b, int h, int rt,
                                            PromptUnit& u) {
  u.h = h;
  u.b = b;
  u.s = load_sequence(p.c, b, DK_PROMPT);
  u.row0 = rt * kPromptRows;
  u.rows = u.s.n * p.group;
  u.tiles = 0;
  if (u.row0 >= u.rows) return false;
  const int last = u.row0 + kPromptRows < u.rows ? u.row0 + kPromptRows - 1 : u.rows - 1;
  u.start = u.s.len - u.s.n;
  u.kv_end = u.start + last / p.group + 1;
  u.tiles = (u.kv_end + kPromptKeys - 1) / kPromptKeys;
  u.row_tiles = u.rows - u.row0 > 128 ? 2 : 1;
  return true;
}

// Drafted trees.  All rows of a sequence see its older tokens, few of them new ones, so that a
// sequence's units all walk the same key tiles, and one sequence may have nearly all of them.  Where the
// units leave SMs idle, those of more than L key tiles are cut into equal pieces of at most L, with
// a CTA each, and a further kernel joins their parts; L is an even share of all key tiles over the SMs or up
// to three of them, whichever takes the least time in whole waves, at least kMinPieceTiles.  A small kernel
// ahead writes the pieces down from the lengths.
//
// A unit of one row tile (`pairs`) gives every other key tile to the second softmax, with S, P and O of its
// own over a second copy of Q, so that two chains are on their way; at the end the two are merged.  Warps
// whose 32 rows are all past the unit's pass.  The codes of the tile after next are asked for into L2.
// 32 sequences of up to 8 nodes over up to 4096 tokens, 32 heads on 8 of 128, bf16: 92 us without the three,
// 86 with pairs, 80 with L2 ahead too, 74 with all.
//
// A CTA's own start and end are ~11 us.  A tile of 128 channels is 1.2 us in pairs and 1.5 us with two row tiles
// (bf16; 0.67 and 1.34 at the library's dense rate), 2.0 and 2.4 us in fp16 (LO below; 1.0 and 2.0): with two
// row tiles the products are the bound.  In pairs a tile takes ~2300 clocks, and three parts take 2200 to 2400 each,
// by clocks read in every role: the key warps (1000 to 1600 until the tile is stored, 1000 for its scales, the next
// tile's loads and the line ahead), the issuing warp (waits of ~200, P V 350, S 570) and half of a softmax's chain
// (of ~2000 of its own and 2400 of hand-offs and products).  Without the exponentials, the conversion or the memory's
// latency the time stays the same.  The scales and the lines ahead on an idle warp: 74 -> 82 us below; the next
// tile's loads inside the store loop with all waits of the issuing warp ahead of P V: 74.5.  16 sequences of up to 60 nodes over up
// to 4096 tokens, 32 heads on 8, bf16: 71 us.  1 sequence of 64 nodes over 131072 tokens, 16 heads on 2: 73 us in
// bf16, 0.94 PFLOP/s, 97 in fp16 (1919 us uncut; pieces of half the share 30 % slower).
constexpr int kMinPieceTiles = 4;
// The most new tokens of a sequence: what some rows see and others do not has to fit kEdgeTokens.
constexpr int kMostTreeTokens = kEdgeTokens - kPromptKeys;

struct TreePiece {
  int b, h, rt, slot, t0, t1, pad[2];
};
// The workspace: [count of pieces, 3 unused], the pieces, per sequence {first slot, pieces of a unit},
// the parts (256 rows of D sums, then 256 log2 sums, fp32).
struct TreePlan {
  int32_t* count;
  TreePiece* pieces;
  int2* cuts;
  float* parts;
};
__host__ __device__ inline int64_t tree_plan_bytes(int64_t pieces, int64_t B) {
  return 16 + pieces * static_cast<int64_t>(sizeof(TreePiece)) + (B + 1) / 2 * 16;
}
__host__ __device__ inline TreePlan tree_plan(void* workspace, int64_t pieces, int64_t B) {
  TreePlan t;
  char* at = static_cast<char*>(workspace);
  t.count = reinterpret_cast<int32_t*>(at);
  t.pieces = reinterpret_cast<TreePiece*>(at + 16);
  t.cuts = reinterpret_cast<int2*>(at + 16 + pieces * static_cast<int64_t>(sizeof(TreePiece)));
  t.parts = reinterpret_cast<float*>(at + tree_plan_bytes(pieces, B));
  return t;
}

// The piece that CTA `i` works on; false where there are fewer.
__device__ __forceinline__ bool tree_unit(const AttendParams& p, const TreePlan& plan, int i, PromptUnit& u) {
  if (i >= *plan.count) return false;
  const TreePiece piece = plan.pieces[i];
  u.b = piece.b;
  u.h = piece.h;
  u.s = load_sequence(p.c, u.b, DK_PROMPT);
  u.row0 = piece.rt * kPromptRows;
  u.rows = u.s.n * p.group;
  u.start = u.s.len - u.s.n;
  u.kv_end = u.s.len;
  u.t0 = piece.t0;
  u.tiles = piece.t1 - piece.t0;
  u.slot = piece.slot;
  u.row_tiles = u.rows - u.row0 > 128 ? 2 : 1;
  return true;
}

// The (sequence, row tile) pair that a CTA works on.  CTAs start in the order of their numbers, and
// the most key tiles should start first.  Within a sequence that is the last row tile; over ragged
// sequences, while there are few pairs (with many, the last ones to finish weigh little), a small
// kernel ahead ranks the pairs by their key tiles.  (It is a kernel of its own because a pair read
// from global memory is known to be the same for the whole CTA; ranked inside, every size of the
// unit took a register per thread, and the spills cost more than the order gained.)
constexpr int kRankedPairs = 256;

__device__ __forceinline__ void plain_pair(const AttendParams& p, int row_tiles, int order, int& b,
                                           int& rt) {
  b = order % p.c.B;
  rt = row_tiles - 1 - order / p.c.B;
}

// ------------------------------------------------------------------------------------
// producers: 128 tokens of a page walk as fp16 tiles [D / 64][token][64 channels], 128B swizzle
// ------------------------------------------------------------------------------------
template <int D>
struct PromptProducer {
  static constexpr int kPieces = D / 16;              // 16-byte runs of codes per token
  static constexpr int kLanes = kPieces > 4 ? 8 : 4;  // threads per token
  static constexpr int kTokens = 128 / kLanes;        // tokens of the warpgroup's one load
  static constexpr int kEach = kLanes;                // loads per thread and tile
  uint32_t tid;
  int page;                                           // number of granule lane & 7's page, next tile
  int later;                                          // trees: of the tile behind it

  // The thread's run in load j: token j kTokens + tid / kLanes.  A load's tokens lie in one 16-token
  // granule (two with kTokens = 32, one per half of the warpgroup), and so in one page.
  __device__ __forceinline__ int token(int j) const { return j * kTokens + tid / kLanes; }
  __device__ __forceinline__ uint32_t piece() const { return tid % kLanes; }
  __device__ __forceinline__ int granule(int j) const {
    return kLanes == 8 ? j : 2 * j + static_cast<int>(tid >> 6);
  }

  // Reads the page numbers of a tile (used a tile later, so that nothing waits for them).
  __device__ __forceinline__ void locate(const AttendParams& p, const PromptUnit& u, int tile) {
    const int at = tile * kPromptKeys + static_cast<int>(tid & 7) * kGranule;
    page = at < u.kv_end ? p.c.page_table[static_cast<int64_t>(u.b) * p.c.max_pages +
                                          (at >> p.c.page_shift)]
                         : 0;
  }
  // The same two tiles ahead; its codes are asked for into L2 by `ahead`.
  __device__ __forceinline__ void locate_later(const AttendParams& p, const PromptUnit& u, int tile) {
    const int at = tile * kPromptKeys + static_cast<int>(tid & 7) * kGranule;
    later = at < u.kv_end ? p.c.page_table[static_cast<int64_t>(u.b) * p.c.max_pages +
                                           (at >> p.c.page_shift)]
                          : -1;
  }
  // Asks for the codes of `tile`, a 128-byte line per thread, and moves on by a tile.
  __device__ __forceinline__ void ahead(const AttendParams& p, const PromptUnit& u, int tile, const uint8_t* pool) {
    constexpr int kLines = D * kGranule / 128;
    const CacheView& c = p.c;
    const int g = static_cast<int>(tid) / kLines, line = static_cast<int>(tid) % kLines;
    const int id = __shfl_sync(0xffffffffu, later, g & 7);
    if (g < kGranules && static_cast<uint32_t>(id) < static_cast<uint32_t>(c.pages)) {
      const int slot = (tile * kPromptKeys + g * kGranule) & ((1 << c.page_shift) - 1);
      const uint8_t* at = pool + (((static_cast<int64_t>(id) * c.heads + u.h) << c.page_shift) + slot) * D + line * 128;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
    }
    page = later;
    locate_later(p, u, tile + 1);
  }
  // Starts the loads of this thread's runs of the located tile.  A number outside the pool is
  // replaced (it is recorded with the scales, which become NaN); slots at or past kv_end are read
  // as they are.
  __device__ __forceinline__ void fetch(const AttendParams& p, const PromptUnit& u, int tile,
                                        const uint8_t* pool, uint4 (&raw)[kEach]) const {
    const CacheView& c = p.c;
    const int mask = (1 << c.page_shift) - 1;
    const int64_t page_bytes = (static_cast<int64_t>(c.heads) << c.page_shift) * D;
    const uint32_t run = piece() < kPieces ? piece() : 0;
    const uint8_t* head = pool + ((static_cast<int64_t>(u.h) << c.page_shift) * D) +
                          static_cast<int>(tid / kLanes % kGranule) * D + 16 * run;
    const int id = static_cast<uint32_t>(page) < static_cast<uint32_t>(c.pages) ? page : 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int g = granule(j);
      const int slot = (tile * kPromptKeys + g * kGranule) & mask;
      raw[j] = *reinterpret_cast<const uint4*>(
          head + __shfl_sync(0xffffffffu, id, g) * page_bytes + slot * D);
    }
  }
  // A run is two 16-byte units of a row.  Runs of the second 64 channels store theirs in the other
  // order, so that the eight lanes of a token fill eight different units at a time.
  __device__ __forceinline__ void store(const uint4 (&raw)[kEach], uint32_t tile_at) const {
    const bool flip = piece() >= 4;
    const uint32_t unit = ((piece() % 4) * 2 + (flip ? 1 : 0)) ^ (token(0) & 7);
    const uint32_t row = tile_at + (piece() / 4) * 16384 + token(0) * 128;
    if (piece() >= kPieces) return;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const uint32_t w0 = flip ? raw[j].z : raw[j].x, w1 = flip ? raw[j].w : raw[j].y;
      const uint32_t w2 = flip ? raw[j].x : raw[j].z, w3 = flip ? raw[j].y : raw[j].w;
      uint32_t h[4];
      e4m3x4_to_f16(w0, h[0], h[1]);
      e4m3x4_to_f16(w1, h[2], h[3]);
      st_shared16(row + j * (kTokens * 128) + (unit << 4), h[0], h[1], h[2], h[3]);
      e4m3x4_to_f16(w2, h[0], h[1]);
      e4m3x4_to_f16(w3, h[2], h[3]);
      st_shared16(row + j * (kTokens * 128) + ((unit ^ 1u) << 4), h[0], h[1], h[2], h[3]);
    }
  }
};

// A warp's 32 query rows of a drafted tree (r0 .. r0 + 31 of `rows`) as fp16 at q_at + 128 row_in .., and
// each thread's mask: a piece of a tree's unit is short, so its rows come whole (D / 8 lanes each) and
// all at once, straight to where the products want them; then each thread turns its row there.  Returns the
// power of two that goes back into its scores.  (Loads by a thread per row, 16 in registers: 8.5 us of a
// piece's 30; by whole rows, 16 times unrolled: 5.5, mostly instructions that are not in the cache yet.  A
// function of its own, since inlined it cost the loops registers.)
template <int D>
__device__ __forceinline__ float stage_tree_rows(const uint16_t* q, const uint16_t* any, int64_t ldq, int group, int r0,
                                              int rows, uint32_t q_at, int row_in, const uint32_t* mask,
                                              uint32_t* mask_to, int words, int is_bf16, bool negative) {
  constexpr int kPer = D / 8, kRows = 32 / kPer;
  const int lane = threadIdx.x & 31, sub = lane / kPer, at = lane % kPer;
  {
    int r = r0 + sub, tok = r / group, in_tok = r - tok * group;
#pragma unroll 1
    for (int k = sub; k < 32; k += kRows, r += kRows) {
      const int in = row_in + k;
      const bool take = sub < kRows && r < rows;
      const uint16_t* from = q + tok * ldq + in_tok * D + 8 * at;
      const int bytes = take ? 16 : 0;               // 0: zeros
      if (sub < kRows)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         q_at + in * 128 + (at / 8) * 16384 + (((at % 8) ^ (in & 7)) << 4)),
                     "l"(take ? from : any), "r"(bytes)
                     : "memory");
      in_tok += kRows;
      while (in_tok >= group) {
        in_tok -= group;
        ++tok;
      }
    }
  }
  for (int i = 0; i < words; i += 4) {
    uint32_t word[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) word[k] = i + k < words ? mask[i + k] : 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) mask_to[(i + k) * kPromptRows] = word[k];
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  float unit = 1.f, inv = 1.f;
  if (!is_bf16 && !negative) return unit;
  const int mine = row_in + lane;
  auto place = [&](int i) -> uint32_t {
    return q_at + mine * 128 + (i / 8) * 16384 + (((i % 8) ^ (mine & 7)) << 4);
  };
  auto load = [&](int i) -> uint4 {
    const float4 v = ld_shared_f4(place(i));
    return make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
  };
  if (is_bf16) {
    // the largest magnitude: 16-bit patterns without their signs order like it
    uint32_t most = 0u;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
      const uint4 w = load(i);
      most = __vmaxu2(most, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                     __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
    }
    const uint32_t hi = most & 0xFFFF0000u, lo = most << 16;
    unit = row_unit<true>(__uint_as_float(hi > lo ? hi : lo), inv);
  }
  if (negative) inv = -inv;                          // the softmax's maximum wants positive factors
#pragma unroll 2
  for (int i = 0; i < D / 8; ++i) {
    uint4 w = load(i);
    if (is_bf16) {
      float f[8];
      widen8<true>(w, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= inv;
      w = narrow8<false>(f);
    } else {
      w.x ^= 0x80008000u;
      w.y ^= 0x80008000u;
      w.z ^= 0x80008000u;
      w.w ^= 0x80008000u;
    }
    st_shared16(place(i), w.x, w.y, w.z, w.w);
  }
  return unit;
}

// KIND: prompts, or drafted trees, their units whole (kTreeWhole) or cut in pieces.  LO (fp16 outputs of
// trees): P V is formed of P and of what its rounding to fp16 leaves, so that only the output's own rounding
// is left (error of 64 nodes over 131072 tokens against 64 bits 3.2e-4 without, 2.1e-4 with it).
enum PromptKind { kCausal, kTreeWhole, kTreeCut };
template <int D, bool MODS, PromptKind KIND, bool LO>
__global__ void __launch_bounds__(kPromptThreads, 1) prompt_kernel(const AttendParams p,
                                                                   int row_tiles) {
  using L = PromptSmem<D>;
  constexpr bool TREE = KIND != kCausal, CUT = KIND == kTreeCut;
  extern __shared__ uint8_t raw_smem[];
  const uint32_t base = (smem_u32(raw_smem) + 1023u) & ~1023u;
  uint8_t* smem = raw_smem + (base - smem_u32(raw_smem));
  PromptBars* bars = reinterpret_cast<PromptBars*>(smem + L::kBar);
  float2* scales = reinterpret_cast<float2*>(smem + L::kScales);
  uint32_t* nan_bits = reinterpret_cast<uint32_t*>(smem + L::kNan);
  [[maybe_unused]] uint32_t* masks = reinterpret_cast<uint32_t*>(smem + L::kMasks);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  PromptUnit u;
  {
    int b, rt;
    int order = static_cast<int>(blockIdx.x) / p.c.heads;
    grid_launch_dependents();
    grid_dependency_wait();                                // launched early
    if constexpr (CUT) {
      const TreePlan plan = tree_plan(p.meta, gridDim.x, p.c.B);
      if (!tree_unit(p, plan, static_cast<int>(blockIdx.x), u)) return;                // the whole CTA
    } else {
      if (p.meta != nullptr) {
        order = static_cast<int>(p.meta[order]);
      }
      plain_pair(p, row_tiles, order, b, rt);
      if (!prompt_unit(p, b, static_cast<int>(blockIdx.x) % p.c.heads, rt, u)) return; // the whole CTA
      if constexpr (TREE) {                                // every row may see every new token
        u.kv_end = u.s.len;
        u.tiles = (u.kv_end + kPromptKeys - 1) / kPromptKeys;
      }
    }
  }
  const int first_tile = CUT ? u.t0 : 0;
  // One row tile: both softmaxes work on it, on every other key tile each, and are merged at the end.  A softmax
  // that has only seen pages of no value has its sum in units of 2^-96 or less, and so its weight.
  const bool pairs = TREE && u.row_tiles == 1 && u.tiles > 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->qfull[i]), 4);
      mbar_init(smem_u32(&bars->kfull[i]), 4);
      mbar_init(smem_u32(&bars->kempty[i]), 1);
      mbar_init(smem_u32(&bars->vfull[i]), 4);
      mbar_init(smem_u32(&bars->vempty[i]), 1);
      mbar_init(smem_u32(&bars->sfull[i]), 1);
      mbar_init(smem_u32(&bars->pready[i]), 4);
      mbar_init(smem_u32(&bars->ofull[i]), 1);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    mbar_init(smem_u32(&bars->merge), 4);
    bars->abort_flag = 0u;
    bars->nan_any = 0u;
    fence_barrier_init();
  }
  for (int i = threadIdx.x; i < kEdgeTokens * (D / 32); i += kPromptThreads) nan_bits[i] = 0u;
  if (warp == 16) {
    tmem_alloc(smem_u32(&bars->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem;
  volatile uint32_t* abort_flag = &bars->abort_flag;
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
    // one answer for the warp, also when it gives up: what follows is warp-wide
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.wait_limit_ns, abort_flag,
                                             p.c.err, DK_PROMPT, site, blockIdx.x));
  };
  // first token that some row of the CTA does not see, down to its tile
  const int edge0 = (TREE ? u.start : u.start + u.row0 / p.group + 1) / kPromptKeys * kPromptKeys;

  if (warp < 8) {
    more_registers<kSoftmaxRegs>();
    // ================= softmax =================
    const int t = warp >> 2;
    const int tile_row = u.row0 + (pairs ? 0 : 128 * t);
    const int row = tile_row + (threadIdx.x & 127);
    const bool valid = row < u.rows;
    if (t < u.row_tiles || pairs) {
      const uint32_t tm = tmem + ((warp & 3) << 21);          // this warp's 32 lanes
      const uint32_t s_col = 256u * t, o_col = 256u * t + 128u;
      const int tq = valid ? row / p.group : 0;
      const int head = u.h * p.group + (valid ? row - tq * p.group : 0);
      // ---- Q: this thread's row as fp16, 128B-swizzled ----
      float fac;
      {
        const uint16_t* src = p.q + (u.s.row + static_cast<int64_t>(tq)) * p.ldq +
                              static_cast<int64_t>(head) * D;
        float inv = 1.f, unit = 1.f;
        if constexpr (TREE) {
          const int64_t first_row = u.s.row;
          unit = stage_tree_rows<D>(p.q + first_row * p.ldq + static_cast<int64_t>(u.h * p.group) * D, p.q, p.ldq, p.group,
                                    tile_row + (warp & 3) * 32, u.rows, base + L::kQ + t * L::kTile,
                                    (threadIdx.x & 127) - lane, p.masks + (first_row + tq) * p.mask_words,
                                    masks + (threadIdx.x & 255), (u.s.n + 31) / 32, p.is_bf16, p.scale < 0.f);
        } else {
          if (p.is_bf16) {
            float amax = 0.f;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
              uint4 w = make_uint4(0u, 0u, 0u, 0u);
              if (valid) w = reinterpret_cast<const uint4*>(src)[i];
              float f[8];
              widen8<true>(w, f);
#pragma unroll
              for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
            }
            unit = row_unit<true>(amax, inv);
          }
          if (p.scale < 0.f) inv = -inv;           // the maximum below wants positive factors
          const uint32_t dst = base + L::kQ + t * L::kTile + (threadIdx.x & 127) * 128;
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (valid) w = reinterpret_cast<const uint4*>(src)[i];
            if (p.is_bf16) {
              float f[8];
              widen8<true>(w, f);
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] *= inv;
              w = narrow8<false>(f);
            } else if (p.scale < 0.f) {
              w.x ^= 0x80008000u;
              w.y ^= 0x80008000u;
              w.z ^= 0x80008000u;
              w.w ^= 0x80008000u;
            }
            st_shared16(dst + (i / 8) * 16384 + (((i % 8) ^ (threadIdx.x & 7)) << 4), w.x, w.y, w.z, w.w);
          }
        }
        fac = unit * fabsf(p.scale) * (MODS ? 1.f : kLog2e);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->qfull[t]));

      // the last token that the row sees; of a tree's, the position for the distance bias
      int limit = valid ? u.start + tq : 0x7FFFFFFF;
      if (TREE && MODS && p.positions != nullptr)
        limit = p.positions[u.s.row + static_cast<int64_t>(tq)];
      const int low_limit = TREE ? u.start - 1 : u.start + (u.row0 + 128 * t) / p.group;
      // which of the 16 tokens from `tok` on the row sees (its thread has put its mask there)
      auto window = [&](int tok) -> uint32_t {
        const int off = tok - u.start;
        if (off <= -kGranule) return 0xFFFFu;
        return off < u.s.n ? tree_window(masks + (threadIdx.x & 255), kPromptRows, (kEdgeTokens - kPromptKeys) / 32, off, u.s.n) : 0u;
      };
      const float slope = MODS && p.slopes != nullptr && valid ? p.slopes[head] : 0.f;
      float m = -1e30f, l = 0.f;                   // m: the reference of z + log2 value scale
      bool ok = true;

      const int first = pairs ? t : 0;
      const bool idle = TREE && tile_row + 32 * (warp & 3) >= u.rows;      // no rows
      for (int i = first; i < u.tiles && ok; i += pairs ? 2 : 1) {
        const float2* sc = scales + (i & 3) * kGranules;
        const int tok0 = (first_tile + i) * kPromptKeys;
        const bool edge = tok0 + kPromptKeys - 1 > low_limit;
        ok = wait(&bars->sfull[t], (pairs ? i >> 1 : i) & 1, PS_SFULL);
        if (!ok) break;
        if (idle) {                                // whatever P is: it stays in its row
          if (lane == 0) mbar_arrive(smem_u32(&bars->pready[t]));
          continue;
        }
        tc_fence_after_sync();
        // the reference, and what O and the row's sum have to be scaled by for it
        auto move_reference = [&](float top, uint32_t (&r)[32]) -> float {
          float f = 1.f;
          if (top > m + 15.f) {
            f = exp2_fast(m - (top - 7.f));
            m = top - 7.f;
            l *= f;
          }
          if (i > first && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              tmem_load32(tm + o_col + 32 * q, r);
              tmem_wait32(r);
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
              tmem_st32(tm + o_col + 32 * q, r);
            }
          }
          return f;
        };
        // a score in the log2 domain
        auto score = [&](uint32_t raw, float f, int tok) -> float {
          float z = __uint_as_float(raw) * f;
          if (MODS) {
            if (p.softcap > 0.f) z = capped(z, p.softcap, p.inv_softcap);
            int at = tok;
            if (TREE && edge && p.positions != nullptr && tok >= u.start && tok < u.kv_end)
              at = p.positions[u.s.row + static_cast<int64_t>(tok - u.start)];
            z = fmaf(slope, static_cast<float>(at - limit), z) * kLog2e;
          }
          return z;
        };
        // LO: 64 keys at a time, whose P and rest (32 columns each) take the place of their scores.  As
        // below, inner tiles take one pass and a second two only if some exponent turns out above 15; where
        // the reference then moves for the second 64 keys, the first ones' P and rest are scaled too.
        [[maybe_unused]] auto half_with_rest = [&](auto half, auto scores) {
          constexpr int kHalf = decltype(half)::value, kFirst = 4 * kHalf;
          constexpr bool SCORES = decltype(scores)::value;
          const uint32_t at = tm + s_col + 64 * kHalf;
          uint32_t r[2][16], hi[32], lo[32];
          // P, its rest and the sums; false, and nothing done, where an exponent is above 15 and that was not
          // ruled out before
          auto take = [&](auto masked, bool ruled_out) -> bool {
            constexpr bool MASKED = decltype(masked)::value;
            float high = -INFINITY, more = 0.f;
            tmem_ld16(at, r[0]);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              tmem_wait_ld(r[g & 1]);
              if (g + 1 < 4) tmem_ld16(at + 16 * (g + 1), r[(g + 1) & 1]);
              const float2 s2 = sc[kFirst + g];
              const float fg = MASKED ? 1.f : fac * s2.x;
              // (a page that the row does not reach may have any scale, a NaN too)
              const bool past = MASKED && window(tok0 + 16 * (kFirst + g)) == 0u;
              const float back = past ? 0.f : exp2_fast(-s2.y), c = past ? 0.f : s2.y - m;
              const float2 f2 = make_float2(fg, fg), c2 = make_float2(c, c);
              float2 sum = make_float2(0.f, 0.f);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                const uint32_t* x = &r[g & 1][e];
                float2 y = fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), f2, c2);
                high = max3(high, y.x, y.y);
                y.x = exp2_fast(y.x);
                y.y = exp2_fast(y.y);
                sum = add2(sum, y);
                const uint32_t h = narrow2<false>(y.x, y.y);
                const float2 kept = widen2<false>(h);
                hi[8 * g + e / 2] = h;
                lo[8 * g + e / 2] = narrow2<false>(y.x - kept.x, y.y - kept.y);
              }
              more = fmaf(sum.x + sum.y, back, more);
            }
            if (!ruled_out && __any_sync(0xffffffffu, high > 15.f)) return false;
            l += more;
            tmem_st32(at, hi);
            tmem_st32(at + 32, lo);
            return true;
          };
          if (!SCORES && __all_sync(0xffffffffu, m > -1e29f) && take(std::false_type{}, false)) return;
          // ---- the largest z + log2 value scale; capped, biased or masked scores go back to TMEM ----
          float top = -INFINITY;
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {
            uint32_t (&x)[16] = r[0];
            tmem_ld16(at + 16 * g, x);
            tmem_wait_ld(x);
            const float2 s2 = sc[kFirst + g];
            const float f = fac * s2.x;
            float most = -INFINITY;                  // of the granule's tokens that the row sees
            if constexpr (SCORES) {
              const uint32_t sees = window(tok0 + 16 * (kFirst + g));
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float z =
                    ((sees >> e) & 1u) == 0u ? -INFINITY : score(x[e], f, tok0 + 16 * (kFirst + g) + e);
                x[e] = __float_as_uint(z);
                most = fmaxf(most, z);
              }
              tmem_store16(at + 16 * g, x);
            } else {
              float a = __uint_as_float(x[0]);
#pragma unroll
              for (int e = 1; e + 1 < 16; e += 2) a = max3(a, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
              most = fmaxf(a, __uint_as_float(x[15])) * f;
            }
            top = fmaxf(top, most + s2.y);
          }
          // (also for what the first half has stored: its P and rest, and O where the reference moved there)
          if constexpr (SCORES || kHalf == 1) tmem_wait_st();
          const float f = move_reference(top, hi);
          if (kHalf == 1 && __any_sync(0xffffffffu, f != 1.f)) {
            tmem_load32(tm + s_col, hi);
            tmem_wait32(hi);
            tmem_load32(tm + s_col + 32, lo);
            tmem_wait32(lo);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float2 a = widen2<false>(hi[e]), b = widen2<false>(lo[e]);
              const float x = (a.x + b.x) * f, y = (a.y + b.y) * f;
              hi[e] = narrow2<false>(x, y);
              const float2 kept = widen2<false>(hi[e]);
              lo[e] = narrow2<false>(x - kept.x, y - kept.y);
            }
            tmem_st32(tm + s_col, hi);
            tmem_st32(tm + s_col + 32, lo);
            tmem_wait_st();
          }
          (void)take(std::integral_constant<bool, SCORES>{}, true);
        };
        [[maybe_unused]] auto tile_with_rest = [&](auto scores) {
          half_with_rest(std::integral_constant<int, 0>{}, scores);
          half_with_rest(std::integral_constant<int, 1>{}, scores);
        };
        auto tile = [&](auto scores) {
        constexpr bool SCORES = decltype(scores)::value;
        // ---- the tile's largest z + log2 value scale; capped, biased or masked scores go back to TMEM ----
        uint32_t r[32];
        float top = -INFINITY;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          tmem_load32(tm + s_col + 32 * q, r);
          tmem_wait32(r);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float2 s2 = sc[2 * q + g];
            const float f = fac * s2.x;
            uint32_t* x = &r[16 * g];
            float most = -INFINITY;                  // of the granule's tokens that the row sees
            if constexpr (SCORES) {
              const uint32_t sees = TREE ? window(tok0 + 32 * q + 16 * g) : 0u;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int tok = tok0 + 32 * q + 16 * g + e;
                const bool hidden = TREE ? ((sees >> e) & 1u) == 0u : tok > limit;
                const float z = hidden ? -INFINITY : score(x[e], f, tok);
                x[e] = __float_as_uint(z);
                most = fmaxf(most, z);
              }
            } else {
              float a = __uint_as_float(x[0]);
#pragma unroll
              for (int e = 1; e + 1 < 16; e += 2)
                a = max3(a, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
              most = fmaxf(a, __uint_as_float(x[15])) * f;
            }
            top = fmaxf(top, most + s2.y);
          }
          if constexpr (SCORES) tmem_st32(tm + s_col + 32 * q, r);
        }
        if constexpr (SCORES) tmem_wait_st();
        (void)move_reference(top, r);
        // ---- P, and the row's sum ----
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          tmem_load32(tm + s_col + 32 * q, r);
          tmem_wait32(r);
          uint32_t pk[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float2 s2 = sc[2 * q + g];
            const float fg = SCORES ? 1.f : fac * s2.x;
            // (a page that the row does not reach may have any scale, a NaN too)
            const bool past = SCORES && (TREE ? window(tok0 + 32 * q + 16 * g) == 0u
                                              : tok0 + 32 * q + 16 * g > limit);
            const float back = past ? 0.f : exp2_fast(-s2.y), c = past ? 0.f : s2.y - m;
            const float2 f2 = make_float2(fg, fg), c2 = make_float2(c, c);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float2 y = fma2(make_float2(__uint_as_float(r[16 * g + e]),
                                          __uint_as_float(r[16 * g + e + 1])), f2, c2);
              y.x = exp2_fast(y.x);
              y.y = exp2_fast(y.y);
              sum = add2(sum, y);
              pk[8 * g + e / 2] = narrow2<false>(y.x, y.y);
            }
            l = fmaf(sum.x + sum.y, back, l);
          }
          tmem_store16(tm + s_col + 16 * q, pk);
        }
        };
        // Inner tiles of a plain softmax take one pass with the reference as it is: P and the sums are
        // formed while the columns arrive, and only if some exponent turns out above 15 is the tile
        // done again in two passes.
        bool done = false;
        if constexpr (LO) {
          if (MODS || edge) tile_with_rest(std::true_type{});
          else tile_with_rest(std::false_type{});
          done = true;
        }
        if (!LO && !MODS && !edge && __all_sync(0xffffffffu, m > -1e29f)) {
          uint32_t r[2][16], pk[4][16];
          float high = -INFINITY, more = 0.f;
          tmem_ld16(tm + s_col, r[0]);
#pragma unroll
          for (int g = 0; g < kGranules; ++g) {
            tmem_wait_ld(r[g & 1]);
            if (g + 1 < kGranules) tmem_ld16(tm + s_col + 16 * (g + 1), r[(g + 1) & 1]);
            const float2 s2 = sc[g];
            const float fg = fac * s2.x, back = exp2_fast(-s2.y), c = s2.y - m;
            const float2 f2 = make_float2(fg, fg), c2 = make_float2(c, c);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const uint32_t* x = &r[g & 1][e];
              float2 y = fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), f2, c2);
              high = max3(high, y.x, y.y);
              y.x = exp2_fast(y.x);
              y.y = exp2_fast(y.y);
              sum = add2(sum, y);
              pk[g / 2][8 * (g & 1) + e / 2] = narrow2<false>(y.x, y.y);
            }
            more = fmaf(sum.x + sum.y, back, more);
          }
          if (!__any_sync(0xffffffffu, high > 15.f)) {
            l += more;
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_store16(tm + s_col + 16 * q, pk[q]);
            done = true;
          }
        }
        if constexpr (!LO) {
          if (!done) {
            if (MODS || edge) tile(std::true_type{});
            else tile(std::false_type{});
          }
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->pready[t]));
      }

      // ---- the output row ----
      ok = ok && wait(&bars->ofull[t], 0, PS_OFULL);
      if (ok) tc_fence_after_sync();
      // (all products with Q and K have been issued before the last P V of either softmax)
      const uint32_t merge_at = base + L::kK + (warp & 3) * (32 * D * 4) + lane * (D * 4);
      if (pairs && t == 1) {
        if (ok) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t r[32];
            tmem_load32(tm + o_col + 32 * q, r);
            tmem_wait32(r);
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              st_shared16(merge_at + (((8 * q + e / 4) ^ (lane & 7)) << 4), r[e], r[e + 1], r[e + 2], r[e + 3]);
          }
          masks[threadIdx.x & 255] = __float_as_uint(m);
          masks[kPromptRows + (threadIdx.x & 255)] = __float_as_uint(l);
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->merge));
        }
      } else if (ok && (!pairs || wait(&bars->merge, 0, PS_MERGE))) {
        float mine = 1.f, other = 0.f;             // what the sums of the two are multiplied by
        bool seen = true, other_seen = false;
        if (pairs) {
          const float m1 = __uint_as_float(masks[128 + threadIdx.x]);
          const float l1 = __uint_as_float(masks[kPromptRows + 128 + threadIdx.x]);
          seen = l != 0.f;
          other_seen = l1 != 0.f;
          const float top = fmaxf(m, m1);
          mine = exp2_fast(m - top);
          other = exp2_fast(m1 - top);
          l = (seen ? mine * l : 0.f) + (other_seen ? other * l1 : 0.f);
          m = top;
        }
        const float inv = l == 0.f || l > kNoValues ? 0.f : 1.f / l;
        mine *= inv;
        other *= inv;
        float* part = nullptr;
        if (CUT && u.slot >= 0) {
          part = tree_plan(p.meta, gridDim.x, p.c.B).parts +
                 static_cast<int64_t>(u.slot) * (kPromptRows * (D + 1));
          if (valid) part[kPromptRows * D + row - u.row0] = l == 0.f ? -1e30f : m + log2f(l);
        }
        // (trees: staged in shared memory that the products no longer read, and stored by rows)
        const uint32_t stage = base + (t == 0 ? L::kQ : L::kK) + (warp & 3) * (32 * D * 4);
        const int tq_out = valid ? tq : 0;
        uint16_t* dst = p.out + ((u.s.row + static_cast<int64_t>(tq_out)) * p.q_heads + head) * D;
        const bool nans = bars->nan_any != 0u;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t r[32];
          tmem_load32(tm + o_col + 32 * q, r);
          tmem_wait32(r);
          uint32_t bad = 0u;
          if (nans) {
            for (int tok = edge0; (TREE || tok <= limit) && tok < u.kv_end; ++tok) {
              if (TREE && tok >= u.start && (window(tok) & 1u) == 0u) continue;
              bad |= nan_bits[(tok - edge0) * (D / 32) + q];
            }
          }
          if (TREE || valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              float o[8], more[8];
              if (pairs) {
                const int chunk = 8 * q + e / 4;
                const float4 a = ld_shared_f4(merge_at + ((chunk ^ (lane & 7)) << 4));
                const float4 z = ld_shared_f4(merge_at + (((chunk + 1) ^ (lane & 7)) << 4));
                more[0] = a.x, more[1] = a.y, more[2] = a.z, more[3] = a.w;
                more[4] = z.x, more[5] = z.y, more[6] = z.z, more[7] = z.w;
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                o[k] = inv == 0.f || !seen ? 0.f : __uint_as_float(r[e + k]) * mine;
                if (pairs && other_seen && inv != 0.f) o[k] = fmaf(more[k], other, o[k]);
                if ((bad >> (e + k)) & 1u) o[k] = __uint_as_float(0x7FC00000u);
              }
              if constexpr (TREE) {
                const int chunk = 8 * q + e / 4;               // 16-byte units of the row, xor-ed by it
                st_shared16(stage + lane * (D * 4) + ((chunk ^ (lane & 7)) << 4), __float_as_uint(o[0]),
                            __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3]));
                st_shared16(stage + lane * (D * 4) + (((chunk + 1) ^ (lane & 7)) << 4), __float_as_uint(o[4]),
                            __float_as_uint(o[5]), __float_as_uint(o[6]), __float_as_uint(o[7]));
              } else {
                *reinterpret_cast<uint4*>(dst + 32 * q + e) = p.is_bf16 ? narrow8<true>(o) : narrow8<false>(o);
              }
            }
          }
        }
        if constexpr (TREE) {
          __syncwarp();
          const int first = row - lane;                        // the warp's first row
          if (CUT && part != nullptr) {
            for (int i = lane; i < 32 * D / 4; i += 32) {
              const int r = i / (D / 4), chunk = i % (D / 4);
              if (first + r >= u.rows) break;
              const float4 v = ld_shared_f4(stage + r * (D * 4) + ((chunk ^ (r & 7)) << 4));
              *reinterpret_cast<float4*>(part + static_cast<int64_t>(first + r - u.row0) * D + 4 * chunk) = v;
            }
          } else {
            for (int i = lane; i < 32 * D / 8; i += 32) {
              const int r = i / (D / 8), chunk = 2 * (i % (D / 8)), at = first + r;
              if (at >= u.rows) break;
              const float4 a = ld_shared_f4(stage + r * (D * 4) + ((chunk ^ (r & 7)) << 4));
              const float4 z = ld_shared_f4(stage + r * (D * 4) + (((chunk + 1) ^ (r & 7)) << 4));
              const float o[8] = {a.x, a.y, a.z, a.w, z.x, z.y, z.z, z.w};
              const int tok = at / p.group, mine = u.h * p.group + (at - tok * p.group);
              *reinterpret_cast<uint4*>(p.out + ((u.s.row + static_cast<int64_t>(tok)) * p.q_heads + mine) * D +
                                        4 * chunk) = p.is_bf16 ? narrow8<true>(o) : narrow8<false>(o);
            }
          }
        }
      }
    }
  } else if (warp < 12) {
    fewer_registers<kProducerRegs>();
    // ================= keys, and the scales of both pools =================
    PromptProducer<D> prod;
    prod.tid = threadIdx.x - 256;
    uint4 raw[PromptProducer<D>::kEach];
    // thread g < kGranules: the scales of granule g, whose page number it has
    auto scales_of = [&](int tile, int id) -> float2 {
      if (prod.tid >= kGranules ||
          tile * kPromptKeys + static_cast<int>(prod.tid) * kGranule >= u.kv_end)
        return make_float2(0.f, 0.f);
      if (id < 0 || id >= p.c.pages) {
        index_error(p.c.err, DK_PROMPT, DEC_ERR_PAGE, static_cast<uint32_t>(u.b));
        return make_float2(__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u));
      }
      const int64_t at = static_cast<int64_t>(id) * p.c.heads + u.h;
      return make_float2(p.c.k_scale[at], p.c.v_scale[at]);
    };
    prod.locate(p, u, first_tile);
    prod.fetch(p, u, first_tile, p.c.k, raw);
    float2 s2 = scales_of(first_tile, prod.page);
    prod.locate(p, u, first_tile + 1);
    if constexpr (TREE) prod.locate_later(p, u, first_tile + 2);
    bool ok = true;
    for (int i = 0; i < u.tiles && ok; ++i) {
      const int slot = i & 1;
      if (i >= 2) ok = wait(&bars->kempty[slot], ((i >> 1) - 1) & 1, PS_KEMPTY);
      if (!ok) break;
      prod.store(raw, base + L::kK + slot * L::kTile);
      if (prod.tid < kGranules) scales[(i & 3) * kGranules + prod.tid] = make_float2(s2.x, exponent_of(s2.y));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->kfull[slot]));
      if (i + 1 < u.tiles) {
        prod.fetch(p, u, first_tile + i + 1, p.c.k, raw);
        s2 = scales_of(first_tile + i + 1, prod.page);
        if constexpr (TREE) prod.ahead(p, u, first_tile + i + 2, p.c.k);
        else prod.locate(p, u, first_tile + i + 2);
      }
    }
  } else if (warp < 16) {
    fewer_registers<kProducerRegs>();
    // ================= values =================
    PromptProducer<D> prod;
    prod.tid = threadIdx.x - 384;
    constexpr int kEach = PromptProducer<D>::kEach;
    uint4 raw[kEach];
    prod.locate(p, u, first_tile);
    prod.fetch(p, u, first_tile, p.c.v, raw);
    prod.locate(p, u, first_tile + 1);
    if constexpr (TREE) prod.locate_later(p, u, first_tile + 2);
    bool ok = true;
    for (int i = 0; i < u.tiles && ok; ++i) {
      const int slot = i & 1;
      if (i >= 2) ok = wait(&bars->vempty[slot], ((i >> 1) - 1) & 1, PS_VEMPTY);
      if (!ok) break;
      const int tile = first_tile + i;
      if (tile * kPromptKeys >= edge0) {
        // Slots past every row's reach may hold anything: taken as zeros.  A NaN that only some rows
        // see comes out of the product too (0 * NaN is one) and is noted for the rows that see it.
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          if (tile * kPromptKeys + prod.token(j) >= u.kv_end) raw[j] = make_uint4(0u, 0u, 0u, 0u);
          uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
          uint32_t any = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e) any |= ((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          if (any != 0u) {
            uint32_t bits = 0u;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (((w[e / 4] >> (8 * (e % 4))) & 0x7Fu) == 0x7Fu) {
                bits |= 1u << e;
                w[e / 4] &= ~(0xFFu << (8 * (e % 4)));
              }
            raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
            const int at = tile * kPromptKeys + prod.token(j);
            if (at - edge0 < kEdgeTokens && prod.piece() < PromptProducer<D>::kPieces) {
              atomicOr(&nan_bits[(at - edge0) * (D / 32) + prod.piece() / 2],
                       bits << (16 * (prod.piece() & 1)));
              bars->nan_any = 1u;
            }
          }
        }
      }
      prod.store(raw, base + L::kV + slot * L::kTile);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->vfull[slot]));
      if (i + 1 < u.tiles) {
        prod.fetch(p, u, first_tile + i + 1, p.c.v, raw);
        if constexpr (TREE) prod.ahead(p, u, first_tile + i + 2, p.c.v);
        else prod.locate(p, u, first_tile + i + 2);
      }
    }
  } else {
    fewer_registers<kIssueRegs>();
  }
  if (warp == 16) {
    // ================= MMA =================
    // One issuer for both row tiles: P V and the next Q K^T of a tile stay together in the tensor
    // core's queue, which keeps the two tiles' softmaxes out of step (two issuers mix the tiles'
    // products, and both tiles then wait for both).
    const uint32_t lead = elect_one();
    const uint32_t idesc_s = idesc_f16_f32(0u, 0u, 128, kPromptKeys);
    const uint32_t idesc_o = idesc_f16_f32(0u, 1u, 128, D);
    const uint64_t q_desc = sdesc_sw128(base + L::kQ, 16u, 1024u);
    const uint64_t k_desc = sdesc_sw128(base + L::kK, 16u, 1024u);
    const uint64_t v_desc = sdesc_sw128(base + L::kV, 16384u, 1024u);
    auto issue_s = [&](int t, int slot) {
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint64_t step = static_cast<uint64_t>((ks / 4) * (16384 >> 4) + (ks % 4) * 2);
        mma_f16_ss(lead, tmem + 256u * t, q_desc + t * (L::kTile >> 4) + step,
                   k_desc + slot * (L::kTile >> 4) + step, idesc_s, ks == 0 ? 0u : 1u);
      }
      mma_commit(lead, smem_u32(&bars->sfull[t]));
    };
    auto issue_o = [&](int t, int slot, bool fresh) {
#pragma unroll
      for (int ks = 0; ks < kPromptKeys / 16; ++ks) {
        const uint32_t at = tmem + 256u * t + 8u * ks + (LO && ks >= 4 ? 32u : 0u);
        const uint64_t v = v_desc + slot * (L::kTile >> 4) + ks * (2048u >> 4);
        mma_f16_ts(lead, tmem + 256u * t + 128u, at, v, idesc_o, fresh && ks == 0 ? 0u : 1u);
        if constexpr (LO) mma_f16_ts(lead, tmem + 256u * t + 128u, at + 32u, v, idesc_o, 1u);
      }
    };
    bool ok = wait(&bars->kfull[0], 0, PS_KFULL);
    if (pairs) {
      // key tile i has operands and softmax i & 1: S of tile i + 2 follows P V of tile i
      for (int i = 0; i < u.tiles + 2 && ok; ++i) {
        const int t = i & 1, n = i >> 1;                   // tile i - 2 leaves the softmax, tile i enters
        if (i >= 2) {
          ok = wait(&bars->vfull[t], (n - 1) & 1, PS_VFULL) && wait(&bars->pready[t], (n - 1) & 1, PS_PREADY);
          if (!ok) break;
          tc_fence_after_sync();
          issue_o(t, t, i < 4);
          mma_commit(lead, smem_u32(&bars->vempty[t]));
          if (i >= u.tiles) mma_commit(lead, smem_u32(&bars->ofull[t]));
        }
        if (i < u.tiles) {
          if (i > 0) ok = wait(&bars->kfull[t], n & 1, PS_KFULL);
          if (ok && i < 2) ok = wait(&bars->qfull[t], 0, PS_QFULL);
          if (!ok) break;
          tc_fence_after_sync();
          issue_s(t, t);
          mma_commit(lead, smem_u32(&bars->kempty[t]));
        }
      }
    }
    for (int t = 0; t < u.row_tiles && ok && !pairs; ++t) {
      ok = wait(&bars->qfull[t], 0, PS_QFULL);
      if (ok) {
        tc_fence_after_sync();
        issue_s(t, 0);
      }
    }
    if (ok && !pairs) mma_commit(lead, smem_u32(&bars->kempty[0]));
    for (int i = 0; i < u.tiles && ok && !pairs; ++i) {
      const int slot = i & 1, next = slot ^ 1;
      const bool more = i + 1 < u.tiles;
      ok = wait(&bars->vfull[slot], (i >> 1) & 1, PS_VFULL);
      if (ok && more) ok = wait(&bars->kfull[next], ((i + 1) >> 1) & 1, PS_KFULL);
      for (int t = 0; t < u.row_tiles && ok; ++t) {
        ok = wait(&bars->pready[t], i & 1, PS_PREADY);
        if (!ok) break;
        tc_fence_after_sync();
        issue_o(t, slot, i == 0);
        if (more) issue_s(t, next);
        else mma_commit(lead, smem_u32(&bars->ofull[t]));
      }
      if (!ok) break;
      mma_commit(lead, smem_u32(&bars->vempty[slot]));
      if (more) mma_commit(lead, smem_u32(&bars->kempty[next]));
    }
    // nothing is in flight when TMEM is freed, also after a wait was given up
    mma_commit(lead, smem_u32(&bars->drain));
    (void)mbar_wait(smem_u32(&bars->drain), 0u, p.wait_limit_ns, nullptr, p.c.err, DK_PROMPT,
                    PS_DRAIN, blockIdx.x);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// `ctas`: one per unit, or for drafted trees at least one per piece.
template <int D, PromptKind KIND, bool LO = false>
cudaError_t launch_prompt_d(const AttendParams& p, int row_tiles, int64_t ctas, cudaStream_t s) {
  constexpr int smem = KIND != kCausal ? PromptSmem<D>::kTreeAlloc : PromptSmem<D>::kAlloc;
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  const bool mods = p.softcap > 0.f || p.slopes != nullptr;
  auto* fn = mods ? prompt_kernel<D, true, KIND, LO> : prompt_kernel<D, false, KIND, LO>;
  static thread_local int set_on[2] = {-1, -1};
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (set_on[mods] != dev) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    set_on[mods] = dev;
  }
  return launch_early(fn, ctas, kPromptThreads, smem, s, p, row_tiles);
}

template <int D>
cudaError_t launch_tree_d(bool cut, const AttendParams& p, int row_tiles, int64_t ctas, cudaStream_t s) {
  if (p.is_bf16)
    return cut ? launch_prompt_d<D, kTreeCut>(p, row_tiles, ctas, s) : launch_prompt_d<D, kTreeWhole>(p, row_tiles, ctas, s);
  return cut ? launch_prompt_d<D, kTreeCut, true>(p, row_tiles, ctas, s)
             : launch_prompt_d<D, kTreeWhole, true>(p, row_tiles, ctas, s);
}

}  // namespace b2b
