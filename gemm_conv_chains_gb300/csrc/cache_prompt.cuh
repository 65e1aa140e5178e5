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
  PS_QFULL = 48, PS_KFULL, PS_KEMPTY, PS_VFULL, PS_VEMPTY, PS_SFULL, PS_PREADY, PS_OFULL, PS_DRAIN
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
};

struct PromptBars {
  uint64_t qfull[2], kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pready[2], ofull[2], drain;
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

template <int D, bool MODS>
__global__ void __launch_bounds__(kPromptThreads, 1) prompt_kernel(const AttendParams p,
                                                                   int row_tiles) {
  using L = PromptSmem<D>;
  extern __shared__ uint8_t raw_smem[];
  const uint32_t base = (smem_u32(raw_smem) + 1023u) & ~1023u;
  uint8_t* smem = raw_smem + (base - smem_u32(raw_smem));
  PromptBars* bars = reinterpret_cast<PromptBars*>(smem + L::kBar);
  float2* scales = reinterpret_cast<float2*>(smem + L::kScales);
  uint32_t* nan_bits = reinterpret_cast<uint32_t*>(smem + L::kNan);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  PromptUnit u;
  {
    int b, rt;
    int order = static_cast<int>(blockIdx.x) / p.c.heads;
    grid_launch_dependents();
    grid_dependency_wait();                                // launched early
    if (p.meta != nullptr) {
      order = static_cast<int>(p.meta[order]);
    }
    plain_pair(p, row_tiles, order, b, rt);
    if (!prompt_unit(p, b, static_cast<int>(blockIdx.x) % p.c.heads, rt, u)) return;   // the whole CTA
  }

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
  const int edge0 = (u.start + u.row0 / p.group + 1) / kPromptKeys * kPromptKeys;

  if (warp < 8) {
    more_registers<kSoftmaxRegs>();
    // ================= softmax =================
    const int t = warp >> 2;
    const int row = u.row0 + 128 * t + (threadIdx.x & 127);
    const bool valid = row < u.rows;
    if (t < u.row_tiles) {
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
        if (p.scale < 0.f) inv = -inv;             // the maximum below wants positive factors
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
        fac = unit * fabsf(p.scale) * (MODS ? 1.f : kLog2e);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->qfull[t]));

      const int limit = valid ? u.start + tq : 0x7FFFFFFF;
      const int low_limit = u.start + (u.row0 + 128 * t) / p.group;
      const float slope = MODS && p.slopes != nullptr && valid ? p.slopes[head] : 0.f;
      float m = -1e30f, l = 0.f;                   // m: the reference of z + log2 value scale
      bool ok = true;

      for (int i = 0; i < u.tiles && ok; ++i) {
        const float2* sc = scales + (i & 3) * kGranules;
        const int tok0 = i * kPromptKeys;
        const bool edge = tok0 + kPromptKeys - 1 > low_limit;
        ok = wait(&bars->sfull[t], i & 1, PS_SFULL);
        if (!ok) break;
        tc_fence_after_sync();
        auto tile = [&](auto scores) {
        constexpr bool SCORES = decltype(scores)::value;
        // a score in the log2 domain
        auto score = [&](uint32_t raw, float f, int tok) -> float {
          float z = __uint_as_float(raw) * f;
          if (MODS) {
            if (p.softcap > 0.f) z = capped(z, p.softcap, p.inv_softcap);
            z = fmaf(slope, static_cast<float>(tok - limit), z) * kLog2e;
          }
          return z;
        };
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
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int tok = tok0 + 32 * q + 16 * g + e;
                const float z = tok > limit ? -INFINITY : score(x[e], f, tok);
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
        // ---- the reference, and what O and the row's sum have to be scaled by for it ----
        float f = 1.f;
        if (top > m + 15.f) {
          f = exp2_fast(m - (top - 7.f));
          m = top - 7.f;
          l *= f;
        }
        if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            tmem_load32(tm + o_col + 32 * q, r);
            tmem_wait32(r);
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
            tmem_st32(tm + o_col + 32 * q, r);
          }
        }
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
            const bool past = SCORES && tok0 + 32 * q + 16 * g > limit;
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
        if (!MODS && !edge && __all_sync(0xffffffffu, m > -1e29f)) {
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
        if (!done) {
          if (MODS || edge) tile(std::true_type{});
          else tile(std::false_type{});
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->pready[t]));
      }

      // ---- the output row ----
      if (ok && wait(&bars->ofull[t], 0, PS_OFULL)) {
        tc_fence_after_sync();
        const float inv = l == 0.f || l > kNoValues ? 0.f : 1.f / l;
        const int tq_out = valid ? tq : 0;
        uint16_t* dst = p.out + ((u.s.row + static_cast<int64_t>(tq_out)) * p.q_heads + head) * D;
        const bool nans = bars->nan_any != 0u;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t r[32];
          tmem_load32(tm + o_col + 32 * q, r);
          tmem_wait32(r);
          uint32_t bad = 0u;
          if (nans)
            for (int tok = edge0; tok <= limit && tok < u.kv_end; ++tok)
              bad |= nan_bits[(tok - edge0) * (D / 32) + q];
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              float o[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                o[k] = inv == 0.f ? 0.f : __uint_as_float(r[e + k]) * inv;
                if ((bad >> (e + k)) & 1u) o[k] = __uint_as_float(0x7FC00000u);
              }
              *reinterpret_cast<uint4*>(dst + 32 * q + e) = p.is_bf16 ? narrow8<true>(o) : narrow8<false>(o);
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
    prod.locate(p, u, 0);
    prod.fetch(p, u, 0, p.c.k, raw);
    float2 s2 = scales_of(0, prod.page);
    prod.locate(p, u, 1);
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
        prod.fetch(p, u, i + 1, p.c.k, raw);
        s2 = scales_of(i + 1, prod.page);
        prod.locate(p, u, i + 2);
      }
    }
  } else if (warp < 16) {
    fewer_registers<kProducerRegs>();
    // ================= values =================
    PromptProducer<D> prod;
    prod.tid = threadIdx.x - 384;
    constexpr int kEach = PromptProducer<D>::kEach;
    uint4 raw[kEach];
    prod.locate(p, u, 0);
    prod.fetch(p, u, 0, p.c.v, raw);
    prod.locate(p, u, 1);
    bool ok = true;
    for (int i = 0; i < u.tiles && ok; ++i) {
      const int slot = i & 1;
      if (i >= 2) ok = wait(&bars->vempty[slot], ((i >> 1) - 1) & 1, PS_VEMPTY);
      if (!ok) break;
      if (i * kPromptKeys >= edge0) {
        // Slots past every row's reach may hold anything: taken as zeros.  A NaN that only some rows
        // see comes out of the product too (0 * NaN is one) and is noted for the rows that see it.
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          if (i * kPromptKeys + prod.token(j) >= u.kv_end) raw[j] = make_uint4(0u, 0u, 0u, 0u);
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
            const int at = i * kPromptKeys + prod.token(j);
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
        prod.fetch(p, u, i + 1, p.c.v, raw);
        prod.locate(p, u, i + 2);
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
    bool ok = wait(&bars->kfull[0], 0, PS_KFULL);
    for (int t = 0; t < u.row_tiles && ok; ++t) {
      ok = wait(&bars->qfull[t], 0, PS_QFULL);
      if (ok) {
        tc_fence_after_sync();
        issue_s(t, 0);
      }
    }
    if (ok) mma_commit(lead, smem_u32(&bars->kempty[0]));
    for (int i = 0; i < u.tiles && ok; ++i) {
      const int slot = i & 1, next = slot ^ 1;
      const bool more = i + 1 < u.tiles;
      ok = wait(&bars->vfull[slot], (i >> 1) & 1, PS_VFULL);
      if (ok && more) ok = wait(&bars->kfull[next], ((i + 1) >> 1) & 1, PS_KFULL);
      for (int t = 0; t < u.row_tiles && ok; ++t) {
        ok = wait(&bars->pready[t], i & 1, PS_PREADY);
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int ks = 0; ks < kPromptKeys / 16; ++ks)
          mma_f16_ts(lead, tmem + 256u * t + 128u, tmem + 256u * t + 8u * ks,
                     v_desc + slot * (L::kTile >> 4) + ks * (2048u >> 4), idesc_o,
                     i == 0 && ks == 0 ? 0u : 1u);
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

template <int D>
cudaError_t launch_prompt_d(const AttendParams& p, int row_tiles, cudaStream_t s) {
  constexpr int smem = PromptSmem<D>::kAlloc;
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  const bool mods = p.softcap > 0.f || p.slopes != nullptr;
  auto* fn = mods ? prompt_kernel<D, true> : prompt_kernel<D, false>;
  static thread_local int set_on[2] = {-1, -1};
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (set_on[mods] != dev) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    set_on[mods] = dev;
  }
  return launch_early(fn, static_cast<int64_t>(row_tiles) * p.c.heads * p.c.B, kPromptThreads, smem, s,
                      p, row_tiles);
}

}  // namespace b2b
