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
//   warps 8-11       producers: e4m3 pages -> fp16 K and V tiles, 128B-swizzled, two of each
//   warp 12          TMEM, MMA issue:  S = Q K^T,  O += P V
//
// TMEM: S and O of both row tiles (4 x 128 columns); P (fp16 pairs) lies over the first half of
// its S.  The two row tiles alternate: while one is in its softmax the tensor core works on the
// other (P V of this key tile, then Q K^T of the next; MMAs of one thread run in issue order,
// so S of the next tile follows the products that read the P it covers).
//
// Precision as in cache_attention.cuh.  The scales of the value pages enter the exponent
// (log2, relative to a running power of two) and are divided out of the row sum, so that a
// probability costs one multiply-add, one exponential and one addition.  The row maximum only
// moves when it is exceeded by 2^8, and O, in TMEM, is rescaled only then.
#pragma once

#include "decoder_device.cuh"

namespace b2b {

constexpr int kPromptRows = 256;       // query rows of a CTA: two M = 128 tiles
constexpr int kPromptKeys = 128;       // keys per tile
constexpr int kPromptThreads = 13 * 32;
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a CTA works on: up to 256 query rows of one sequence and kv head.
struct PromptUnit {
  Sequence s;
  int b, h, row0, rows, start, kv_end, tiles, row_tiles;
};

template <int D>
__device__ __forceinline__ bool prompt_unit(const AttendParams& p, int units_per_head,
                                            PromptUnit& u) {
  // the last row tiles see the most keys: they start first
  int x = static_cast<int>(blockIdx.x);
  const int rt = units_per_head - 1 - x / (p.c.heads * p.c.B);
  x %= p.c.heads * p.c.B;
  u.h = x % p.c.heads;
  u.b = x / p.c.heads;
  u.s = load_sequence(p.c, u.b, DK_PROMPT);
  u.row0 = rt * kPromptRows;
  u.rows = u.s.n * p.group;
  if (u.row0 >= u.rows) return false;
  const int last = u.row0 + kPromptRows < u.rows ? u.row0 + kPromptRows - 1 : u.rows - 1;
  u.start = u.s.len - u.s.n;
  u.kv_end = u.start + last / p.group + 1;
  u.tiles = (u.kv_end + kPromptKeys - 1) / kPromptKeys;
  u.row_tiles = u.rows - u.row0 > 128 ? 2 : 1;
  return true;
}

// ------------------------------------------------------------------------------------
// producers: 128 tokens of a page walk as fp16 tiles [D / 64][token][64 channels], 128B swizzle
// ------------------------------------------------------------------------------------
template <int D>
struct PromptProducer {
  static constexpr int kPieces = D / 16;          // 16-byte runs of codes per token
  static constexpr int kEach = 128 * kPieces / 128;
  int64_t off[kEach];                             // byte offset of this thread's runs, -1: none

  __device__ __forceinline__ void locate(const AttendParams& p, const PromptUnit& u, int tile,
                                         int tid) {
    const CacheView& c = p.c;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int run = j * 128 + tid, token = run / kPieces, piece = run % kPieces;
      const int at = tile * kPromptKeys + token;
      off[j] = -1;
      if (at < u.kv_end) {
        int id = __ldg(c.page_table + static_cast<int64_t>(u.b) * c.max_pages + (at >> c.page_shift));
        if (id < 0 || id >= c.pages) id = 0;      // recorded, and its scales made NaN, below
        off[j] = (((static_cast<int64_t>(id) * c.heads + u.h) << c.page_shift) +
                  (at & ((1 << c.page_shift) - 1))) * D + 16 * piece;
      }
    }
  }
  __device__ __forceinline__ void fetch(const uint8_t* pool, uint4 (&raw)[kEach]) const {
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      raw[j] = off[j] >= 0 ? __ldg(reinterpret_cast<const uint4*>(pool + off[j]))
                           : make_uint4(0u, 0u, 0u, 0u);
  }
  static __device__ __forceinline__ void store(const uint4 (&raw)[kEach], uint32_t tile_at, int tid) {
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int run = j * 128 + tid, token = run / kPieces, piece = run % kPieces;
      uint32_t h[8];
      e4m3x4_to_f16(raw[j].x, h[0], h[1]);
      e4m3x4_to_f16(raw[j].y, h[2], h[3]);
      e4m3x4_to_f16(raw[j].z, h[4], h[5]);
      e4m3x4_to_f16(raw[j].w, h[6], h[7]);
      // the two 16-byte units of the run; pieces of the second 64 channels store theirs in the
      // other order, so that the eight lanes of a token fill eight different units of a row
      const uint32_t row = tile_at + (piece / 4) * 16384 + token * 128;
      const uint32_t unit = (piece % 4) * 2, sw = token & 7;
      const bool flip = piece >= 4;
      const uint32_t a0 = row + ((unit ^ sw) << 4), a1 = row + (((unit + 1) ^ sw) << 4);
      st_shared16(flip ? a1 : a0, flip ? h[4] : h[0], flip ? h[5] : h[1], flip ? h[6] : h[2],
                  flip ? h[7] : h[3]);
      st_shared16(flip ? a0 : a1, flip ? h[0] : h[4], flip ? h[1] : h[5], flip ? h[2] : h[6],
                  flip ? h[3] : h[7]);
    }
  }
};

template <int D, bool MODS>
__global__ void __launch_bounds__(kPromptThreads, 1) prompt_kernel(const AttendParams p,
                                                                   int units_per_head) {
  using L = PromptSmem<D>;
  extern __shared__ uint8_t raw_smem[];
  const uint32_t base = (smem_u32(raw_smem) + 1023u) & ~1023u;
  uint8_t* smem = raw_smem + (base - smem_u32(raw_smem));
  PromptBars* bars = reinterpret_cast<PromptBars*>(smem + L::kBar);
  float2* scales = reinterpret_cast<float2*>(smem + L::kScales);
  uint32_t* nan_bits = reinterpret_cast<uint32_t*>(smem + L::kNan);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  PromptUnit u;
  if (!prompt_unit<D>(p, units_per_head, u)) return;       // the whole CTA

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
  if (warp == 12) {
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
            if (valid) w = __ldg(reinterpret_cast<const uint4*>(src) + i);
            float f[8];
            widen8<true>(w, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
          }
          const uint32_t e = (__float_as_uint(amax) >> 23) & 0xFFu;
          if (e != 0u && e < 253u) {               // as in the split kernel
            inv = __uint_as_float((254u - e) << 23);
            unit = __uint_as_float(e << 23);
          }
        }
        if (p.scale < 0.f) inv = -inv;             // the maximum below wants positive factors
        const uint32_t dst = base + L::kQ + t * L::kTile + (threadIdx.x & 127) * 128;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (valid) w = __ldg(reinterpret_cast<const uint4*>(src) + i);
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
        fac = unit * fabsf(p.scale) * (MODS ? 1.f : 1.4426950408889634f);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->qfull[t]));

      const int limit = valid ? u.start + tq : 0x7FFFFFFF;
      const int low_limit = u.start + (u.row0 + 128 * t) / p.group;
      const float slope = MODS && p.slopes != nullptr && valid ? __ldg(p.slopes + head) : 0.f;
      const float cap2 = MODS && p.softcap > 0.f ? 2.f * 1.4426950408889634f / p.softcap : 0.f;
      float m = -1e30f, l = 0.f, vref = 0.f, lvref = 0.f;
      bool ok = true;

      for (int i = 0; i < u.tiles && ok; ++i) {
        const float2* sc = scales + (i & 3) * kGranules;
        const int tok0 = i * kPromptKeys;
        const bool edge = tok0 + kPromptKeys - 1 > low_limit;
        ok = wait(&bars->sfull[t], i & 1, PS_SFULL);
        if (!ok) break;
        tc_fence_after_sync();
        // a score in the log2 domain
        auto score = [&](uint32_t raw, float f, int tok) -> float {
          float z = __uint_as_float(raw) * f;
          if (MODS) {
            if (cap2 > 0.f) {                      // cap tanh(z / cap)
              float r;
              asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(z * cap2) + 1.f));
              z = p.softcap - 2.f * p.softcap * r;
            }
            z = fmaf(slope, static_cast<float>(tok - limit), z) * 1.4426950408889634f;
          }
          return z;
        };
        // ---- pass 1: the tile's largest score ----
        uint32_t r[32];
        float top = -INFINITY, vtop = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tmem_load32(tm + s_col + 32 * q, r);
          tmem_wait32(r);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float2 s2 = sc[2 * q + g];
            const float f = fac * s2.x;
            vtop = fmaxf(vtop, s2.y);
            if (MODS || edge) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int tok = tok0 + 32 * q + 16 * g + e;
                const float z = score(r[16 * g + e], f, tok);
                top = fmaxf(top, tok > limit ? -INFINITY : z);
              }
            } else {
              float raw_top = -INFINITY;
#pragma unroll
              for (int e = 0; e < 16; ++e) raw_top = fmaxf(raw_top, __uint_as_float(r[16 * g + e]));
              top = fmaxf(top, raw_top * f);
            }
          }
        }
        // ---- the references, and what O has to be scaled by for them ----
        float f = 1.f;
        if (top > m + 8.f) {
          f = ex2(m - top);
          m = top;
          l *= f;
        }
        if (vtop > vref) {
          const float now = __uint_as_float((__float_as_uint(vtop) & 0x7F800000u) + 0x00800000u);
          f *= vref / now;
          vref = now;
          lvref = log2f(now);
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
        // ---- pass 2: P, and the row's sum ----
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tmem_load32(tm + s_col + 32 * q, r);
          tmem_wait32(r);
          uint32_t pk[16];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const float2 s2 = sc[2 * q + g];
            const float fg = fac * s2.x;
            // log2 of the page's value scale relative to vref; 2^-60 stands for zero (its codes'
            // share vanishes, the row's sum does not)
            float lv = log2f(s2.y) - lvref;
            if (lv < -60.f) lv = -60.f;
            const float back = ex2(-lv), c = lv - m;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float y[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int tok = tok0 + 32 * q + 16 * g + e + k;
                if (MODS) y[k] = score(r[16 * g + e + k], fg, tok) + c;
                else y[k] = fmaf(__uint_as_float(r[16 * g + e + k]), fg, c);
                if (edge && tok > limit) y[k] = -INFINITY;
                y[k] = ex2(y[k]);
              }
              sum += y[0] + y[1];
              pk[8 * g + e / 2] = narrow2<false>(y[0], y[1]);
            }
            l = fmaf(sum, back, l);
          }
          tmem_store16(tm + s_col + 16 * q, pk);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->pready[t]));
      }

      // ---- the output row ----
      if (ok && wait(&bars->ofull[t], 0, PS_OFULL)) {
        tc_fence_after_sync();
        const float inv = l == 0.f ? 0.f : vref / l;
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
                o[k] = l == 0.f ? 0.f : __uint_as_float(r[e + k]) * inv;
                if ((bad >> (e + k)) & 1u) o[k] = __uint_as_float(0x7FC00000u);
              }
              *reinterpret_cast<uint4*>(dst + 32 * q + e) = p.is_bf16 ? narrow8<true>(o) : narrow8<false>(o);
            }
          }
        }
      }
    }
  } else if (warp < 12) {
    // ================= producers =================
    const int tid = threadIdx.x - 256;
    PromptProducer<D> prod;
    constexpr int kEach = PromptProducer<D>::kEach;
    uint4 raw_k[kEach], raw_v[kEach];
    prod.locate(p, u, 0, tid);
    prod.fetch(p.c.k, raw_k);
    prod.fetch(p.c.v, raw_v);
    bool ok = true;
    for (int i = 0; i < u.tiles && ok; ++i) {
      const int slot = i & 1;
      // ---- K, and the tile's scales ----
      if (i >= 2) ok = wait(&bars->kempty[slot], ((i >> 1) - 1) & 1, PS_KEMPTY);
      if (!ok) break;
      PromptProducer<D>::store(raw_k, base + L::kK + slot * L::kTile, tid);
      if (tid < kGranules) {
        const int at = i * kPromptKeys + tid * kGranule;
        float2 s2 = make_float2(0.f, 0.f);
        if (at < u.kv_end) {
          const int id = __ldg(p.c.page_table + static_cast<int64_t>(u.b) * p.c.max_pages +
                               (at >> p.c.page_shift));
          if (id < 0 || id >= p.c.pages) {
            index_error(p.c.err, DK_PROMPT, DEC_ERR_PAGE, static_cast<uint32_t>(u.b));
            s2.x = s2.y = __uint_as_float(0x7FC00000u);
          } else {
            const int64_t sa = static_cast<int64_t>(id) * p.c.heads + u.h;
            s2 = make_float2(__ldg(p.c.k_scale + sa), __ldg(p.c.v_scale + sa));
          }
        }
        scales[(i & 3) * kGranules + tid] = s2;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->kfull[slot]));
      if (i + 1 < u.tiles) {
        prod.locate(p, u, i + 1, tid);
        prod.fetch(p.c.k, raw_k);
      }
      // ---- V ----
      if (i >= 2) ok = wait(&bars->vempty[slot], ((i >> 1) - 1) & 1, PS_VEMPTY);
      if (!ok) break;
      if (i * kPromptKeys >= edge0) {
        // a NaN that only some rows see: out of the product (0 * NaN is one), noted for the rows
        // that do see it
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          uint32_t w[4] = {raw_v[j].x, raw_v[j].y, raw_v[j].z, raw_v[j].w};
          uint32_t any = 0u;
#pragma unroll
          for (int e = 0; e < 4; ++e) any |= ((w[e] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          if (any != 0u) {
            const int run = j * 128 + tid, token = run / (D / 16), piece = run % (D / 16);
            uint32_t bits = 0u;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (((w[e / 4] >> (8 * (e % 4))) & 0x7Fu) == 0x7Fu) {
                bits |= 1u << e;
                w[e / 4] &= ~(0xFFu << (8 * (e % 4)));
              }
            raw_v[j] = make_uint4(w[0], w[1], w[2], w[3]);
            const int at = i * kPromptKeys + token - edge0;
            if (at < kEdgeTokens)
              atomicOr(&nan_bits[at * (D / 32) + piece / 2], bits << (16 * (piece & 1)));
            bars->nan_any = 1u;
          }
        }
      }
      PromptProducer<D>::store(raw_v, base + L::kV + slot * L::kTile, tid);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->vfull[slot]));
      if (i + 1 < u.tiles) prod.fetch(p.c.v, raw_v);
    }
  } else {
    // ================= MMA =================
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
      for (int t = 0; t < u.row_tiles && ok; ++t) {
        ok = wait(&bars->pready[t], i & 1, PS_PREADY);
        if (ok && t == 0 && more) ok = wait(&bars->kfull[next], ((i + 1) >> 1) & 1, PS_KFULL);
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
  if (warp == 12) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_prompt_d(const AttendParams& p, cudaStream_t s) {
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
  const int64_t rows = static_cast<int64_t>(p.c.max_new) * p.group;
  const int64_t units = (rows + kPromptRows - 1) / kPromptRows;
  const int64_t blocks = units * p.c.heads * p.c.B;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  fn<<<static_cast<unsigned>(blocks), kPromptThreads, smem, s>>>(p, static_cast<int>(units));
  return cudaGetLastError();
}

}  // namespace b2b
