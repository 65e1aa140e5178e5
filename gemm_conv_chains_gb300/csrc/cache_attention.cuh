// cache_attention.cuh -- attention over a paged e4m3 cache for a few query rows per sequence
// and kv head (single tokens, drafts), split along the context; right for any number of rows.
//
// out = softmax(z) V with z = cap tanh(q k scale / cap) + slope (j - i) over the keys j <= i
// of a sequence (cap and bias optional), k and v = code * the page's scale.  Each cached byte
// is read once for all query heads that share it, so the bound is HBM: 2 D bytes per token and
// kv head.  Every SM has to turn ~24 bytes per clock into fp16 and multiply them with all rows,
// more than its fp32 lanes can; warp-level tensor-core products (m16n8k16) have the rate, and
// with so few rows the 128-row tcgen05 tile would be nearly empty.
//
// The tokens are the M side of both products (S^T = K Q^T, O^T = V^T P^T) and the query rows
// the N side, in tiles of 8, so that up to 8 rows (a usual group of query heads) waste nothing.
// The order of the summed index is free as long as both operands share it, and so are the orders
// of tokens and channels, which removes every transposition of 8-bit data: a lane reads runs of
// channels of its own fragment rows (lane = 4 g + t; keys: two tokens by g, channel run t;
// values: four tokens by t, channel run by g), and only P^T crosses lanes (movmatrix).  A strip
// is copied as it lies (whole 128-byte lines, each written to shared memory at once: lines
// scattered to the lanes that want them took 20 shared-memory cycles per instruction instead of
// 4, and bounded the kernel), its 16-byte units xor-ed so that the reads meet no bank twice.  A
// warp's ring is its own: no block barrier, only cp.async groups and a warp barrier.
//
// Work is cut evenly: the tiles of 64 tokens of all (sequence, kv head, row tile) are numbered
// in a row and each CTA takes an equal run of them, found from the lengths on the device; runs
// that split a row tile leave fp32 partial results (normalised, with their log2 sums) that a
// second small kernel joins.  A CTA's four warps take the 16-token strips in turn, each with a
// running maximum and sum of its own, joined in shared memory.
//
// Precision: codes are exact in fp16, and so are bf16 queries down to 2^-31 of the largest channel of
// their row, which a power of two puts near the top of fp16 (smaller channels to 2^-39 of it); the
// products sum in fp32; the softmax is fp32.  P is rounded to fp16: 11 bits, much finer than a
// bf16 output.  For fp16 outputs, whose own rounding is no coarser, the rest that this rounding
// leaves is multiplied as well (one token over 250001 cached, error against 64 bits 3.0e-4
// without it, 2.1e-4 with it, which is the output's own rounding; 30.8 us -> 31.9).  The value
// scales go into P before the rounding, and a row's running reference is that of the products (of
// z + log2 scale), not of z alone: what a row's output mostly consists of keeps all of P's bits,
// whatever the scales of the pages that it attends to less.
//
// Measured: 128 sequences of 8192 tokens, 32 query heads on 8 of 128 channels: 334 us, 6.45 TB/s,
// 0.95 of the copy rate; 64 ragged ones of up to 4096: 62 us, 4.9 TB/s (a run's start, its page
// numbers and the joining weigh more); 5 drafted tokens, 256 channels, softcap and bias: 49.5 us,
// 3.1 TB/s, where the arithmetic counts too (two CTAs per SM for the registers of 16 rows).
#pragma once

#include "decoder_device.cuh"

namespace b2b {

constexpr int kAttendWarps = 4;
constexpr int kTileTokens = 64;        // tokens per numbered tile: one strip per warp
constexpr int kStrip = 16;
constexpr float kNoMax = -1e30f;       // "no key seen": finite, so that no inf - inf arises

__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t* src, uint32_t* w) {
  if constexpr (BYTES == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(src);
  }
}

template <int D_, int NT>
struct CacheDims {
  static constexpr int D = D_;
  static constexpr int kKBytes = D / 4;                                   // per lane and token
  static constexpr int kVBytes = D / 8;
  static constexpr int kKRun = kKBytes % 16 == 0 ? 16 : 8;                // bytes per copy
  static constexpr int kVRun = kVBytes % 16 == 0 ? 16 : kVBytes % 8 == 0 ? 8 : 4;
  // Fragment row r (0..7) holds token r, or with kSpread token (r & 1) * 4 + (r >> 1): then the four
  // tokens that a lane's values come from are neighbours (t, t + 4, t + 8, t + 12).
  static constexpr bool kSpread = D == 64 || D == 128 || D == 256;
  static __device__ __forceinline__ int token_of_row(int r) {
    return kSpread ? (r & 1) * 4 + (r >> 1) : r;
  }
  static __device__ __forceinline__ int value_token(int t, int i) {
    return kSpread ? t + 4 * i : 2 * t + (i & 1) + 8 * (i >> 1);
  }
  // Run of channels that lane row g takes of a value row (the first of its runs).
  static __device__ __forceinline__ int value_run(int g) {
    return D == 128 || D == 256 ? (g & 1) * 4 + (g >> 1) : g;
  }
  // Byte offset of byte b of token `tok` in a strip: the 16-byte units of a 128-byte line change
  // places by the token.
  static __device__ __forceinline__ uint32_t at(int tok, int b) {
    uint32_t o = tok * D + b;
    if constexpr (D == 128 || D == 256) o ^= (tok & 7) << 4;
    else if constexpr (D == 64) o ^= (((tok >> 2) & 1) << 6) ^ (((tok >> 1) & 1) << 5);
    return o;
  }
  static constexpr int kStage = kStrip * 2 * D;                           // bytes per warp
  // what fits the CTAs per SM (64 or 96 KB of ring each): ~150 KB in flight per SM, several times
  // what the HBM latency asks for
  static constexpr int kCtas = attend_ctas_per_sm(D, NT);
  static constexpr int kStages =
      kCtas == 3 ? (D <= 64 ? 8 : D <= 96 ? 5 : 4) : (D <= 64 ? 8 : D <= 96 ? 7 : D <= 128 ? 6 : D <= 192 ? 4 : 3);
  static constexpr int kRing = kStages * kStage;
};

template <int D, int NT>
constexpr int attend_smem() {
  constexpr int ring = kAttendWarps * CacheDims<D, NT>::kRing;
  constexpr int join = kAttendWarps * NT * 8 * (D + 6) * 4;
  return (ring > join ? ring : join) + kAttendWarps * CacheDims<D, NT>::kStages * 8 +
         (NT > 1 ? D / 16 * NT * 256 : 0) + NT * 8 * 4;
}

// MODS: capped or biased scores.  F16: fp16 queries and outputs, else bf16.
template <int D, int NT, bool MODS, bool F16>
__global__ void __launch_bounds__(kAttendWarps * 32, attend_ctas_per_sm(D, NT)) attend_kernel(const AttendParams p) {
  using C = CacheDims<D, NT>;
  constexpr int RT = NT * 8;
  constexpr int KS = D / 16;           // k steps of S^T, m tiles of O^T
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const CacheView& c = p.c;

  constexpr int kJoin = kAttendWarps * RT * (D + 6) * 4;
  constexpr int kBody = kAttendWarps * C::kRing > kJoin ? kAttendWarps * C::kRing : kJoin;
  uint8_t* ring = smem + warp * C::kRing;
  const uint32_t ring_at = smem_u32(ring);
  float2* stage_scales = reinterpret_cast<float2*>(smem + kBody) + warp * C::kStages;
  uint2* q_frags = reinterpret_cast<uint2*>(smem + kBody + kAttendWarps * C::kStages * 8);
  float* row_units = reinterpret_cast<float*>(smem + kBody + kAttendWarps * C::kStages * 8 +
                                              (NT > 1 ? KS * NT * 256 : 0));

  // ---- this CTA's run of tiles ----
  // (Counts of tiles fit 32 bits: the host refuses more.  The plan is latency, in a kernel whose
  // instructions are not in the cache yet: one pass of loads, 32-bit arithmetic, short code.)
  auto work_of = [&](const Sequence& s) -> uint32_t {
    if (s.n <= 0) return 0u;
    const uint32_t row_tiles = (static_cast<uint32_t>(s.n) * p.group + RT - 1) / RT;
    const uint32_t tiles = p.whole ? 1u : (s.len + kTileTokens - 1) / kTileTokens;
    return row_tiles * c.heads * tiles;
  };
  // lane's share of the first kHeld x 32 sequences stays in registers for the search
  constexpr int kHeld = 4;
  grid_dependency_wait();                              // launched early
  uint32_t held[kHeld], total = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    held[i] = 0u;
    if (32 * i + lane < c.B) held[i] = work_of(load_sequence(c, 32 * i + lane, DK_ATTEND));
    total += held[i];
  }
  for (int b = 32 * kHeld + lane; b < c.B; b += 32) total += work_of(load_sequence(c, b, DK_ATTEND));
  total = __reduce_add_sync(0xffffffffu, total);
  uint32_t per = (total + gridDim.x - 1) / gridDim.x;
  if (!p.whole && per < static_cast<uint32_t>(p.min_tiles)) per = p.min_tiles;
  uint32_t at = blockIdx.x * per;
  const uint32_t run_begin = at, run_end = at + per < total ? at + per : total;
  const bool scribe = p.meta != nullptr && blockIdx.x == 0 && warp == 0;
  if (scribe && lane == 0) p.meta[0] = per;            // for the kernel that joins the runs
  grid_launch_dependents();
  if (at >= run_end && !scribe) return;

  // the sequence that holds tile `at`, and the number of its first tile
  int b = 0;
  uint32_t base = 0;
  {
    uint32_t before = 0;
    bool found = false;
#pragma unroll 1
    for (int i = 0; 32 * i < c.B; ++i) {
      uint32_t w = 0u;
      if (i < kHeld) w = i == 0 ? held[0] : i == 1 ? held[1] : i == 2 ? held[2] : held[3];
      else if (32 * i + lane < c.B) w = work_of(load_sequence(c, 32 * i + lane, DK_ATTEND));
      uint32_t upto = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      upto += before;
      if (scribe && 32 * i + lane < c.B) p.meta[1 + 32 * i + lane] = upto - w;
      const uint32_t hit = __ballot_sync(0xffffffffu, upto > at);
      if (hit != 0u && !found) {
        const int src = __ffs(hit) - 1;
        b = 32 * i + src;
        base = __shfl_sync(0xffffffffu, upto - w, src);
        found = true;
        if (!scribe) break;
      }
      before = __shfl_sync(0xffffffffu, upto, 31);
    }
  }

  Sequence s = at < run_end ? load_sequence(c, b, DK_ATTEND) : Sequence{0, 0, 0};
  while (at < run_end) {
    // ---- the next piece: (sequence b, kv head h, row tile rt), tiles [t0, t1) of it ----
    uint32_t work = work_of(s);
    while (at >= base + work) {
      base += work;
      s = load_sequence(c, ++b, DK_ATTEND);
      work = work_of(s);
    }
    const int rows = s.n * p.group;
    const uint32_t row_tiles = static_cast<uint32_t>(rows + RT - 1) / RT;
    const uint32_t tiles = p.whole ? 1u : static_cast<uint32_t>(s.len + kTileTokens - 1) / kTileTokens;
    const uint32_t piece = (at - base) / tiles;
    const int h = row_tiles == 1 ? piece : piece / row_tiles;
    const int rt = static_cast<int>(piece - h * row_tiles);
    const uint32_t t0 = at - base - piece * tiles;
    uint32_t t1 = t0 + (run_end - at);
    if (t1 > tiles) t1 = tiles;
    const bool partial = t0 != 0 || t1 != tiles;
    const int slot = (t0 == 0 && at != run_begin) ? 1 : 0;
    at += t1 - t0;

    const int row0 = rt * RT;
    const int last_row = row0 + RT - 1 < rows ? row0 + RT - 1 : rows - 1;
    const int start = s.len - s.n;
    const int low_limit = start + row0 / p.group;         // last key of the tile's first row
    const int high_limit = start + last_row / p.group;    // and of its last
    int strip = static_cast<int>(p.whole ? 0 : t0 * (kTileTokens / kStrip)) + warp;
    const int strips_all = high_limit / kStrip + 1;
    const int strips_run = p.whole ? strips_all : static_cast<int>(t1 * (kTileTokens / kStrip));
    const int strip_end = strips_run < strips_all ? strips_run : strips_all;

    // ---- page numbers and scales of this warp's next 32 strips, one per lane ----
    const int32_t* pages_of = c.page_table + static_cast<int64_t>(b) * c.max_pages;
    const int page_strips_shift = c.page_shift - 4;
    auto fetch_page = [&](int first) -> int {
      const int st = first + lane * kAttendWarps;
      if (st >= strip_end) return -2;
      return pages_of[st >> page_strips_shift];
    };
    auto fetch_scales = [&](int id, float2& sc) {
      sc = make_float2(0.f, 0.f);
      if (id == -2) return;
      if (id < 0 || id >= c.pages) {
        index_error(c.err, DK_ATTEND, DEC_ERR_PAGE, static_cast<uint32_t>(b));
        sc = make_float2(__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u));
        return;
      }
      const int64_t at_scale = static_cast<int64_t>(id) * c.heads + h;
      sc = make_float2(c.k_scale[at_scale], c.v_scale[at_scale]);
    };
    int issue_strip = strip, issue_n = 0;            // next strip to copy, and its count
    int issue_stage = 0;
    int ids = fetch_page(strip), next_ids = fetch_page(strip + 32 * kAttendWarps);
    float2 scs = make_float2(0.f, 0.f), next_scs = scs;

    const int64_t head_bytes = static_cast<int64_t>(D) << c.page_shift;
    // The next strip's bytes, then (they are needed later, and come from another load) its scales.
    auto issue_copy = [&]() {
      if (issue_strip < strip_end) {
        int id = __shfl_sync(0xffffffffu, ids, issue_n & 31);
        if (static_cast<uint32_t>(id) >= static_cast<uint32_t>(c.pages)) id = 0;   // its scales are NaN
        const int slot0 = (issue_strip << 4) & ((1 << c.page_shift) - 1);
        const int64_t off =
            (static_cast<int64_t>(id) * c.heads + h) * head_bytes + slot0 * D + 16 * lane;
        const uint32_t dst = ring_at + issue_stage * C::kStage;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int unit = 32 * i + lane;
          const uint32_t to = dst + C::at(unit / (D / 16), 16 * (unit % (D / 16)));
          copy_async(to, c.k + off + 512 * i);
          copy_async(to + kStrip * D, c.v + off + 512 * i);
        }
      }
      copy_commit();
    };
    auto issue_scales = [&]() {
      if (issue_strip < strip_end) {
        const int k = issue_n & 31;
        const float ks = __shfl_sync(0xffffffffu, scs.x, k);
        const float vs = __shfl_sync(0xffffffffu, scs.y, k);
        if (lane == 0) stage_scales[issue_stage] = make_float2(ks, vs);
      }
    };
    auto advance = [&]() {
      if (issue_strip >= strip_end) return;
      issue_stage = issue_stage + 1 == C::kStages ? 0 : issue_stage + 1;
      issue_strip += kAttendWarps;
      ++issue_n;
      if ((issue_n & 31) == 16) {
        fetch_scales(next_ids, next_scs);
      } else if ((issue_n & 31) == 0) {              // the prefetched 32 take over
        ids = next_ids;
        scs = next_scs;
        next_ids = fetch_page(issue_strip + 32 * kAttendWarps);
      }
    };
    static_assert(C::kStages <= 16, "the first fill stays within the first 32 strips' half");
    // ---- the query rows as fp16 fragments ----
    // k step u, lane (g, t): row 8 nt + g, channels kKRun * (t + 4 j) + 4 * (u mod run) + 0..3.
    // One row tile of 8: every warp holds it; more: warp nt turns tile nt, through shared memory.
    // The loads go out here, behind the page numbers and ahead of what waits for those.
    constexpr int kPerRun = C::kKRun / 4;            // k steps per run of channels
    const int q_nt = NT == 1 ? 0 : warp;
    const int q_row = row0 + 8 * q_nt + g;
    const bool q_valid = q_nt < NT && q_row < rows;
    uint32_t raw[KS][2];
    {
      const int tq = q_valid ? q_row / p.group : 0;
      const uint16_t* src = p.q + (s.row + static_cast<int64_t>(tq)) * p.ldq +
                            static_cast<int64_t>(h * p.group + (q_valid ? q_row - tq * p.group : 0)) * D;
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        const int d = C::kKRun * (t + 4 * (u / kPerRun)) + 4 * (u % kPerRun);
        uint2 w = make_uint2(0u, 0u);
        if (q_valid) w = *reinterpret_cast<const uint2*>(src + d);
        raw[u][0] = w.x;
        raw[u][1] = w.y;
      }
    }
    {
      const int strip0 = issue_strip;
#pragma unroll 1
      for (int i = 0; i < C::kStages - 1; ++i) {
        issue_copy();
        issue_stage = i + 1;
        issue_strip += kAttendWarps;
        ++issue_n;
      }
      fetch_scales(ids, scs);
      issue_strip = strip0;
      issue_n = issue_stage = 0;
    }
    uint32_t qf[NT == 1 ? KS : 1][2];
    float qfactor[NT][2];                            // of rows 8 nt + 2 t, + 1
    // The last key that each of them sees; with MODS as how far it lies behind the tile's last row's,
    // which gives the distance of key and row as well.
    int limit[MODS ? 1 : NT][2];
    float slope[MODS ? NT : 1][2], behind[MODS ? NT : 1][2];
    {
      float amax = 0.f;
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        const float2 a = widen2<!F16>(raw[u][0]);
        const float2 z = widen2<!F16>(raw[u][1]);
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(z.x), fabsf(z.y))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float inv;
      const float unit = row_unit<!F16>(amax, inv);
      // (q_frags and row_units are free: the last piece ended in a block barrier)
      if (t == 0 && (NT == 1 ? warp == 0 : warp < NT)) row_units[8 * q_nt + g] = unit;
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        uint32_t w[2] = {raw[u][0], raw[u][1]};
        if constexpr (!F16) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 a = widen2<true>(w[i]);
            w[i] = narrow2<false>(a.x * inv, a.y * inv);
          }
        }
        if constexpr (NT == 1) {
          qf[u][0] = w[0];
          qf[u][1] = w[1];
        } else {
          if (warp < NT) q_frags[(u * NT + warp) * 32 + lane] = make_uint2(w[0], w[1]);
        }
      }
      __syncthreads();
    }
    // the scales of the first strips, asked for with their bytes
#pragma unroll 1
    for (int i = 0; i < C::kStages - 1; ++i) {
      issue_scales();
      advance();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row0 + 8 * nt + 2 * t + i;
        const bool valid = r < rows;
        const int tq = valid ? r / p.group : 0;
        qfactor[nt][i] = row_units[8 * nt + 2 * t + i] * p.scale * (MODS ? 1.f : kLog2e);
        if constexpr (MODS) {
          behind[nt][i] = static_cast<float>(valid ? high_limit - (start + tq) : 0);
          slope[nt][i] = 0.f;
          if (p.slopes != nullptr && valid) slope[nt][i] = p.slopes[h * p.group + (r - tq * p.group)];
        } else {
          limit[nt][i] = valid ? start + tq : 0x7FFFFFFF;
        }
      }

    float o[KS][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNoMax;
      l[nt][0] = l[nt][1] = 0.f;
    }

    // ---- the strips ----
    for (int stage = 0; strip < strip_end; strip += kAttendWarps) {
      copy_wait<C::kStages - 2>();
      __syncwarp();
      const float2 sc = stage_scales[stage];
      const uint8_t* src = ring + stage * C::kStage;
      stage = stage + 1 == C::kStages ? 0 : stage + 1;
      float x[NT][4], x2[NT][4];           // even and odd k steps: two shorter chains of MMAs
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = x2[nt][e] = 0.f;
      {
        uint32_t kw[2][C::kKBytes / 4];
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int j = 0; j < C::kKBytes / C::kKRun; ++j)
            load_words<C::kKRun>(src + C::at(C::token_of_row(g) + 8 * half, C::kKRun * (t + 4 * j)),
                                 kw[half] + j * (C::kKRun / 4));
#pragma unroll
        for (int u = 0; u < KS; ++u) {
          uint32_t a[4];
          e4m3x4_to_f16(kw[0][u], a[0], a[2]);
          e4m3x4_to_f16(kw[1][u], a[1], a[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint2 q;
            if constexpr (NT == 1) q = make_uint2(qf[u][0], qf[u][1]);
            else q = q_frags[(u * NT + nt) * 32 + lane];
            mma_m16n8k16(u & 1 ? x2[nt] : x[nt], a, q.x, q.y);
          }
        }
      }
      const int tok0 = strip * kStrip + C::token_of_row(g);   // of x[.][0], x[.][1]; + 8: of x[.][2], x[.][3]
      const bool edge = strip * kStrip + kStrip - 1 > low_limit;
      // scores in the log2 domain
      const float away = MODS ? static_cast<float>(tok0 - high_limit) : 0.f;
      auto hidden = [&](int nt, int i, int k) -> bool {      // token tok0 + 8 k from row 8 nt + 2 t + i
        if constexpr (MODS) return away + static_cast<float>(8 * k) + behind[nt][i] > 0.f;
        else return tok0 + 8 * k > limit[nt][i];
      };
      // (a value scale that is no number enters here, so that rows that do not reach its page stay clear)
      const float bad = sc.y - sc.y, vs = bad == 0.f ? sc.y : 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float z = fmaf(x[nt][e] + x2[nt][e], qfactor[nt][e & 1] * sc.x, bad);
          if constexpr (MODS) {
            if (p.softcap > 0.f) z = capped(z, p.softcap, p.inv_softcap);
            z = fmaf(slope[nt][e & 1], away + static_cast<float>(8 * (e >> 1)) + behind[nt][e & 1], z) * kLog2e;
          }
          if (edge && hidden(nt, e & 1, e >> 1)) z = -INFINITY;
          x[nt][e] = z;
        }
      // A row's reference m is for e = 2^(z - m) times the page's value scale, which is P: it moves
      // when one would be above 2^15, inside fp16, and then to where that one is 2^7, so that most
      // strips neither reduce nor rescale.  e itself, which the row sum takes, stays below 2^96.
      const float room = fminf(15.f - log2_fast(vs), 96.f);
      bool above = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) above |= x[nt][e] > m[nt][e & 1] + room;
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(x[nt][i], x[nt][i + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float now = fmaxf(m[nt][i], top - (room - 8.f));
            const float f = exp2_fast(m[nt][i] - now);
            m[nt][i] = now;
            l[nt][i] *= f;
#pragma unroll
            for (int u = 0; u < KS; ++u) {
              o[u][nt][i] *= f;
              o[u][nt][i + 2] *= f;
            }
          }
      }
      uint32_t pf[NT][2], rest[NT][2];     // P, and for fp16 outputs what its rounding left
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = exp2_fast(x[nt][i] - m[nt][i & 1]);
          l[nt][i & 1] += e[i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = e[2 * i] * vs, z = e[2 * i + 1] * vs;
          const uint32_t r = narrow2<false>(a, z);
          pf[nt][i] = transpose8x8(r);
          if constexpr (F16) {
            const float2 kept = widen2<false>(r);
            rest[nt][i] = transpose8x8(narrow2<false>(a - kept.x, z - kept.y));
          }
        }
      }
      // ---- O^T += V^T P^T ----
      uint32_t vw[4][C::kVBytes / 4];
#pragma unroll
      for (int tok = 0; tok < 4; ++tok)
#pragma unroll
        for (int j = 0; j < C::kVBytes / C::kVRun; ++j)
          load_words<C::kVRun>(src + kStrip * D + C::at(C::value_token(t, tok),
                                                        C::kVRun * (C::value_run(g) + 8 * j)),
                               vw[tok] + j * (C::kVRun / 4));
      auto value_tile = [&](int i, uint32_t (&a)[4]) {
        const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
        e4m3x4_to_f16(__byte_perm(vw[0][i / 2], vw[1][i / 2], sel), a[0], a[1]);
        e4m3x4_to_f16(__byte_perm(vw[2][i / 2], vw[3][i / 2], sel), a[2], a[3]);
      };
      if (edge) {
        // Slots past every row's reach may hold anything, a NaN too (0 * NaN is one): they are
        // taken as zeros.  A NaN in a token that only some rows reach is taken out as well and
        // put into the rows that do reach it.
        uint32_t nan = 0;
#pragma unroll
        for (int tok = 0; tok < 4; ++tok) {
          const int at_tok = strip * kStrip + C::value_token(t, tok);
#pragma unroll
          for (int w = 0; w < C::kVBytes / 4; ++w) {
            if (at_tok > high_limit) vw[tok][w] = 0u;
            nan |= ((vw[tok][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
          }
        }
        if (__any_sync(0xffffffffu, nan != 0u)) {
          uint32_t seen[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              seen[nt][i] = transpose8x8((hidden(nt, 0, i) ? 0u : 0x3C00u) |
                                         (hidden(nt, 1, i) ? 0u : 0x3C000000u));
          uint32_t keep[4][C::kVBytes / 4];
#pragma unroll
          for (int tok = 0; tok < 4; ++tok)
#pragma unroll
            for (int w = 0; w < C::kVBytes / 4; ++w) {
              const uint32_t bad =
                  ((((vw[tok][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu;
              keep[tok][w] = vw[tok][w] & ~bad;
              vw[tok][w] = bad & 0x38383838u;        // e4m3 1.0 where a NaN was
            }
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            uint32_t a[4];
            value_tile(i, a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float hits[4] = {0.f, 0.f, 0.f, 0.f};
              mma_m16n8k16(hits, a, seen[nt][0], seen[nt][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (hits[e] > 0.f) o[i][nt][e] = __uint_as_float(0x7FC00000u);
            }
          }
#pragma unroll
          for (int tok = 0; tok < 4; ++tok)
#pragma unroll
            for (int w = 0; w < C::kVBytes / 4; ++w) vw[tok][w] = keep[tok][w];
        }
      }
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        uint32_t a[4];
        value_tile(i, a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_m16n8k16(o[i][nt], a, pf[nt][0], pf[nt][1]);
          if constexpr (F16) mma_m16n8k16(o[i][nt], a, rest[nt][0], rest[nt][1]);
        }
      }
      issue_copy();
      issue_scales();
      advance();
    }
    copy_wait<0>();

    // ---- the four warps' results joined ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 4);
        l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 8);
        l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], 16);
      }
    __syncthreads();                                 // every ring is drained
    float* join = reinterpret_cast<float*>(smem);
    // rows of D + 4 floats; the pairs of a 16-channel block change places by the block, so that the
    // lanes of a store, whose channels are 16 apart, meet few banks twice
    constexpr int kRow = D + 4;
    auto place = [](int d) { return (d & ~15) | ((d & 15) ^ (((d >> 4) & 7) << 1)); };
    float* mine = join + warp * RT * kRow;
    float2* stats = reinterpret_cast<float2*>(join + kAttendWarps * RT * kRow);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int w = i / 2;
      const int d =
          place(C::kVRun * (C::value_run(g) + 8 * (4 * w / C::kVRun)) + (4 * w) % C::kVRun + 2 * (i & 1));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = 8 * nt + 2 * t;
        *reinterpret_cast<float2*>(mine + r * kRow + d) =
            make_float2(o[i][nt][0], o[i][nt][2]);
        *reinterpret_cast<float2*>(mine + (r + 1) * kRow + d) =
            make_float2(o[i][nt][1], o[i][nt][3]);
      }
    }
    if (g == 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          stats[warp * RT + 8 * nt + 2 * t + i] = make_float2(m[nt][i], l[nt][i]);
    }
    __syncthreads();
    float* part = nullptr;
    if (partial) part = p.part + (2 * static_cast<int64_t>(blockIdx.x) + slot) * RT * (D + 1);
    for (int j = threadIdx.x; j < RT * D / 4; j += kAttendWarps * 32) {
      const int r = j / (D / 4), d = 4 * (j % (D / 4));
      if (row0 + r >= rows) break;
      float2 st[kAttendWarps];
      float top = kNoMax;
#pragma unroll
      for (int w = 0; w < kAttendWarps; ++w) {
        st[w] = stats[w * RT + r];
        top = fmaxf(top, st[w].x);
      }
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kAttendWarps; ++w) {
        const float f = exp2_fast(st[w].x - top);
        sum += f * st[w].y;
        const float4 v = *reinterpret_cast<const float4*>(join + (w * RT + r) * kRow + (place(d) & ~3));
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
      }
      if ((d >> 4) & 1) acc = make_float4(acc.z, acc.w, acc.x, acc.y);   // an odd block: pairs swapped
      const float inv = sum == 0.f ? 0.f : 1.f / sum;     // a row that sees no key is zero
      acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
      if (partial) {
        *reinterpret_cast<float4*>(part + r * D + d) = acc;
        if (d == 0) part[RT * D + r] = sum == 0.f ? kNoMax : top + log2f(sum);
      } else {
        const int tq = (row0 + r) / p.group;
        uint16_t* dst = p.out + ((s.row + static_cast<int64_t>(tq)) * p.q_heads + h * p.group +
                                 (row0 + r - tq * p.group)) * D + d;
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(narrow2<!F16>(acc.x, acc.y), narrow2<!F16>(acc.z, acc.w));
      }
    }
    __syncthreads();                                 // the ring may be filled again
  }
}

template <int D, int NT, bool MODS, bool F16>
cudaError_t launch_attend_one(const AttendParams& p, cudaStream_t s) {
  constexpr int smem = attend_smem<D, NT>();
  static_assert(smem * attend_ctas_per_sm(D, NT) <= 226 * 1024, "CTAs per SM");
  auto* fn = attend_kernel<D, NT, MODS, F16>;
  // per device: a process that moves between devices sets it again, which is harmless
  static thread_local int set_on = -1;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (set_on != dev) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    set_on = dev;
  }
  return launch_early(fn, p.grid, kAttendWarps * 32, smem, s, p);
}

template <int D, int NT>
cudaError_t launch_attend_nt(const AttendParams& p, cudaStream_t s) {
  if (p.softcap > 0.f || p.slopes != nullptr)
    return p.is_bf16 ? launch_attend_one<D, NT, true, false>(p, s) : launch_attend_one<D, NT, true, true>(p, s);
  return p.is_bf16 ? launch_attend_one<D, NT, false, false>(p, s) : launch_attend_one<D, NT, false, true>(p, s);
}

template <int D>
cudaError_t launch_attend_d(int nt, const AttendParams& p, cudaStream_t s) {
  if (nt == 1) return launch_attend_nt<D, 1>(p, s);
  if constexpr (D <= 128) {
    if (nt == 4) return launch_attend_nt<D, 4>(p, s);
  }
  return launch_attend_nt<D, 2>(p, s);
}

}  // namespace b2b
