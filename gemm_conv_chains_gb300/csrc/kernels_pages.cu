// kernels_pages.cu -- the pages of the paged e4m3 cache: the page table of a step's sequences, copies
// of pages, and the tokens that a sequence keeps moved together.
#include "decoder_device.cuh"

namespace b2b {
namespace {

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_store(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void begin() {
  grid_launch_dependents();
  grid_dependency_wait();                              // launched early
}

// ------------------------------------------------------------------------------------
// the page table of a step's sequences
// ------------------------------------------------------------------------------------
// Row r follows row parents[r] of the old table for kept[r] tokens and gets room for new[r] more.  No
// count of a page's holders is kept between calls: a page is in use if a new row keeps it.  One word
// per page, the minimum over the rows that keep it of
//   0      the row only reads it
//   r + 1  row r keeps a part of it and will write behind that part
// says everything: nobody's (all ones: free), 0 (some row reads it: all who would write take a
// copy), r + 1 (all would write: the lowest of them does, the others take copies).  A minimum does not
// depend on the order.  Free pages are given out in the order of their numbers, to the rows in the
// order of theirs, so that the same call gives the same table.
//
// Steps: words cleared; a warp per row copies its old entries and lowers their words, eight entries of
// a lane on their way at once; what each row needs, and the sums of that over the rows; free pages counted and
// listed, a run of words per warp; each one that is needed finds its row.  All of it is latency, two to
// four dependent accesses a step.  Few rows on a small pool run in one CTA, words in shared memory.
// Otherwise two kernels spread over the card clear and mark words in the workspace, and one cluster,
// whose CTAs each have a part of the pool and meet once for its counts, does the rest: lowering the
// words in one cluster's shared memory from its eight SMs took 15 us of 25.  64 beams on 4160 pages 5.7 us, 512
// sequences on 102000 15 us.
constexpr int kPagesThreads = 1024;
constexpr int kPagesCluster = 8;
constexpr int kSmallPool = 40 * 1024;                  // words in one CTA's shared memory
constexpr int kSmallRows = 128;
constexpr int kFlight = 8;                             // entries of a lane on their way
constexpr uint32_t kNobody = 0xFFFFFFFFu;

struct PageRow {
  int parent, kept, total;
  int have;                                            // pages that hold the kept tokens
  bool writes;                                         // on the last of them
};

__device__ __forceinline__ PageRow page_row(const PagesParams& p, int r, bool report) {
  PageRow w;
  w.parent = p.parents != nullptr ? p.parents[r] : r;
  if (w.parent < -1 || w.parent >= p.B) {
    if (report) index_error(p.err, DK_PAGES, DEC_ERR_PARENT, static_cast<uint32_t>(r));
    w.parent = -1;
  }
  const int most = p.width << p.page_shift;            // fits: checked by the host
  int held = w.parent >= 0 ? p.lens[w.parent] : 0;
  w.kept = p.kept != nullptr ? p.kept[r] : held;
  const int fresh = p.fresh != nullptr ? p.fresh[r] : 0;
  const int64_t total = static_cast<int64_t>(w.kept) + fresh;
  if (held < 0 || held > most || w.kept < 0 || w.kept > held || fresh < 0 || total > most) {
    if (report) index_error(p.err, DK_PAGES, DEC_ERR_LENGTH, static_cast<uint32_t>(r));
    held = held < 0 ? 0 : held > most ? most : held;
    w.kept = w.kept < 0 ? 0 : w.kept > held ? held : w.kept;
    const int room = most - w.kept;
    w.total = w.kept + (fresh < 0 ? 0 : fresh > room ? room : fresh);
  } else {
    w.total = static_cast<int>(total);
  }
  const int mask = (1 << p.page_shift) - 1;
  w.have = (w.kept >> p.page_shift) + ((w.kept & mask) != 0 ? 1 : 0);
  w.writes = (w.kept & mask) != 0 && w.total > w.kept;
  return w;
}

// What is kept of a row whose entries have been copied.
struct KeptRow {
  int last;                                            // the page that the row writes on, -1: none
  int have, pages, tokens;                             // pages held and in all; tokens on the last one
};

// A warp: row r's old pages.
__device__ __forceinline__ KeptRow mark_row(const PagesParams& p, int r, uint32_t* words) {
  const int lane = threadIdx.x & 31;
  const PageRow w = page_row(p, r, lane == 0);
  const int32_t* from = p.table + static_cast<int64_t>(w.parent < 0 ? 0 : w.parent) * p.width;
  int32_t* to = p.table_out + static_cast<int64_t>(r) * p.width;
  int last = -1;
  for (int j0 = lane; j0 < p.width; j0 += 32 * kFlight) {
    int id[kFlight];
#pragma unroll
    for (int e = 0; e < kFlight; ++e) {
      const int j = j0 + 32 * e;
      id[e] = -1;
      if (j < w.have) id[e] = from[j];
    }
#pragma unroll
    for (int e = 0; e < kFlight; ++e) {
      const int j = j0 + 32 * e;
      if (j < w.have) {
        if (id[e] < 0 || id[e] >= p.pages) {
          index_error(p.err, DK_PAGES, DEC_ERR_PAGE, static_cast<uint32_t>(r));
          id[e] = -1;
        } else {
          const bool write = w.writes && j == w.have - 1;
          atomicMin(words + id[e], write ? static_cast<uint32_t>(r) + 1u : 0u);
          if (write) last = id[e];
        }
      }
      if (j < p.width) to[j] = id[e];
    }
  }
  last = __reduce_max_sync(0xffffffffu, last);
  if (lane < 3) p.copies[3 * static_cast<int64_t>(r) + lane] = lane < 2 ? -1 : 0;
  if (lane == 3) p.lens_out[r] = w.total;
  const int64_t up = (1 << p.page_shift) - 1;
  return KeptRow{last, w.have, static_cast<int>((w.total + up) >> p.page_shift),
                 w.kept & static_cast<int>(up)};
}

__global__ void __launch_bounds__(256) pages_clear_kernel(const PagesParams p) {
  begin();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < p.pages;
       i += static_cast<int64_t>(gridDim.x) * 256)
    p.owners[i] = kNobody;
}
__global__ void __launch_bounds__(128) pages_mark_kernel(const PagesParams p) {
  begin();
  const int r = static_cast<int>(blockIdx.x) * 4 + static_cast<int>(threadIdx.x >> 5);
  if (r >= p.rows) return;
  const KeptRow kept = mark_row(p, r, p.owners);
  if ((threadIdx.x & 31) == 0) static_cast<KeptRow*>(p.kept_rows)[r] = kept;
}

// ONE: everything, in one CTA.  Else what follows on the marks, in one cluster.
template <bool ONE>
__global__ void __launch_bounds__(kPagesThreads, 1) pages_kernel(const PagesParams p, uint32_t chunk) {
  extern __shared__ __align__(16) uint32_t pages_smem[];
  __shared__ uint32_t warp_sums[32], free_before[32];  // free pages of the warps' runs ahead of a warp's
  __shared__ uint32_t free_of[kPagesCluster];          // free pages of each CTA's chunk
  uint32_t* needs = pages_smem;                        // [rows]: pages that the row needs; then the first's rank
  uint32_t* takes = needs + p.rows;                    // [rows]: its slot, and bit 31: it is a copy
  KeptRow* kept = ONE ? reinterpret_cast<KeptRow*>(takes + p.rows + (-2 * p.rows & 3)) : static_cast<KeptRow*>(p.kept_rows);
  const uint32_t rank = ONE ? 0u : cluster_ctarank(), ctas = ONE ? 1u : cluster_size();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t pages = static_cast<uint32_t>(p.pages);
  const uint32_t lo = rank * chunk < pages ? rank * chunk : pages;
  const uint32_t n = (lo + chunk < pages ? lo + chunk : pages) - lo;
  uint32_t* all_words = ONE ? reinterpret_cast<uint32_t*>(kept + p.rows) : p.owners;
  uint32_t* words = all_words + lo;                    // this CTA's

  if constexpr (!ONE) asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  begin();
  if constexpr (ONE) {
    for (uint32_t i = threadIdx.x; i < n; i += kPagesThreads) words[i] = kNobody;
    __syncthreads();
    for (int r = warp; r < p.rows; r += 32) {
      const KeptRow k = mark_row(p, r, words);
      if (lane == 0) kept[r] = k;
    }
    __syncthreads();
  }
  // ---- the free pages of this CTA's chunk: a warp counts a run of 32 k words ----
  const uint32_t run = (n + 32 * 32 - 1) / (32 * 32) * 32;
  auto run_of = [&](uint32_t w) -> uint32_t { return w * run < n ? w * run : n; };
  const uint32_t run_lo = run_of(warp), run_hi = run_of(warp + 1);
  uint32_t free_here = 0;
#pragma unroll 8
  for (uint32_t i = run_lo + lane; i < run_hi; i += 32) free_here += words[i] == kNobody ? 1u : 0u;
  free_here = __reduce_add_sync(0xffffffffu, free_here);
  if (lane == 0) warp_sums[warp] = free_here;
  __syncthreads();
  uint32_t v = warp_sums[lane];
  const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0u);
  const uint32_t here = __reduce_add_sync(0xffffffffu, v);
  if (lane == 0) free_before[warp] = before;
  if constexpr (ONE) {
    if (threadIdx.x == 0) free_of[0] = here;
  } else {
    // (the others' shared memory may be written once they have started, which this tells)
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    if (threadIdx.x < ctas) cluster_store(mapa_shared(smem_u32(&free_of[rank]), threadIdx.x), here);
  }
  // ---- what the rows need, and the rank of each one's first page ----
  uint32_t needed = 0;
  for (int r0 = 0; r0 < p.rows; r0 += kPagesThreads) {
    const int r = r0 + static_cast<int>(threadIdx.x);
    uint32_t need = 0;
    if (r < p.rows) {
      const KeptRow w = kept[r];
      const bool copy = w.last >= 0 && all_words[w.last] != static_cast<uint32_t>(r) + 1u;
      const uint32_t slot = static_cast<uint32_t>(w.have) - (copy ? 1u : 0u);
      need = static_cast<uint32_t>(w.pages) - slot;
      takes[r] = slot | (copy ? 0x80000000u : 0u);
    }
    uint32_t upto = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    __syncthreads();                                   // warp_sums is free
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    v = warp_sums[lane];
    const uint32_t base = needed + __reduce_add_sync(0xffffffffu, lane < warp ? v : 0u);
    needed += __reduce_add_sync(0xffffffffu, v);
    if (r < p.rows) needs[r] = base + upto - need;
  }
  // every CTA has read the words of the pages that its rows write on, and has all counts
  if constexpr (ONE) __syncthreads();
  else cluster_sync();
  const uint32_t* first_rank = needs;
  uint32_t ahead = 0, all = 0;
  for (uint32_t i = 0; i < ctas; ++i) {
    if (i < rank) ahead += free_of[i];
    all += free_of[i];
  }
  // ---- the free pages that are needed, listed over the words of the warp's own run ----
  uint32_t put = run_lo;
  for (uint32_t i0 = run_lo; i0 < run_hi && ahead + before + (put - run_lo) < needed; i0 += 32) {
    const uint32_t i = i0 + lane;
    const bool is_free = i < run_hi && words[i] == kNobody;
    const uint32_t vote = __ballot_sync(0xffffffffu, is_free);
    if (is_free) words[put + __popc(vote & ((1u << lane) - 1u))] = lo + i;
    put += __popc(vote);
    __syncwarp();
  }
  __syncthreads();
  // ---- each goes to the row whose ranks hold its own ----
  const uint32_t end = ahead + here < needed ? ahead + here : needed;
  for (uint32_t q = ahead + threadIdx.x; q < end; q += kPagesThreads) {
    uint32_t w = 0;                                    // the last warp with fewer free pages ahead
#pragma unroll
    for (uint32_t o = 16; o > 0; o >>= 1)
      if (free_before[w + o] <= q - ahead) w += o;
    const int page = static_cast<int>(words[run_of(w) + (q - ahead - free_before[w])]);
    int a = 0, z = p.rows - 1;                         // the last row whose first rank is at most q
    while (a < z) {
      const int mid = (a + z + 1) / 2;
      if (first_rank[mid] <= q) a = mid;
      else z = mid - 1;
    }
    const uint32_t k = q - first_rank[a], slot = takes[a] & 0x7FFFFFFFu;
    if (k == 0 && (takes[a] >> 31) != 0u) p.copies[3 * static_cast<int64_t>(a) + 1] = page;
    p.table_out[static_cast<int64_t>(a) * p.width + slot + k] = page;
  }
  if (rank == 0) {
    // where copies come from; a copy that there is no page for is none, and the row cannot have the old
    // page either
    for (int r = threadIdx.x; r < p.rows; r += kPagesThreads) {
      if ((takes[r] >> 31) == 0u) continue;
      if (first_rank[r] < all) {
        p.copies[3 * static_cast<int64_t>(r)] = kept[r].last;
        p.copies[3 * static_cast<int64_t>(r) + 2] = kept[r].tokens;
      } else {
        p.table_out[static_cast<int64_t>(r) * p.width + (takes[r] & 0x7FFFFFFFu)] = -1;
      }
    }
    if (threadIdx.x == 0) *p.left = static_cast<int32_t>(all) - static_cast<int32_t>(needed);
  }
}

// ------------------------------------------------------------------------------------
// copies of pages
// ------------------------------------------------------------------------------------
// One block per (copy, pool, head): the first `tokens` tokens of the head's part of a page lie in a row.
// Bound by memory: 1536 copies of pages of 64 tokens, 8 heads of 128 (two times 201 MB): 65 us, 0.92 of a plain
// copy's rate.  A few copies: one launch, 1.7 us in a graph, 3.4 as calls of their own.
constexpr int kCopyThreads = 256;

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyParams p) {
  begin();
  const CacheView& c = p.c;
  const int64_t items = p.n * c.heads * 2;
  for (int64_t x = blockIdx.x; x < items; x += gridDim.x) {
    const int value = static_cast<int>(x & 1), h = static_cast<int>((x >> 1) % c.heads);
    const int64_t i = (x >> 1) / c.heads;
    const int32_t* pair = p.copies + 3 * i;
    const int from = pair[0], to = pair[1], tokens = pair[2];
    if (from < 0 || to < 0 || from == to || tokens == 0) continue;
    if (from >= c.pages || to >= c.pages || tokens < 0 || tokens > (1 << c.page_shift)) {
      if (threadIdx.x == 0)
        index_error(c.err, DK_COPY, from >= c.pages || to >= c.pages ? DEC_ERR_PAGE : DEC_ERR_LENGTH,
                    static_cast<uint32_t>(i));
      continue;
    }
    const int64_t a = static_cast<int64_t>(from) * c.heads + h, z = static_cast<int64_t>(to) * c.heads + h;
    const int64_t part = static_cast<int64_t>(c.D) << c.page_shift;
    uint8_t* pool = value ? c.v : c.k;
    const uint4* src = reinterpret_cast<const uint4*>(pool + a * part);
    uint4* dst = reinterpret_cast<uint4*>(pool + z * part);
    const int n = tokens * c.D / 16;
    for (int j = threadIdx.x; j < n; j += kCopyThreads) dst[j] = src[j];
    if (threadIdx.x == 0) {
      float* scale = value ? c.v_scale : c.k_scale;
      scale[z] = scale[a];
    }
  }
}

// ------------------------------------------------------------------------------------
// kept tokens moved together
// ------------------------------------------------------------------------------------
// Token tokens[b][i] of sequence b goes to position first[b] + i, at or below its own.  A page that
// receives tokens takes the largest scale s' of the pages that its tokens come from (its own among them
// if it keeps some in place), and codes of a smaller one become e4m3(code * (s / s')).
//
// A cluster (of one CTA unless there are few of them) per sequence, kv head and pool walks the
// positions upwards in waves of `wave` tokens per CTA, whole pages each.  All CTAs read a wave's tokens,
// meet at the cluster's barrier, and write it: what a wave reads lies at or above its own positions, so
// no write reaches what a later wave has still to read, and reading ahead is safe at any time.  So the
// tokens of the next wave are on their way (cp.async) while one is written, and their numbers, pages and
// scales, three dependent loads, are asked for one, two and three waves ahead and looked at no earlier
// than a wave later (looked at as they arrive: 62 -> 114 us on the batch below).  Tokens that stay in
// place are read only where their page's scale grows.  Many tokens: instructions and barriers of the waves,
// 4.3 TB/s; few: the chain of five dependent loads.
//
// A token that is refused (out of order, or on a page that is none) is recorded, and the slot's own token
// stays in its place as one that is kept: what the page holds keeps its values, whatever its scale becomes.
constexpr int kCompactThreads = 256;
constexpr int kMostWave = 256;                         // a page or several

template <int D>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p, int wave, int buffers) {
  constexpr int kUnits = D / 16;                       // vectors of a token
  extern __shared__ __align__(16) uint8_t compact_smem[];          // [buffers][wave][D]
  __shared__ int64_t source[2][kMostWave];             // byte offset of a token's codes in the pool,
                                                       // or -1: none, -2: it stays in place
  // Where a token goes in the pool (-1: nowhere), its source again, and what its codes are multiplied
  // by (1: nothing changes, also where the scales are equal zeros or infinities).
  struct __align__(8) Place {
    int64_t at, from;
    float ratio;
  };
  __shared__ Place place[kMostWave];
  __shared__ uint32_t most[kMostWave / 16];            // of the wave's pages, the largest scale that comes in
  begin();
  const CacheView& c = p.c;
  const uint32_t rank = cluster_ctarank(), ctas = cluster_size();
  const int64_t x = blockIdx.x / ctas;
  const int value = static_cast<int>(x & 1), h = static_cast<int>((x >> 1) % c.heads);
  const int b = static_cast<int>((x >> 1) / c.heads);
  const int first = p.first[b], count = p.counts[b], len = c.lens[b];
  const int64_t room = static_cast<int64_t>(c.max_pages) << c.page_shift;
  if (first < 0 || count < 0 || count > p.max_tokens || len > room ||
      static_cast<int64_t>(first) + count > len) {
    if (threadIdx.x == 0) index_error(c.err, DK_COMPACT, DEC_ERR_LENGTH, static_cast<uint32_t>(b));
    return;                                            // the whole cluster
  }
  if (count == 0) return;
  const int t = threadIdx.x;
  const int mask = (1 << c.page_shift) - 1, end = first + count;
  const int32_t* table = c.page_table + static_cast<int64_t>(b) * c.max_pages;
  const int32_t* tokens = p.tokens + static_cast<int64_t>(b) * p.max_tokens;
  uint8_t* pool = value ? c.v : c.k;
  float* scales = value ? c.v_scale : c.k_scale;
  const int64_t part = static_cast<int64_t>(D) << c.page_shift;
  const uint32_t buffer_at = smem_u32(compact_smem);

  // the position that this thread's token of wave w goes to
  const int64_t base = (first & ~mask) + static_cast<int64_t>(wave) * rank + t;
  const int64_t step = static_cast<int64_t>(wave) * ctas;
  const int waves = static_cast<int>((end - (first & ~mask) + step - 1) / step);
  auto goes_to = [&](int w) -> int64_t { return t < wave && w < waves ? base + w * step : end; };

  // Three dependent loads, each looked at no earlier than a wave after it was asked for.
  struct Token { int from, before; };                  // its position, and the last token's
  struct Pages { int from, id, to; };                  // the position, its page, the page it goes to
  struct Scale { int to, id; float s; };               // checked pages, -1: none
  auto ask_token = [&](int w) -> Token {
    const int64_t dst = goes_to(w);
    Token m{static_cast<int>(dst), -1};
    if (dst >= first && dst < end) {
      const int i = static_cast<int>(dst - first);
      m.from = tokens[i];
      if (i > 0) m.before = tokens[i - 1];
    }
    return m;
  };
  auto ask_pages = [&](int w, const Token& token) -> Pages {
    const int64_t dst = goes_to(w);
    Pages m{-1, -1, -1};
    if (dst >= end) return m;
    m.from = token.from;
    if (m.from < dst || m.from >= len || token.before >= m.from) {
      index_error(c.err, DK_COMPACT, DEC_ERR_TOKEN, static_cast<uint32_t>(b));
      m.from = static_cast<int>(dst);
    }
    m.to = table[dst >> c.page_shift];
    m.id = table[m.from >> c.page_shift];
    return m;
  };
  // the tokens of wave w on their way to its buffer; their scales
  auto ask_codes = [&](int w, const Pages& at) -> Scale {
    const int64_t dst = goes_to(w);
    Scale m{-1, -1, 0.f};
    bool moves = false;
    if (dst < end) {
      const bool known = at.to >= 0 && at.to < c.pages, comes = at.id >= 0 && at.id < c.pages;
      if (!known || !comes) index_error(c.err, DK_COMPACT, DEC_ERR_PAGE, static_cast<uint32_t>(b));
      moves = comes && at.from != dst;
      if (known) m = Scale{at.to, moves ? at.id : at.to, 0.f};
    }
    int64_t off = -1;
    if (m.id >= 0) off = moves ? (static_cast<int64_t>(m.id) * c.heads + h) * part + (at.from & mask) * D : -2;
    if (t < wave) source[w & 1][t] = off;
    if (m.id >= 0) m.s = scales[static_cast<int64_t>(m.id) * c.heads + h];
    return m;
  };
  // a thread's vector of a token, and its first token of a wave
  constexpr int kTokens = kCompactThreads / kUnits;    // tokens of a pass
  const int tok0 = t / kUnits, unit = t - tok0 * kUnits;
  const int tok_end = tok0 < kTokens ? wave : 0;
  auto copy_codes = [&](int w) {                       // after a barrier
    if (w < waves) {
      const uint32_t to = buffer_at + (buffers > 1 ? (w & 1) * wave * D : 0) + 16 * unit;
#pragma unroll 4
      for (int tok = tok0; tok < tok_end; tok += kTokens) {
        const int64_t from = source[w & 1][tok];
        if (from >= 0)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + tok * D), "l"(pool + from + 16 * unit)
                       : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  Token token = ask_token(0), token1 = ask_token(1), token2 = ask_token(2);
  Pages pages0 = ask_pages(0, token), pages1 = ask_pages(1, token1);
  Scale now = ask_codes(0, pages0);
  __syncthreads();
  copy_codes(0);
  for (int w = 0; w < waves; ++w) {
    // (a call of one wave has one buffer)
    const Scale next = ask_codes(w + 1, pages1);
    pages1 = ask_pages(w + 2, token2);
    token2 = ask_token(w + 3);
    if (t < kMostWave / 16) most[t] = 0u;
    __syncthreads();
    copy_codes(w + 1);
    {                                                  // (16 tokens lie on one page)
      uint32_t top = now.id >= 0 && now.s > 0.f ? __float_as_uint(now.s) : 0u;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, top, o);
        top = other > top ? other : top;
      }
      if ((t & 15) == 0 && t < wave) atomicMax(&most[t >> c.page_shift], top);
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    // ---- every CTA has the wave's tokens and scales: where each goes, and its factor ----
    const int64_t at0 = base - t + w * step;
    if (t < wave) {
      const int64_t from = source[w & 1][t];
      const float s = __uint_as_float(most[t >> c.page_shift]);
      Place to{-1, from, 1.f};
      if (from != -1 && !(from == -2 && now.s == s)) {
        to.at = (static_cast<int64_t>(now.to) * c.heads + h) * part + ((at0 + t) & mask) * D;
        if (now.s != s) to.ratio = __fdiv_rn(now.s, s);
      }
      place[t] = to;
    }
    __syncthreads();
    const uint8_t* held = compact_smem + (buffers > 1 ? (w & 1) * wave * D : 0) + 16 * unit;
#pragma unroll 2
    for (int tok = tok0; tok < tok_end; tok += kTokens) {
      const Place to = place[tok];
      if (to.at < 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(pool + to.at + 16 * unit);
      uint4 v = to.from == -2 ? *dst : *reinterpret_cast<const uint4*>(held + tok * D);
      if (to.ratio != 1.f) {
        uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t f0, f1;
          e4m3x4_to_f16(in[e], f0, f1);
          const float2 a = widen2<false>(f0), z = widen2<false>(f1);
          in[e] = e4m3x2(__fmul_rn(a.x, to.ratio), __fmul_rn(a.y, to.ratio)) |
                  (e4m3x2(__fmul_rn(z.x, to.ratio), __fmul_rn(z.y, to.ratio)) << 16);
        }
        v = make_uint4(in[0], in[1], in[2], in[3]);
      }
      *dst = v;
    }
    if (t < wave && (t & mask) == 0 && now.to >= 0)
      scales[static_cast<int64_t>(now.to) * c.heads + h] = __uint_as_float(most[t >> c.page_shift]);
    __syncthreads();                                   // the buffer, source, place and most are free
    now = next;
  }
}

}  // namespace

static bool pages_small(int64_t pages, int64_t rows) { return pages <= kSmallPool && rows <= kSmallRows; }

int64_t pages_workspace(int64_t pages, int64_t rows) {
  return pages_small(pages, rows) ? 0 : 16 * rows + (4 * pages + 15) / 16 * 16;
}

template <bool ONE>
static cudaError_t launch_pages_in(const PagesParams& p, uint32_t chunk, int smem, cudaStream_t s) {
  constexpr int kMost = ONE ? 24 * kSmallRows + 16 + 4 * kSmallPool : 8 * kMostPageRows;
  static_assert(kMost <= 227 * 1024 - 1024, "shared memory of one CTA");
  static thread_local int set_on = -1;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (set_on != dev) {
    e = cudaFuncSetAttribute(pages_kernel<ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    set_on = dev;
  }
  const int ctas = ONE ? 1 : kPagesCluster;
  return launch_early_clusters(pages_kernel<ONE>, ctas, ctas, kPagesThreads, smem, s, p, chunk);
}

cudaError_t launch_pages(PagesParams p, void* workspace, int num_sms, cudaStream_t s) {
  if (pages_small(p.pages, p.rows))
    return launch_pages_in<true>(p, static_cast<uint32_t>(p.pages),
                                 static_cast<int>(24 * p.rows + 16 + 4 * p.pages), s);
  p.kept_rows = workspace;
  p.owners = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + 16 * static_cast<int64_t>(p.rows));
  const int64_t blocks = (p.pages + 1023) / 1024;
  cudaError_t e = cudaSuccess;
  if (p.pages > 0) e = launch_early(pages_clear_kernel, blocks < 4 * num_sms ? blocks : 4 * num_sms, 256, 0, s, p);
  if (e == cudaSuccess && p.rows > 0) e = launch_early(pages_mark_kernel, (p.rows + 3) / 4, 128, 0, s, p);
  if (e != cudaSuccess) return e;
  return launch_pages_in<false>(p, static_cast<uint32_t>((p.pages + kPagesCluster - 1) / kPagesCluster),
                                8 * p.rows, s);
}

cudaError_t launch_copy(const CopyParams& p, int num_sms, cudaStream_t s) {
  const int64_t items = p.n * p.c.heads * 2, most = static_cast<int64_t>(num_sms) * 64;
  return launch_early(copy_kernel, items < most ? items : most, kCopyThreads, 0, s, p);
}

// The largest cluster of at most `most` CTAs that the current device holds at all: above 8 that is not the
// same on every one, and a launch of a larger cluster fails.
template <class... P>
static int resident_cluster(void (*fn)(P...), int most, int block, int smem) {
  for (; most > 1; most /= 2) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(most));
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(most);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg) == cudaSuccess && clusters > 0) break;
    cudaGetLastError();
  }
  return most;
}

template <int D>
static cudaError_t launch_compact_d(const CompactParams& p, int num_sms, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(p.c.B) * p.c.heads * 2;
  const int page = 1 << p.c.page_shift;
  // Half of 16 sequences of 8192 tokens kept, 8 heads of 128: 62 us with waves of 256 tokens and one CTA
  // per sequence, head and pool, 74 of 128, 68 of 128 and two CTAs, 83 of 256 and two.  30011 of 100001
  // tokens, 2 heads of 64, 16 CTAs: 18.8 us of 256, 27.5 of 128; 33 with 8 CTAs.
  const int wave = p.max_tokens > 64 ? kMostWave : page > 64 ? page : 64;
  static thread_local int set_on = -1, most = 1;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (set_on != dev) {
    e = cudaFuncSetAttribute(compact_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kMostWave * D);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(compact_kernel<D>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    most = resident_cluster(compact_kernel<D>, kMostCompactCluster, kCompactThreads, 2 * kMostWave * D);
    set_on = dev;
  }
  const int ctas = compact_ctas(items, wave, p.max_tokens, num_sms, most);
  const int buffers = page - 1 + static_cast<int64_t>(p.max_tokens) > static_cast<int64_t>(wave) * ctas ? 2 : 1;
  const int smem = buffers * wave * D;
  return launch_early_clusters(compact_kernel<D>, items * ctas, ctas, kCompactThreads, smem, s, p, wave, buffers);
}

cudaError_t launch_compact(const CompactParams& p, int num_sms, cudaStream_t s) {
  switch (p.c.D) {
    case 64: return launch_compact_d<64>(p, num_sms, s);
    case 96: return launch_compact_d<96>(p, num_sms, s);
    case 128: return launch_compact_d<128>(p, num_sms, s);
    case 192: return launch_compact_d<192>(p, num_sms, s);
    case 256: return launch_compact_d<256>(p, num_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace b2b
