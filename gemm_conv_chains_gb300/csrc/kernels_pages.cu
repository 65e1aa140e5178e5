// kernels_pages.cu -- the pages of the paged e4m3 cache: the page table of a step's sequences, copies
// of pages, and the tokens that a sequence keeps moved together.
#include "decoder_device.cuh"

namespace b2b {
namespace {

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The address of `local` (shared memory) in the CTA `rank` of this cluster.
__device__ __forceinline__ uint32_t cluster_address(uint32_t local, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t cluster_load(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_store(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_min(uint32_t at, uint32_t v) {
  asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
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
// One cluster (of one CTA for small tables) in four steps with a cluster barrier between them: words
// cleared; old entries copied and words lowered, a warp per row; pages that each row needs, their
// prefix sums (every CTA the same, a thread per row) and each CTA's count of free pages; each free page
// finds the row that takes it.  The words lie in the shared memory of the cluster, or in the
// workspace for pools that are too large for that.  Bound by latency: each step is one or two
// dependent accesses.
constexpr int kPagesThreads = 1024;
constexpr int kPagesCluster = 8;
constexpr int kPagesShared = 40 * 1024;                // words of a CTA
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

// The word of a page.  SHARED: chunks of `chunk` words in the CTAs of the cluster.
template <bool SHARED>
struct Owners {
  uint32_t* global;
  uint32_t shared_at, chunk;
  __device__ __forceinline__ uint32_t at(uint32_t page) const {
    const uint32_t rank = page / chunk;
    return cluster_address(shared_at + 4u * (page - rank * chunk), rank);
  }
  __device__ __forceinline__ void lower(uint32_t page, uint32_t v) const {
    if constexpr (SHARED) cluster_min(at(page), v);
    else atomicMin(global + page, v);
  }
  __device__ __forceinline__ uint32_t load(uint32_t page) const {
    if constexpr (SHARED) return cluster_load(at(page));
    else return __ldcg(global + page);
  }
};

template <bool SHARED>
__global__ void __launch_bounds__(kPagesThreads, 1) pages_kernel(const PagesParams p, uint32_t chunk) {
  extern __shared__ __align__(16) uint32_t pages_smem[];
  __shared__ uint32_t warp_sums[32];
  __shared__ uint32_t free_of[kPagesCluster];          // free pages of each CTA's chunk
  uint32_t* first_rank = pages_smem;                   // [rows]: the first new page's rank
  uint32_t* takes = pages_smem + p.rows;               // [rows]: its slot, and bit 31: it is a copy
  uint32_t* words = pages_smem + 2 * p.rows;           // SHARED: this CTA's chunk
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t pages = static_cast<uint32_t>(p.pages);
  const uint32_t lo = rank * chunk < pages ? rank * chunk : pages;
  const uint32_t hi = lo + chunk < pages ? lo + chunk : pages;
  uint32_t* mine = SHARED ? words : p.owners + lo;
  Owners<SHARED> owners{p.owners, smem_u32(words), chunk};

  begin();
  for (uint32_t i = threadIdx.x; i < hi - lo; i += kPagesThreads) mine[i] = kNobody;
  cluster_sync();

  // ---- a warp per row: its old pages ----
  for (int r = static_cast<int>(rank) * 32 + warp; r < p.rows; r += static_cast<int>(ctas) * 32) {
    const PageRow w = page_row(p, r, lane == 0);
    const int32_t* from = p.table + static_cast<int64_t>(w.parent < 0 ? 0 : w.parent) * p.width;
    int32_t* to = p.table_out + static_cast<int64_t>(r) * p.width;
    for (int j = lane; j < p.width; j += 32) {
      int id = -1;
      if (j < w.have) {
        id = from[j];
        if (id < 0 || id >= p.pages) {
          index_error(p.err, DK_PAGES, DEC_ERR_PAGE, static_cast<uint32_t>(r));
          id = -1;
        } else {
          owners.lower(static_cast<uint32_t>(id),
                       w.writes && j == w.have - 1 ? static_cast<uint32_t>(r) + 1u : 0u);
        }
      }
      to[j] = id;
    }
    if (lane < 3) p.copies[3 * static_cast<int64_t>(r) + lane] = lane < 2 ? -1 : 0;
    if (lane == 3) p.lens_out[r] = w.total;
  }
  cluster_sync();

  // ---- the free pages of this CTA's chunk: a warp counts a run of 32 k words ----
  const uint32_t run = ((hi - lo + 32 * 32 - 1) / (32 * 32)) * 32;
  const uint32_t run_lo = warp * run < hi - lo ? warp * run : hi - lo;
  const uint32_t run_hi = run_lo + run < hi - lo ? run_lo + run : hi - lo;
  uint32_t free_here = 0;
  for (uint32_t i = run_lo + lane; i < run_hi; i += 32)
    free_here += (SHARED ? mine[i] : __ldcg(mine + i)) == kNobody ? 1u : 0u;
  free_here = __reduce_add_sync(0xffffffffu, free_here);
  if (lane == 0) warp_sums[warp] = free_here;
  __syncthreads();
  uint32_t before = 0, here = 0;                       // of the warps ahead, of all
  for (int i = 0; i < 32; ++i) {
    const uint32_t v = warp_sums[i];
    before += i < warp ? v : 0u;
    here += v;
  }
  if (threadIdx.x < ctas) cluster_store(cluster_address(smem_u32(&free_of[rank]), threadIdx.x), here);

  // ---- the pages that each row needs, and the ranks of the first ----
  uint32_t needed = 0;
  for (int r0 = 0; r0 < p.rows; r0 += kPagesThreads) {
    const int r = r0 + static_cast<int>(threadIdx.x);
    uint32_t need = 0, slot = 0;
    bool copy = false;
    if (r < p.rows) {
      const PageRow w = page_row(p, r, false);
      if (w.writes) {
        const int id = p.table[static_cast<int64_t>(w.parent) * p.width + w.have - 1];
        copy = id >= 0 && id < p.pages && owners.load(static_cast<uint32_t>(id)) != static_cast<uint32_t>(r) + 1u;
      }
      slot = static_cast<uint32_t>(w.have) - (copy ? 1u : 0u);
      need = static_cast<uint32_t>((static_cast<int64_t>(w.total) + (1 << p.page_shift) - 1) >> p.page_shift) - slot;
    }
    uint32_t upto = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    __syncthreads();                                   // warp_sums is free
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    uint32_t base = needed;
    for (int i = 0; i < 32; ++i) {
      const uint32_t v = warp_sums[i];
      base += i < warp ? v : 0u;
      needed += v;
    }
    if (r < p.rows) {
      first_rank[r] = base + upto - need;
      takes[r] = slot | (copy ? 0x80000000u : 0u);
    }
  }
  cluster_sync();

  // ---- each free page goes to the row whose ranks hold its own ----
  uint32_t ahead = 0, all = 0;
  for (uint32_t i = 0; i < ctas; ++i) {
    const uint32_t v = free_of[i];
    ahead += i < rank ? v : 0u;
    all += v;
  }
  uint32_t at = ahead + before;
  for (uint32_t i0 = run_lo; i0 < run_hi && at < needed; i0 += 32) {
    const uint32_t i = i0 + lane;
    const bool is_free = i < run_hi && (SHARED ? mine[i] : __ldcg(mine + i)) == kNobody;
    const uint32_t vote = __ballot_sync(0xffffffffu, is_free);
    const uint32_t q = at + __popc(vote & ((1u << lane) - 1u));
    at += __popc(vote);
    if (!is_free || q >= needed) continue;
    int a = 0, z = p.rows - 1;                         // the last row whose first rank is at most q
    while (a < z) {
      const int mid = (a + z + 1) / 2;
      if (first_rank[mid] <= q) a = mid;
      else z = mid - 1;
    }
    const uint32_t k = q - first_rank[a], slot = takes[a] & 0x7FFFFFFFu;
    int32_t* entry = p.table_out + static_cast<int64_t>(a) * p.width + slot + k;
    const int page = static_cast<int>(lo + i);
    if (k == 0 && (takes[a] >> 31) != 0u) {
      int32_t* c = p.copies + 3 * static_cast<int64_t>(a);
      const PageRow w = page_row(p, a, false);
      c[0] = p.table[static_cast<int64_t>(w.parent) * p.width + slot];
      c[1] = page;
      c[2] = w.kept & ((1 << p.page_shift) - 1);
    }
    *entry = page;
  }
  if (rank == 0) {
    // a copy that there is no page for: the row cannot have the old one
    for (int r = threadIdx.x; r < p.rows; r += kPagesThreads)
      if ((takes[r] >> 31) != 0u && first_rank[r] >= all)
        p.table_out[static_cast<int64_t>(r) * p.width + (takes[r] & 0x7FFFFFFFu)] = -1;
    if (threadIdx.x == 0) *p.left = static_cast<int32_t>(all) - static_cast<int32_t>(needed);
  }
}

// ------------------------------------------------------------------------------------
// copies of pages
// ------------------------------------------------------------------------------------
// One block per (copy, pool, head): the first `tokens` tokens of the head's part of a page lie in a row.
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
// scales, three dependent loads, are asked for one, two and three waves ahead, each in a register
// of its token's thread.  Tokens that stay in place are read only where their page's scale grows.
constexpr int kCompactThreads = 256;
constexpr int kMostWave = 256;                         // a page or several
constexpr int kMostCompactCluster = 8;

// What a thread knows of its token of a wave.
struct Moving {
  int from;                                            // its position, -1: none
  int id, to;                                          // the pages of that position and of its own
  float scale;
};

__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const CompactParams p, int wave, int buffers) {
  extern __shared__ __align__(16) uint8_t compact_smem[];          // [buffers][wave][D]
  __shared__ int64_t source[2][kMostWave];             // byte offset of a token's codes in the pool,
                                                       // or -1: none, -2: it stays in place
  __shared__ float had[kMostWave];                     // its scale
  __shared__ int32_t goes[kMostWave / 16];             // the pages that 16 tokens each go to, or -1
  __shared__ uint32_t most[kMostWave / 16];            // of the wave's pages, the largest scale that comes in
  begin();
  const CacheView& c = p.c;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
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
  const int64_t part = static_cast<int64_t>(c.D) << c.page_shift;
  const int units = c.D / 16;                          // vectors of a token
  const uint32_t buffer_at = smem_u32(compact_smem);

  // the position that this thread's token of wave w goes to
  const int64_t base = (first & ~mask) + static_cast<int64_t>(wave) * rank + t;
  const int64_t step = static_cast<int64_t>(wave) * ctas;
  const int waves = static_cast<int>((end - (first & ~mask) + step - 1) / step);
  auto goes_to = [&](int w) -> int64_t { return t < wave && w < waves ? base + w * step : end; };

  auto ask_token = [&](int w, Moving& m) {
    const int64_t dst = goes_to(w);
    m.from = -1;
    if (dst < first) {
      m.from = static_cast<int>(dst);
    } else if (dst < end) {
      const int i = static_cast<int>(dst - first);
      m.from = tokens[i];
      if (m.from < dst || m.from >= len || (i > 0 && tokens[i - 1] >= m.from)) {
        index_error(c.err, DK_COMPACT, DEC_ERR_TOKEN, static_cast<uint32_t>(b));
        m.from = -1;
      }
    }
  };
  auto ask_pages = [&](int w, Moving& m) {
    const int64_t dst = goes_to(w);
    m.id = m.to = -1;
    if (dst < end) {
      m.to = table[dst >> c.page_shift];
      if (m.from >= 0) m.id = table[m.from >> c.page_shift];
      const bool bad = m.to < 0 || m.to >= c.pages || (m.from >= 0 && (m.id < 0 || m.id >= c.pages));
      if (bad) {
        index_error(c.err, DK_COMPACT, DEC_ERR_PAGE, static_cast<uint32_t>(b));
        if (m.to < 0 || m.to >= c.pages) m.to = -1;
        m.id = -1;
      }
      if (m.to < 0) m.id = -1;
    }
  };
  auto ask_scale = [&](Moving& m) {
    m.scale = 0.f;
    if (m.id >= 0) m.scale = scales[static_cast<int64_t>(m.id) * c.heads + h];
  };
  // the tokens of wave w on their way to its buffer
  auto ask_codes = [&](int w, const Moving& m) {
    const int64_t dst = goes_to(w);
    int64_t off = -1;
    if (m.id >= 0)
      off = m.from == dst ? -2 : (static_cast<int64_t>(m.id) * c.heads + h) * part + (m.from & mask) * c.D;
    if (t < wave) source[w & 1][t] = off;
    __syncthreads();
    if (w < waves) {
      const uint32_t to = buffer_at + (buffers > 1 ? (w & 1) * wave * c.D : 0);
      for (int j = t; j < wave * units; j += kCompactThreads) {
        const int tok = j / units;
        const int64_t from = source[w & 1][tok];
        if (from >= 0)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16 * j),
                       "l"(pool + from + 16 * (j - tok * units)) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  Moving now, next, after, far;                        // of waves w, w + 1, w + 2, w + 3
  ask_token(0, now);
  ask_token(1, next);
  ask_token(2, after);
  ask_pages(0, now);
  ask_pages(1, next);
  ask_codes(0, now);
  ask_scale(now);
  for (int w = 0; w < waves; ++w) {
    // (a call of one wave has one buffer)
    ask_codes(w + 1, next);
    ask_scale(next);
    ask_pages(w + 2, after);
    ask_token(w + 3, far);
    if (t < kMostWave / 16) most[t] = 0u;
    if (t < wave) had[t] = now.scale;
    if (t < wave && (t & 15) == 0) goes[t >> 4] = now.to;
    __syncthreads();
    if (now.id >= 0 && now.scale > 0.f) atomicMax(&most[t >> c.page_shift], __float_as_uint(now.scale));
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    cluster_sync();
    // ---- every CTA has the wave's tokens and scales ----
    const uint8_t* held = compact_smem + (buffers > 1 ? (w & 1) * wave * c.D : 0);
    const int64_t at0 = base - t + w * step;
    for (int j = t; j < wave * units; j += kCompactThreads) {
      const int tok = j / units;
      const int64_t from = source[w & 1][tok];
      if (from == -1) continue;
      const float s = __uint_as_float(most[tok >> c.page_shift]);
      if (from == -2 && had[tok] == s) continue;
      const int64_t page_at = static_cast<int64_t>(goes[tok >> 4]) * c.heads + h;
      uint4* dst = reinterpret_cast<uint4*>(pool + page_at * part + ((at0 + tok) & mask) * c.D) + (j - tok * units);
      uint4 v = from == -2 ? *dst : *reinterpret_cast<const uint4*>(held + 16 * j);
      if (had[tok] != s) {
        const float ratio = __fdiv_rn(had[tok], s);
        uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t f0, f1;
          e4m3x4_to_f16(in[e], f0, f1);
          const float2 a = widen2<false>(f0), z = widen2<false>(f1);
          in[e] = e4m3x2(__fmul_rn(a.x, ratio), __fmul_rn(a.y, ratio)) |
                  (e4m3x2(__fmul_rn(z.x, ratio), __fmul_rn(z.y, ratio)) << 16);
        }
        v = make_uint4(in[0], in[1], in[2], in[3]);
      }
      *dst = v;
    }
    if (t < wave && (t & mask) == 0 && now.to >= 0)
      scales[static_cast<int64_t>(now.to) * c.heads + h] = __uint_as_float(most[t >> c.page_shift]);
    __syncthreads();                                   // the buffer, source, had, goes and most are free
    now = next;
    next = after;
    after = far;
  }
}

}  // namespace

static int pages_ctas(int64_t pages, int64_t rows, int64_t width) {
  return pages <= kPagesShared && rows * width <= 16384 ? 1 : kPagesCluster;
}

int64_t pages_workspace(int64_t pages) {
  return pages <= static_cast<int64_t>(kPagesShared) * kPagesCluster ? 0 : 4 * pages;
}

template <bool SHARED>
static cudaError_t launch_pages_in(const PagesParams& p, cudaStream_t s) {
  const int ctas = pages_ctas(p.pages, p.rows, p.width);
  const uint32_t chunk = static_cast<uint32_t>((p.pages + ctas - 1) / ctas > 0 ? (p.pages + ctas - 1) / ctas : 1);
  const int smem = 4 * (2 * p.rows + (SHARED ? static_cast<int>(chunk) : 0));
  constexpr int kMost = 4 * (2 * kMostPageRows + kPagesShared);
  static_assert(kMost <= 227 * 1024 - 1024, "shared memory of one CTA");
  static thread_local int set_on = -1;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (set_on != dev) {
    e = cudaFuncSetAttribute(pages_kernel<SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    set_on = dev;
  }
  return launch_early_clusters(pages_kernel<SHARED>, ctas, ctas, kPagesThreads, smem, s, p, chunk);
}

cudaError_t launch_pages(const PagesParams& p, cudaStream_t s) {
  return p.owners == nullptr ? launch_pages_in<true>(p, s) : launch_pages_in<false>(p, s);
}

cudaError_t launch_copy(const CopyParams& p, int num_sms, cudaStream_t s) {
  const int64_t items = p.n * p.c.heads * 2, most = static_cast<int64_t>(num_sms) * 64;
  return launch_early(copy_kernel, items < most ? items : most, kCopyThreads, 0, s, p);
}

cudaError_t launch_compact(const CompactParams& p, int num_sms, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(p.c.B) * p.c.heads * 2;
  const int page = 1 << p.c.page_shift;
  const int wave = p.max_tokens > 64 ? kMostWave : page > 64 ? page : 64;
  int ctas = 1;
  while (ctas < kMostCompactCluster && items * ctas < num_sms && ctas * wave < p.max_tokens) ctas *= 2;
  const int buffers = page - 1 + static_cast<int64_t>(p.max_tokens) > static_cast<int64_t>(wave) * ctas ? 2 : 1;
  const int smem = buffers * wave * p.c.D;
  static thread_local int set_on = -1;
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (set_on != dev) {
    e = cudaFuncSetAttribute(compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 2 * kMostWave * 256);
    if (e != cudaSuccess) return e;
    set_on = dev;
  }
  return launch_early_clusters(compact_kernel, items * ctas, ctas, kCompactThreads, smem, s, p, wave, buffers);
}

}  // namespace b2b
