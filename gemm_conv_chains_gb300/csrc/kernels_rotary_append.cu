// kernels_rotary_append.cu -- rotary positions over rows of heads, the cos/sin table, and the
// append of new keys and values to a paged e4m3 cache.
#include "decoder_device.cuh"

namespace b2b {

// What a kernel launched early (launch_early) starts with.
__device__ __forceinline__ void begin() {
  grid_launch_dependents();
  grid_dependency_wait();
}

// ------------------------------------------------------------------------------------
// rows of heads turned: rotary positions, and the queries of an append
// ------------------------------------------------------------------------------------
// y_a = x_a c - x_b s, y_b = x_b c + x_a s for each channel pair (a, b) of a head's first
// `rot` channels, (c, s) the table's row of the token's position; the inverse takes -s and
// is also the gradient, the rotation being orthogonal.  Every element is read and written
// once and takes two operations: HBM bound, if enough of it is in flight.  A thread keeps one
// unit of a row (16 bytes, or two times 16 that are partners in the half layout; whole sectors
// either way) for all the heads and tokens that it walks, its angles in registers, and copies
// what it will turn into a ring of its own in shared memory, kAhead units ahead (cp.async, no
// barrier: it reads back what it copied itself).  16384 tokens of 40 heads of 128 take 54 us so,
// 6.2 TB/s, 0.92 of the copy rate; one unit per thread, without ring or walk, 66 (and asking for two
// or four units at a time in registers costs as many threads as it gains requests).
constexpr int kTurnThreads = 256;
constexpr int kAhead = 8;

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

struct TurnRows {
  const uint16_t* x;
  uint16_t* out;
  const float2* table;
  int64_t ldx, ldo, table_len;
  int H, D, rot, interleaved;
  float sign;
};

// One unit per thread and step, straight from global to global memory: few registers, so that
// many threads hide the latency of short calls.
template <bool BF16>
__device__ __forceinline__ void turn_one(const TurnRows& r, int64_t t, int h, int u, int pos) {
  const UnitAt at = unit_at(u, r.rot, r.interleaved);
  if (!at.turned && r.x == r.out && r.ldx == r.ldo) return;      // in place: nothing to copy
  const RawUnit raw = load_raw(r.x + t * r.ldx + static_cast<int64_t>(h) * r.D, at, r.rot);
  const AngleRow g = angle_row(r.table + static_cast<int64_t>(pos) * (r.rot / 2), at, r.interleaved);
  store_turned<BF16>(r.out + t * r.ldo + static_cast<int64_t>(h) * r.D, raw, at, g, r.rot,
                     r.interleaved, r.sign);
}

// Turns rows [t0, t1); position(t) gives a row's position, or -1 for a row to leave out.  Threads:
// (units, groups of heads, rows side by side where they are short) in x, idle beyond.
template <bool BF16, class Position>
__device__ __forceinline__ void turn_rows(const TurnRows& r, int64_t t0, int64_t t1, int units,
                                          int G, Position position) {
  extern __shared__ __align__(16) uint4 ring[];
  const int Z = static_cast<int>(blockDim.x) / units / G;        // rows side by side
  const int group = static_cast<int>(threadIdx.x) / units;
  const int z = group / G, first = group - z * G;
  const UnitAt at = unit_at(threadIdx.x - group * units, r.rot, r.interleaved);
  const bool in_place = r.x == r.out && r.ldx == r.ldo;
  if (z >= Z || (in_place && !at.turned)) return;
  t0 += z;
  const int mine = (r.H - first + G - 1) / G;                    // heads of this thread per row
  const int64_t step = static_cast<int64_t>(G) * r.D;
  const uint32_t ring_at = smem_u32(ring) + threadIdx.x * 16;
  const uint32_t part = blockDim.x * 16;

  int64_t row = t0;                                              // of the next unit to copy
  int k = 0, slot = 0;
  const uint16_t* src = r.x + t0 * r.ldx + static_cast<int64_t>(first) * r.D + at.d;
  auto copy = [&]() {
    if (row < t1) {
      const uint32_t dst = ring_at + slot * 2 * part;
      copy16(dst, src);
      if (at.pair) copy16(dst + part, src + r.rot / 2);
      src += step;
      if (++k == mine) {
        k = 0;
        src += Z * r.ldx - mine * step;
        row += Z;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    slot = slot + 1 == kAhead ? 0 : slot + 1;
  };
#pragma unroll 1
  for (int i = 0; i < kAhead - 1; ++i) copy();

  int pos = t0 < t1 ? position(t0) : -1;
  int read = 0;
  for (int64_t t = t0; t < t1; t += Z) {
    Angles g;
    if (pos >= 0) g = load_angles(r.table + static_cast<int64_t>(pos) * (r.rot / 2), at, r.interleaved);
    const int next = t + Z < t1 ? position(t + Z) : -1;
    uint16_t* dst = r.out + t * r.ldo + static_cast<int64_t>(first) * r.D;
    for (int j = 0; j < mine; ++j, dst += step) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 2) : "memory");
      RawUnit raw;
      raw.lo = ring[threadIdx.x + read * 2 * blockDim.x];
      raw.hi = at.pair ? ring[threadIdx.x + (read * 2 + 1) * blockDim.x] : raw.lo;
      read = read + 1 == kAhead ? 0 : read + 1;
      if (pos >= 0) store_turned<BF16>(dst, raw, at, g, r.rot, r.interleaved, r.sign);
      copy();
    }
    pos = next;
  }
}

// Threads and shared memory of a block that turns rows of H heads.
int turn_units(int D, int rot, int interleaved) {
  return interleaved ? D / 8 : rot / 16 + (D - rot) / 8;
}
constexpr int kTurnSmem = kAhead * 2 * kTurnThreads * 16;

// How a call is cut for the walk: heads of a row side by side in a block, and rows per block (0:
// no walk).  A thread takes at least 8 heads of a row, so that its angles, which come from a
// dependent load, serve 8 units; of the splits that allow it, the one that leaves the fewest
// threads idle, and then the widest.  Six waves of blocks: the SMs do not finish alike, and blocks
// of one full wave ran 93 us where these run 82 (32768 rows of 32 heads of 128).  Where a wave
// leaves a thread fewer than 8 units, one unit per thread is faster (16384 rows of 12 heads of 64:
// 11.2 us against 12.1; 8192 rows of 32 heads of 128: 27.0 against 24.8, 16384 of 40: 66 against 54).
struct Walk {
  int heads;
  int64_t rows;
};
constexpr int kWalkCtas = 3;           // per SM, what the rings leave room for
Walk walk_of(int64_t T, int H, int units, int num_sms) {
  constexpr int kLeast = 8, kWaves = 6;
  const int64_t slots = static_cast<int64_t>(num_sms) * kWalkCtas;
  if (T * H * units < kLeast * slots * kTurnThreads) return Walk{1, 0};
  const int groups = kTurnThreads / units;
  int heads = 1, most = 0;
  for (int G = 1; G <= groups && (G == 1 || (H + G - 1) / G >= kLeast); ++G) {
    const int64_t mine = (H + G - 1) / G;
    const int busy = static_cast<int>(int64_t{1024} * H / (mine * G) * (groups / G * G) / groups);
    if (busy >= most) most = busy, heads = G;
  }
  const int Z = groups / heads;        // rows side by side
  const int64_t rows = (T + slots * kWaves - 1) / (slots * kWaves);
  return Walk{heads, (rows + Z - 1) / Z * Z};
}

// position(t) of rotary: the given one, if the table has it.
__device__ __forceinline__ int rotary_position(const RotaryParams& p, int64_t t) {
  const int pos = p.positions[t];
  if (pos >= 0 && pos < p.table_len) return pos;
  index_error(p.err, DK_ROTARY, DEC_ERR_POSITION, static_cast<uint32_t>(t));
  return -1;
}

__device__ __forceinline__ TurnRows rows_of(const RotaryParams& p) {
  return TurnRows{p.x, p.out, p.table, p.ldx, p.ldo, p.table_len, p.H, p.D, p.rot, p.interleaved,
                  p.inverse ? -1.f : 1.f};
}

template <bool BF16>
__global__ void __launch_bounds__(kTurnThreads, kWalkCtas) rotary_walk_kernel(const RotaryParams p, int units,
                                                                      int heads, int64_t rows) {
  begin();
  const int64_t t0 = blockIdx.x * rows, t1 = t0 + rows < p.T ? t0 + rows : p.T;
  turn_rows<BF16>(rows_of(p), t0, t1, units, heads, [&](int64_t t) { return rotary_position(p, t); });
}

template <bool BF16>
__global__ void __launch_bounds__(kTurnThreads) rotary_kernel(const RotaryParams p, int units,
                                                              int tokens_per_block) {
  begin();
  const int per_token = p.H * units;
  for (int j = threadIdx.x; j < per_token * tokens_per_block; j += blockDim.x) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * tokens_per_block + j / per_token;
    if (t >= p.T) break;
    const int q = j % per_token;
    const int pos = rotary_position(p, t);
    if (pos >= 0) turn_one<BF16>(rows_of(p), t, q / units, q % units, pos);
  }
}

// Lets a kernel use `bytes` of dynamic shared memory on the current device.
cudaError_t allow_smem(const void* fn, int bytes, int& set_on) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || set_on == dev) return e;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) set_on = dev;
  return e;
}

cudaError_t launch_rotary(bool bf16, const RotaryParams& p, int num_sms, cudaStream_t s) {
  const int units = turn_units(p.D, p.rot, p.interleaved);
  if (units > kTurnThreads) return cudaErrorInvalidConfiguration;
  if (const Walk w = walk_of(p.T, p.H, units, num_sms); w.rows > 0) {
    static thread_local int set_on[2] = {-1, -1};
    auto* fn = bf16 ? rotary_walk_kernel<true> : rotary_walk_kernel<false>;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), kTurnSmem, set_on[bf16]);
        e != cudaSuccess)
      return e;
    return launch_early(fn, (p.T + w.rows - 1) / w.rows, kTurnThreads, kTurnSmem, s, p, units, w.heads,
                        w.rows);
  }
  const int per_token = p.H * units;
  const int tpb = per_token >= kTurnThreads ? 1 : kTurnThreads / per_token;
  return launch_early(bf16 ? rotary_kernel<true> : rotary_kernel<false>, (p.T + tpb - 1) / tpb,
                      kTurnThreads, 0, s, p, units, tpb);
}

// The table: (cos, sin) of position * frequency in fp64, rounded once to fp32.  params:
// {base, rot, kind, factor, low, high, gain}; frequency of pair i: base^(-2i/rot), scaled
//   kind 1 (linear)  / factor
//   kind 2 (blend)   pairs that turn more than `high` times over the original length keep
//                    their frequency, those that turn fewer than `low` times take it
//                    / factor, and between the two the share of the first falls linearly;
//                    (cos, sin) are multiplied by `gain`
// A changed base (kind 0 with another base) is a caller's own choice of base.
struct TableParams {
  double base, rot, kind, factor, low, high, gain;
  double original;
};

__global__ void __launch_bounds__(256) rotary_table_kernel(float2* table, int64_t total, int half,
                                                           const TableParams p) {
  begin();
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= total) return;
  const int64_t pos = idx / half;
  const int i = static_cast<int>(idx % half);
  double f = pow(p.base, -2.0 * i / p.rot);
  if (p.kind == 1.0) {
    f /= p.factor;
  } else if (p.kind == 2.0) {
    const double turns = p.original * f / 6.283185307179586;
    double keep = (turns - p.low) / (p.high - p.low);
    keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
    f = keep * f + (1.0 - keep) * f / p.factor;
  }
  double sn, cs;
  sincos(static_cast<double>(pos) * f, &sn, &cs);
  table[idx] = make_float2(static_cast<float>(cs * p.gain), static_cast<float>(sn * p.gain));
}

cudaError_t launch_rotary_table(float2* table, int64_t n, int32_t half, const double* v,
                                cudaStream_t s) {
  TableParams p{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
  const int64_t total = n * half;
  return launch_early(rotary_table_kernel, (total + 255) / 256, 256, 0, s, table, total, half, p);
}

// ------------------------------------------------------------------------------------
// append to the paged e4m3 cache
// ------------------------------------------------------------------------------------
// One block per page that a sequence's new tokens touch, kv head, and pool (keys or
// values).  With A the largest finite magnitude of the block's new values (keys after the
// rotation) and s the page's scale if it already holds older tokens of the sequence, else 0:
//   s' = max(s, A / 448, 2^-64);  new codes e4m3(y / s'), saturating (where s' is A / 448, the
//   quotient is y 448 / A, without the rounding of s': an exact tie between two codes, frequent in
//   values of 8 or 11 bits, stays one and goes to even);
//   older codes e4m3(code * (s / s')) if s' > s, else untouched.
// A thread keeps one unit of a row, asks for its first tokens' along with the page number and holds
// them between the maximum and the codes; what a page has beyond that is read twice, in batches, the
// second time from L1 or L2.  One new token per sequence is bound by the latency of its dependent loads
// (sequence, page number and tokens, scale); prompts by their instructions, 0.74 of the
// issue slots (ragged prompts, 18 k tokens, 8 heads of 128, pages of 32: 72 us with an index
// division per unit and an exact division per element, 44 us so; fewer blocks of several heads each,
// larger blocks, or more of them on fewer registers: 2 to 25 % slower).
// The queries of few tokens are turned by further blocks of the same launch; those of many by a
// launch of the walk above.
constexpr int kAppendThreads = 128;

// The largest magnitude (a NaN is none), or only of the finite ones.
template <bool FINITE>
__device__ __forceinline__ void most_of(const float (&v)[8], float& most) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float a = fabsf(v[e]);
    if (!FINITE || a <= 3.402823466e38f) most = fmaxf(most, a);
  }
}

// What values are divided by on the way to their codes: code = (y * up) / by.
struct Divisor {
  float up, by, inv;
};
// Eight values as codes.  FINITE: the quotients by the reciprocal, each corrected once by its
// residual q s - y (Markstein's step; with this sign -0 stays -0), which rounds like the quotient
// itself and not like the product; an infinity has no residual and takes the exact division.
template <bool FINITE>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&v)[8], const Divisor& s) {
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = v[e] * s.up;
    if (FINITE) {
      q[e] = y * s.inv;
      q[e] = fmaf(fmaf(q[e], s.by, -y), -s.inv, q[e]);
    } else {
      q[e] = __fdiv_rn(y, s.by);
    }
  }
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = e4m3x2(q[2 * e], q[2 * e + 1]);
  *reinterpret_cast<uint2*>(dst) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The block's maximum of a value per thread.
__device__ __forceinline__ float block_max(float v) {
  __shared__ float shared[kAppendThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) v = fmaxf(v, shared[w]);
  return v;
}

// ROTATION: 0 none (values, or keys as they are), 1 interleaved, 2 half.  Each is compiled by
// itself: the pairs of the half layout alone hold twice the registers.
template <bool BF16, int ROTATION>
__device__ __forceinline__ void append_page(const AppendParams& p, int b, int j, int h, bool value) {
  const CacheView& c = p.c;
  const Sequence s = load_sequence(c, b, DK_APPEND);
  if (s.n == 0) return;
  const int page = 1 << c.page_shift;
  const int start = s.len - s.n;
  const int first_page = start >> c.page_shift;
  if (j > ((s.len - 1) >> c.page_shift) - first_page) return;
  const int pi = first_page + j;
  const int first_slot = pi << c.page_shift;
  const int lo_tok = first_slot > start ? first_slot : start;
  const int hi_tok = s.len - first_slot > page ? first_slot + page : s.len;
  const int held = first_slot < start ? start - first_slot : 0;
  const int id = c.page_table[static_cast<int64_t>(b) * c.max_pages + pi];
  const int rot = ROTATION != 0 ? p.rot : 0;
  constexpr int inter = ROTATION != 2;                // without a rotation: plain vectors
  const int units = row_units(c.D, rot, inter);
  const int64_t ld = value ? p.ldv : p.ldk;
  const uint16_t* src = (value ? p.v : p.k) + (s.row + (lo_tok - start)) * ld +
                        static_cast<int64_t>(h) * c.D;
  const float2* cs = p.table + static_cast<int64_t>(lo_tok) * (rot / 2);
  // this thread's unit of every row, and its tokens first, first + G, ...
  const int G = kAppendThreads / units, first = static_cast<int>(threadIdx.x) / units;
  UnitAt at = unit_at(threadIdx.x - first * units, rot, inter);
  if (ROTATION == 0) at.turned = false;
  if (ROTATION != 2) at.pair = false;
  const int count = first < G ? hi_tok - lo_tok : 0;
  // a batch of them is in registers at a time; the first is asked for together with the page number
  constexpr int kHeld = ROTATION == 2 ? 2 : 4;        // a pair unit is two vectors
  RawUnit held_raw[kHeld];
  auto ask = [&](int batch) {
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      const int tok = first + (batch * kHeld + k) * G;
      if (tok < count) held_raw[k] = load_raw(src + tok * ld, at, rot);
    }
  };
  ask(0);
  if (id < 0 || id >= c.pages) {
    if (threadIdx.x == 0) index_error(c.err, DK_APPEND, DEC_ERR_PAGE, static_cast<uint32_t>(b));
    return;
  }
  if (ROTATION != 0 && hi_tok > p.table_len) {
    if (threadIdx.x == 0) index_error(c.err, DK_APPEND, DEC_ERR_POSITION, static_cast<uint32_t>(b));
    return;
  }
  const int64_t page_at = static_cast<int64_t>(id) * c.heads + h;
  float* scale_at = (value ? c.v_scale : c.k_scale) + page_at;
  uint8_t* codes = (value ? c.v : c.k) + (page_at << c.page_shift) * c.D;
  const float before = held > 0 ? *scale_at : 0.f;

  // this thread's units, turned: f(token, lo, hi); every other time from the last batch to the first,
  // so that each pass begins with the one that the last pass ended with
  const int batches = (hi_tok - lo_tok + kHeld * G - 1) / (kHeld * G);
  int batch = 0, step = 1;
  auto each = [&](auto f) {
    float lo[8], hi[8];
#pragma unroll 1
    for (int i = 0;;) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const int tok = first + (batch * kHeld + k) * G;
        if (tok >= count) break;
        turn_unit<BF16>(held_raw[k], at, angle_row(cs + tok * (rot / 2), at, inter), inter, 1.f, lo, hi);
        f(tok, lo, hi);
      }
      if (++i == batches) break;
      batch += step;
      ask(batch);
    }
    step = -step;
  };
  float most = 0.f;
  each([&](int, const float (&lo)[8], const float (&hi)[8]) {
    most_of<false>(lo, most);
    if (at.pair) most_of<false>(hi, most);
  });
  most = block_max(most);
  const bool finite = most <= 3.402823466e38f;
  if (!finite) {                                     // an infinity among them: without those, then
    most = 0.f;
    each([&](int, const float (&lo)[8], const float (&hi)[8]) {
      most_of<true>(lo, most);
      if (at.pair) most_of<true>(hi, most);
    });
    most = block_max(most);
  }
  const float fit = __fdiv_rn(most, kE4m3Max);
  const float after = fmaxf(fmaxf(before, fit), kScaleMin);
  // 448 = 0.875 * 2^9: both factors leave 16-bit values exact.  (An equal older scale counts as A's,
  // so that the same call again gives the same codes.)
  Divisor by{1.f, after, 0.f};
  if (after == fit) by = Divisor{0.875f, most * 0.001953125f, 0.f};
  by.inv = __fdiv_rn(1.f, by.by);

  uint8_t* dst = codes + (lo_tok - first_slot) * c.D + at.d;
  if (finite) {
    each([&](int tok, const float (&lo)[8], const float (&hi)[8]) {
      store_codes<true>(dst + tok * c.D, lo, by);
      if (at.pair) store_codes<true>(dst + tok * c.D + rot / 2, hi, by);
    });
  } else {
    each([&](int tok, const float (&lo)[8], const float (&hi)[8]) {
      store_codes<false>(dst + tok * c.D, lo, by);
      if (at.pair) store_codes<false>(dst + tok * c.D + rot / 2, hi, by);
    });
  }
  if (held > 0 && after > before) {
    const float ratio = __fdiv_rn(before, after);
    uint2* old = reinterpret_cast<uint2*>(codes);
    for (int i = threadIdx.x; i < held * c.D / 8; i += kAppendThreads) {
      const uint2 w = old[i];
      const uint32_t in[2] = {w.x, w.y};
      uint32_t out[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t a, z;
        e4m3x4_to_f16(in[e], a, z);
        const float2 fa = widen2<false>(a), fz = widen2<false>(z);
        out[e] = e4m3x2(__fmul_rn(fa.x, ratio), __fmul_rn(fa.y, ratio)) |
                 (e4m3x2(__fmul_rn(fz.x, ratio), __fmul_rn(fz.y, ratio)) << 16);
      }
      old[i] = make_uint2(out[0], out[1]);
    }
  }
  if (threadIdx.x == 0 && after != before) *scale_at = after;
}

// The sequence that row t of the new tokens belongs to: the last b with starts[b] <= t.  Whole
// warp; the loads of a step are independent.
__device__ __forceinline__ int sequence_of(const CacheView& c, int64_t t) {
  if (c.starts == nullptr) return static_cast<int>(t / (c.T / c.B));
  const int lane = threadIdx.x & 31;
  int count = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const bool in = b0 + lane < c.B && c.starts[b0 + lane] <= t;
    const uint32_t vote = __ballot_sync(0xffffffffu, in);
    count += __popc(vote);
    if (vote != 0xffffffffu) break;
  }
  return count > 0 ? count - 1 : 0;
}

// Walks the sequences along ascending rows: the position of row t, or -1.
struct QueryPosition {
  const AppendParams& p;                             // the kernel's own argument
  int b;
  Sequence s;
  __device__ __forceinline__ QueryPosition(const AppendParams& p_, int64_t t0)
      : p(p_), b(sequence_of(p_.c, t0)), s(load_sequence(p_.c, b, DK_APPEND)) {}
  __device__ __forceinline__ int operator()(int64_t t) {
    while (t >= static_cast<int64_t>(s.row) + s.n && b + 1 < p.c.B)
      s = load_sequence(p.c, ++b, DK_APPEND);
    const int64_t i = t - s.row;
    if (i < 0 || i >= s.n) return -1;
    const int pos = static_cast<int>(s.len - s.n + i);
    if (pos < p.table_len) return pos;
    index_error(p.c.err, DK_APPEND, DEC_ERR_POSITION, static_cast<uint32_t>(b));
    return -1;
  }
};

__device__ __forceinline__ TurnRows rows_of(const AppendParams& p) {
  return TurnRows{p.q, p.q_out, p.table, p.ldq, p.ldqo, p.table_len, p.q_heads, p.c.D, p.rot,
                  p.interleaved, 1.f};
}

template <bool BF16>
__global__ void __launch_bounds__(kTurnThreads, kWalkCtas) query_walk_kernel(const AppendParams p, int units,
                                                                     int heads, int64_t rows) {
  begin();
  const int64_t t0 = blockIdx.x * rows, t1 = t0 + rows < p.c.T ? t0 + rows : p.c.T;
  QueryPosition position(p, t0);
  turn_rows<BF16>(rows_of(p), t0, t1, units, heads, [&](int64_t t) { return position(t); });
}

template <bool BF16, int ROTATION>
__global__ void __launch_bounds__(kAppendThreads, 8) append_kernel(const AppendParams p,
                                                                int64_t page_blocks,
                                                                int pages_per_seq) {
  begin();
  const int64_t x = blockIdx.x;
  if (ROTATION != 0 && x >= page_blocks) {           // one token's queries
    const int64_t t = x - page_blocks;
    const int units = row_units(p.c.D, p.rot, p.interleaved);
    QueryPosition position(p, t);
    const int pos = position(t);
    if (pos < 0) return;
    for (int j = threadIdx.x; j < p.q_heads * units; j += kAppendThreads)
      turn_one<BF16>(rows_of(p), t, j / units, j % units, pos);
    return;
  }
  const int value = static_cast<int>(x & 1);
  uint32_t r = static_cast<uint32_t>(x >> 1);
  const int h = static_cast<int>(r % p.c.heads);
  r /= p.c.heads;
  const int b = static_cast<int>(r / pages_per_seq), j = static_cast<int>(r % pages_per_seq);
  if (value) append_page<BF16, 0>(p, b, j, h, true);
  else append_page<BF16, ROTATION>(p, b, j, h, false);
}

cudaError_t launch_append(bool bf16, const AppendParams& p, int num_sms, cudaStream_t s) {
  const int page = 1 << p.c.page_shift;
  // max_new tokens from any slot on touch at most this many pages
  const int per_seq = (p.c.max_new - 1 + page - 1) / page + 1;
  const int64_t page_blocks = static_cast<int64_t>(p.c.B) * per_seq * p.c.heads * 2;
  const int units = turn_units(p.c.D, p.rot, p.interleaved);
  const Walk w = p.q != nullptr ? walk_of(p.c.T, p.q_heads, units, num_sms) : Walk{1, 0};
  const int64_t blocks = page_blocks + (p.q != nullptr && w.rows == 0 ? p.c.T : 0);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  auto* append = p.table == nullptr ? (bf16 ? append_kernel<true, 0> : append_kernel<false, 0>)
                 : p.interleaved    ? (bf16 ? append_kernel<true, 1> : append_kernel<false, 1>)
                                    : (bf16 ? append_kernel<true, 2> : append_kernel<false, 2>);
  if (cudaError_t e = launch_early(append, blocks, kAppendThreads, 0, s, p, page_blocks, per_seq);
      e != cudaSuccess || w.rows == 0)
    return e;
  static thread_local int set_on[2] = {-1, -1};
  auto* fn = bf16 ? query_walk_kernel<true> : query_walk_kernel<false>;
  if (cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), kTurnSmem, set_on[bf16]);
      e != cudaSuccess)
    return e;
  return launch_early(fn, (p.c.T + w.rows - 1) / w.rows, kTurnThreads, kTurnSmem, s, p, units, w.heads,
                      w.rows);
}

}  // namespace b2b
