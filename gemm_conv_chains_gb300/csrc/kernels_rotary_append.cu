// kernels_rotary_append.cu -- rotary positions over rows of heads, the cos/sin table, and the
// append of new keys and values to a paged e4m3 cache.
#include "decoder_device.cuh"

namespace b2b {

// ------------------------------------------------------------------------------------
// rotary positions
// ------------------------------------------------------------------------------------
// y_a = x_a c - x_b s, y_b = x_b c + x_a s for each channel pair (a, b) of a head's first
// `rot` channels, (c, s) the table's row of the token's position; the inverse takes -s and
// is also the gradient, the rotation being orthogonal.  Every element is read and written
// once and takes three operations: HBM bound.  A thread owns one 16-byte vector (its
// partner vector too in the half layout), so that both layouts load and store whole
// sectors, and a block owns whole tokens, so that the heads of a token share its table
// row in L1.
template <bool BF16>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryParams p, int units,
                                                     int tokens_per_block) {
  const int row_units_total = p.H * units;
  const bool in_place = p.x == p.out && p.ldx == p.ldo;
  for (int j = threadIdx.x; j < row_units_total * tokens_per_block; j += blockDim.x) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * tokens_per_block + j / row_units_total;
    if (t >= p.T) break;
    const int r = j % row_units_total;
    const int h = r / units, u = r % units;
    const int pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= p.table_len) {
      index_error(p.err, DK_ROTARY, DEC_ERR_POSITION, static_cast<uint32_t>(t));
      continue;
    }
    const uint16_t* row = p.x + t * p.ldx + static_cast<int64_t>(h) * p.D;
    uint16_t* dst = p.out + t * p.ldo + static_cast<int64_t>(h) * p.D;
    if (in_place && (p.interleaved ? 8 * u >= p.rot : u >= p.rot / 16)) continue;
    float lo[8], hi[8];
    bool pair;
    const int d = load_unit<BF16>(row, p.table + static_cast<int64_t>(pos) * (p.rot / 2), u, p.rot,
                                  p.interleaved, p.inverse != 0, lo, hi, pair);
    *reinterpret_cast<uint4*>(dst + d) = narrow8<BF16>(lo);
    if (pair) *reinterpret_cast<uint4*>(dst + d + p.rot / 2) = narrow8<BF16>(hi);
  }
}

cudaError_t launch_rotary(bool bf16, const RotaryParams& p, cudaStream_t s) {
  const int units = p.interleaved ? p.D / 8 : p.rot / 16 + (p.D - p.rot) / 8;
  const int per_token = p.H * units;
  const int tpb = per_token >= 256 ? 1 : 256 / per_token;
  const int64_t blocks = (p.T + tpb - 1) / tpb;
  if (bf16)
    rotary_kernel<true><<<static_cast<unsigned>(blocks), 256, 0, s>>>(p, units, tpb);
  else
    rotary_kernel<false><<<static_cast<unsigned>(blocks), 256, 0, s>>>(p, units, tpb);
  return cudaGetLastError();
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
  rotary_table_kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, s>>>(table, total, half,
                                                                                p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------------------------
// append to the paged e4m3 cache
// ------------------------------------------------------------------------------------
// One block per page that a sequence's new tokens touch, kv head, and pool (keys or
// values); further blocks rotate the queries.  With A the largest finite magnitude of the
// block's new values (keys after the rotation) and s the page's scale if it already holds
// older tokens of the sequence, else 0:
//   s' = max(s, A / 448, 2^-64);  new codes e4m3(y / s'), saturating;
//   older codes e4m3(code * (s / s')) if s' > s, else untouched.
// The new tokens are read twice (the maximum first), the second time from L1 or L2: a page
// of new tokens is at most 128 KB.  The rest is one pass; with one new token per sequence
// a call is bound by its latency (three dependent loads before the first store).
constexpr int kAppendThreads = 128;

template <bool BF16>
__device__ __forceinline__ void append_page(const AppendParams& p, int b, int j, int h, bool value,
                                            float* shared) {
  const CacheView& c = p.c;
  const Sequence s = load_sequence(c, b, DK_APPEND);
  if (s.n == 0) return;
  const int page = 1 << c.page_shift;
  const int start = s.len - s.n;
  const int64_t pi = (start >> c.page_shift) + static_cast<int64_t>(j);
  const int64_t first_slot = pi << c.page_shift;
  if (first_slot >= s.len) return;
  const int64_t lo_tok = first_slot > start ? first_slot : start;
  const int64_t hi_tok = first_slot + page < s.len ? first_slot + page : s.len;
  const int held = first_slot < start ? static_cast<int>(start - first_slot) : 0;
  const int count = static_cast<int>(hi_tok - lo_tok);
  const int id = __ldg(c.page_table + static_cast<int64_t>(b) * c.max_pages + pi);
  if (id < 0 || id >= c.pages) {
    if (threadIdx.x == 0) index_error(c.err, DK_APPEND, DEC_ERR_PAGE, static_cast<uint32_t>(b));
    return;
  }
  const bool rotate = !value && p.table != nullptr;
  if (rotate && hi_tok > p.table_len) {
    if (threadIdx.x == 0) index_error(c.err, DK_APPEND, DEC_ERR_POSITION, static_cast<uint32_t>(b));
    return;
  }
  const int64_t at = static_cast<int64_t>(id) * c.heads + h;
  float* scale_at = (value ? c.v_scale : c.k_scale) + at;
  uint8_t* codes = (value ? c.v : c.k) + (at << c.page_shift) * c.D;
  const float before = held > 0 ? *scale_at : 0.f;

  const int rot = rotate ? p.rot : 0;
  const int inter = rotate ? p.interleaved : 1;       // without a rotation: plain vectors
  const int units = row_units(c.D, rot, inter);
  const int64_t ld = value ? p.ldv : p.ldk;
  const uint16_t* src = (value ? p.v : p.k) +
                        (s.row + (lo_tok - start)) * ld + static_cast<int64_t>(h) * c.D;
  float lo[8], hi[8];
  bool pair = false;
  float most = 0.f;
  const int total = count * units;
  for (int i = threadIdx.x; i < total; i += kAppendThreads) {
    const int tok = i / units, u = i - tok * units;
    load_unit<BF16>(src + tok * ld, p.table + (lo_tok + tok) * (rot / 2), u, rot, inter, false, lo,
                    hi, pair);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = fabsf(lo[e]), z = pair ? fabsf(hi[e]) : 0.f;
      if (a <= 3.402823466e38f) most = fmaxf(most, a);
      if (z <= 3.402823466e38f) most = fmaxf(most, z);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) most = fmaxf(most, shared[w]);
  const float after = fmaxf(fmaxf(before, __fdiv_rn(most, kE4m3Max)), kScaleMin);

  for (int i = threadIdx.x; i < total; i += kAppendThreads) {
    const int tok = i / units, u = i - tok * units;
    const int d = load_unit<BF16>(src + tok * ld, p.table + (lo_tok + tok) * (rot / 2), u, rot,
                                  inter, false, lo, hi, pair);
    uint8_t* dst = codes + static_cast<int64_t>(lo_tok - first_slot + tok) * c.D + d;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = e4m3x2(__fdiv_rn(lo[2 * e], after), __fdiv_rn(lo[2 * e + 1], after));
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    if (pair) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = e4m3x2(__fdiv_rn(hi[2 * e], after), __fdiv_rn(hi[2 * e + 1], after));
      *reinterpret_cast<uint2*>(dst + rot / 2) =
          make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
  }
  if (held > 0 && after > before) {
    const float ratio = __fdiv_rn(before, after);
    uint2* old = reinterpret_cast<uint2*>(codes);
    for (int i = threadIdx.x; i < held * c.D / 8; i += kAppendThreads) {
      uint2 w = old[i];
      uint32_t in[2] = {w.x, w.y}, out[2];
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

// The sequence that row t of the new tokens belongs to: the last b with starts[b] <= t.
__device__ __forceinline__ int sequence_of(const CacheView& c, int64_t t) {
  if (c.starts == nullptr) return static_cast<int>(t / (c.T / c.B));
  int lo = 0, hi = c.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(c.starts + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <bool BF16>
__device__ __forceinline__ void rotate_queries(const AppendParams& p, int64_t t) {
  const CacheView& c = p.c;
  const int b = sequence_of(c, t);
  const Sequence s = load_sequence(c, b, DK_APPEND);
  const int64_t i = t - s.row;
  if (i < 0 || i >= s.n) return;
  const int64_t pos = s.len - s.n + i;
  if (pos >= p.table_len) {
    if (threadIdx.x == 0) index_error(c.err, DK_APPEND, DEC_ERR_POSITION, static_cast<uint32_t>(b));
    return;
  }
  const int units = row_units(c.D, p.rot, p.interleaved);
  const float2* cs = p.table + pos * (p.rot / 2);
  for (int j = threadIdx.x; j < p.q_heads * units; j += kAppendThreads) {
    const int h = j / units, u = j - h * units;
    float lo[8], hi[8];
    bool pair;
    const int d = load_unit<BF16>(p.q + t * p.ldq + static_cast<int64_t>(h) * c.D, cs, u, p.rot,
                                  p.interleaved, false, lo, hi, pair);
    uint16_t* dst = p.q_out + t * p.ldqo + static_cast<int64_t>(h) * c.D + d;
    *reinterpret_cast<uint4*>(dst) = narrow8<BF16>(lo);
    if (pair) *reinterpret_cast<uint4*>(dst + p.rot / 2) = narrow8<BF16>(hi);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p,
                                                                int64_t page_blocks,
                                                                int pages_per_seq) {
  __shared__ float shared[kAppendThreads / 32];
  const int64_t x = blockIdx.x;
  if (x >= page_blocks) {
    rotate_queries<BF16>(p, x - page_blocks);
    return;
  }
  const int value = static_cast<int>(x & 1);
  int64_t r = x >> 1;
  const int h = static_cast<int>(r % p.c.heads);
  r /= p.c.heads;
  append_page<BF16>(p, static_cast<int>(r / pages_per_seq), static_cast<int>(r % pages_per_seq), h,
                    value != 0, shared);
}

cudaError_t launch_append(bool bf16, const AppendParams& p, cudaStream_t s) {
  const int page = 1 << p.c.page_shift;
  // max_new tokens from any slot on touch at most this many pages
  const int per_seq = (p.c.max_new - 1 + page - 1) / page + 1;
  const int64_t page_blocks = static_cast<int64_t>(p.c.B) * per_seq * p.c.heads * 2;
  const int64_t blocks = page_blocks + (p.q != nullptr ? p.c.T : 0);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  if (bf16)
    append_kernel<true><<<static_cast<unsigned>(blocks), kAppendThreads, 0, s>>>(p, page_blocks,
                                                                                 per_seq);
  else
    append_kernel<false><<<static_cast<unsigned>(blocks), kAppendThreads, 0, s>>>(p, page_blocks,
                                                                                  per_seq);
  return cudaGetLastError();
}

}  // namespace b2b
