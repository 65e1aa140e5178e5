// decoder_api.cu -- the extern "C" entry points of the decoder-block operators (declared in
// include/b2b.h): argument checks before anything touches the GPU, the choice of kernel and
// split, and the launches on the caller's stream.  No device memory is allocated here.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "b2b.h"
#include "decoder.h"

namespace b2b {
namespace {

__device__ uint32_t g_decoder_error[4];   // {code, kernel, what, index}

struct DecoderDevice {
  std::once_flag once;
  int num_sms = 0;
  uint32_t* err = nullptr;
  cudaError_t init_error = cudaSuccess;
};
constexpr int kMaxDecoderDevices = 64;
DecoderDevice g_decoder_dev[kMaxDecoderDevices];

DecoderDevice* decoder_device() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDecoderDevices) {
    cudaGetLastError();
    return nullptr;
  }
  DecoderDevice& d = g_decoder_dev[dev];
  std::call_once(d.once, [&d, dev] {
    d.init_error = cudaDeviceGetAttribute(&d.num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (d.init_error == cudaSuccess)
      d.init_error = cudaGetSymbolAddress(reinterpret_cast<void**>(&d.err), g_decoder_error);
    if (d.init_error != cudaSuccess) cudaGetLastError();
  });
  return d.init_error == cudaSuccess ? &d : nullptr;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

b2b_status launched(cudaError_t e) {
  if (e == cudaSuccess) return B2B_OK;
  cudaGetLastError();
  return B2B_ERR_CUDA;
}

constexpr int64_t kMostRows = int64_t{1} << 30;

bool head_size(int32_t D) { return D == 64 || D == 96 || D == 128 || D == 192 || D == 256; }

b2b_status check_rot(int32_t D, int32_t rot, int32_t layout) {
  if (layout != B2B_ROTARY_HALF && layout != B2B_ROTARY_INTERLEAVED) return B2B_ERR_UNSUPPORTED;
  if (rot <= 0 || rot > D) return B2B_ERR_SHAPE;
  if (rot % 16 != 0) return B2B_ERR_ALIGN;
  return B2B_OK;
}

// A row stride of `ld` elements for rows of n elements.
b2b_status check_ld(int64_t ld, int64_t n) {
  if (ld < n) return B2B_ERR_SHAPE;
  return ld % 8 == 0 ? B2B_OK : B2B_ERR_ALIGN;
}

// T rows of n 16-bit elements, ld apart.
struct RowSet {
  const void* at;
  int64_t ld, n;
};
// Whether a row of one is written while a row of the other may still have to be read.  Usually the two
// lie apart as a whole; rows of one buffer (its columns side by side) are looked at row by row.
bool overlap(const RowSet& a, const RowSet& b, int64_t T) {
  // differences of addresses in elements; both are 16-byte aligned
  const int64_t b0 = (static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at)) -
                      static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.at))) / 2;
  const int64_t a_end = (T - 1) * a.ld + a.n, b_end = b0 + (T - 1) * b.ld + b.n;
  if (b0 >= a_end || b_end <= 0) return false;
  if (a.ld == b.ld) {                        // row t of one against rows t + d of the other
    const int64_t d = b0 >= 0 ? b0 / a.ld : -((a.ld - 1 - b0) / a.ld), rest = b0 - d * a.ld;
    return (rest < a.n && d < T && d > -T) || (rest + b.n > a.ld && d + 1 < T && d + 1 > -T);
  }
  for (int64_t t = 0; t < T; ++t) {
    const int64_t lo = t * a.ld - b0, hi = lo + a.n;         // row t of a, in b's elements
    if (hi <= 0) continue;
    const int64_t first = lo < b.n ? 0 : (lo - b.n) / b.ld + 1;   // the first row of b that ends past lo
    if (first >= T) break;
    if (first * b.ld < hi) return true;
  }
  return false;
}
bool same_rows(const RowSet& a, const RowSet& b, int64_t T) {
  return a.at == b.at && (a.ld == b.ld || T == 1) && a.n == b.n;
}

b2b_status check_cache(const b2b_cache* c, int64_t T) {
  if (c == nullptr) return B2B_ERR_NULL;
  if (c->pages < 0 || c->heads <= 0 || c->batch < 0 || c->max_pages < 0 || c->max_new < 0 || T < 0)
    return B2B_ERR_SHAPE;
  if (!head_size(c->head_dim)) return B2B_ERR_UNSUPPORTED;
  const int32_t ps = c->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1)) != 0) return B2B_ERR_UNSUPPORTED;
  if (c->pages > (int64_t{1} << 30) || c->heads > 65536 || T > kMostRows) return B2B_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->max_pages) * ps > 0x7FFFFFFF - 4096) return B2B_ERR_UNSUPPORTED;
  if (T == 0 || c->batch == 0) return T == 0 ? B2B_OK : B2B_ERR_SHAPE;
  if (c->starts == nullptr && T % c->batch != 0) return B2B_ERR_SHAPE;
  if (c->max_new < (c->starts == nullptr ? T / c->batch : 1) || c->max_new > T) return B2B_ERR_SHAPE;
  if (c->pages == 0 || c->max_pages == 0) return B2B_ERR_SHAPE;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->page_table || !c->lens) return B2B_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->page_table, 4) || !aligned(c->lens, 4) || !aligned(c->starts, 4))
    return B2B_ERR_ALIGN;
  return B2B_OK;
}

CacheView view_of(const b2b_cache* c, int64_t T, uint32_t* err) {
  CacheView v;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.page_table = c->page_table;
  v.lens = c->lens;
  v.starts = c->starts;
  v.T = T;
  v.pages = static_cast<int32_t>(c->pages);
  v.heads = c->heads;
  v.page_shift = __builtin_ctz(static_cast<unsigned>(c->page_size));
  v.D = c->head_dim;
  v.B = c->batch;
  v.max_pages = c->max_pages;
  v.max_new = c->max_new;
  v.err = err;
  return v;
}

// How the split kernel runs a call: row tiles of 8 nt rows, the grid, whether row tiles are
// cut along the context, and the workspace that this takes.
struct SplitChoice {
  int nt, grid, whole, prompt;
  int64_t bytes;
};

// The shortest run of 64-token tiles that gets a CTA of its own.  1 sequence of 1500 tokens, 32 query
// heads on 8 of 128: 11.3 us with runs of 8 tiles, 9.8 of 4, 9.3 of 2; 8 sequences of 1000: 12.5,
// 11.5, 13.2.
constexpr int kMinTiles = 4;
// Contexts of up to this many tokens (a page table's room) are not cut, which saves the joining
// kernel: 1 sequence of 700 tokens, 4 heads of 64: 8.5 us whole, 11.0 cut; 8 sequences of 1000
// tokens, 8 kv heads of 128: 12.0 whole, 11.5 cut.
constexpr int kWholeTokens = 768;

// Whether the tcgen05 kernel takes a call, `rows` query rows per sequence and kv head.  Its time goes
// with the key tiles of the longest unit (256 rows of one sequence and head) and the waves of units
// over the SMs: 1.85 us per 128 keys (1.45 where a unit has only one row tile), whatever the head
// size, latency between its softmax and its products.  The split kernel's goes with all the work,
// cut evenly over the SMs: per 32 rows and 128 keys 7.5 ns at head size 128, 5.1 at 64.  (Fitted over 1,
// 4 and 16 sequences of 300 to 30000 tokens on forms of the kernels that have since become 3 to 6 %
// slower, the split one, and 6 to 15 % faster, the tcgen05 one.)  Measured on 8 kv heads of 128, 4
// query heads each, as the kernels are:
//   1 sequence,   128 new tokens, 4000 cached: split  59 us, tcgen05  65
//   1 sequence,   256 new tokens, 4000 cached: split 100 us, tcgen05  66
//   4 sequences,   33 new tokens, 4000 cached: split  66 us, tcgen05  59
//   16 sequences, 128 new tokens, 4000 cached: split 649 us, tcgen05 143
// The split kernel also has the longer start and a second launch: it has to be 15 % ahead.  On
// contexts of up to 512 tokens, where it does not cut sequences, it falls behind earlier.  (Rows and
// contexts are those that max_new and the page table leave room for: the host knows no others.)
bool prompt_pays(int32_t D, int64_t rows, int64_t heads, bool few_keys, int num_sms) {
  if (D > 128 || rows <= 32) return false;
  const double pieces = static_cast<double>((rows + 31) / 32) * heads;      // of the split kernel
  if (few_keys) return pieces >= 150;
  const double units = static_cast<double>((rows + 255) / 256) * heads;
  const double waves = units > num_sms ? units / num_sms : 1.0;
  const double split_ns = D == 64 ? 5.1 : D == 96 ? 6.3 : 7.5;
  return pieces * split_ns >= 0.85 * waves * (rows <= 128 ? 1450.0 : 1850.0);
}

// The limit of each on-chip wait of the tcgen05 kernel.
constexpr uint64_t kDecoderWaitNs = 1000000000ull;

SplitChoice split_of(const b2b_cache* c, int32_t q_heads, int num_sms) {
  SplitChoice s;
  const int64_t rows = static_cast<int64_t>(c->max_new) * (q_heads / c->heads);
  s.nt = rows <= 8 ? 1 : rows <= 16 || c->head_dim > 128 ? 2 : 4;
  s.grid = attend_ctas_per_sm(c->head_dim, s.nt) * num_sms;
  const int64_t most = static_cast<int64_t>(c->max_pages) * c->page_size;
  s.whole = most <= kWholeTokens ? 1 : 0;
  // no more CTAs than there can be runs
  const int64_t pieces = (rows + 8 * s.nt - 1) / (8 * s.nt) * c->heads * c->batch;
  const int64_t runs = s.whole ? pieces : pieces * ((most / 64 + kMinTiles - 1) / kMinTiles);
  if (runs < s.grid) s.grid = static_cast<int>(runs);
  s.prompt = prompt_pays(c->head_dim, rows, static_cast<int64_t>(c->batch) * c->heads, most <= 512,
                         num_sms);
  s.bytes = s.prompt  ? prompt_workspace(rows, c->batch)
            : s.whole ? 0
                    : 16 * ((static_cast<int64_t>(c->batch) + 4) / 4) +
                          static_cast<int64_t>(s.grid) * 2 * s.nt * 8 * (c->head_dim + 1) * 4;
  return s;
}

b2b_status check_attention(const b2b_cache* c, int64_t T, int32_t q_heads, float scale,
                           float softcap) {
  if (b2b_status st = check_cache(c, T); st != B2B_OK) return st;
  if (q_heads <= 0 || q_heads % c->heads != 0) return B2B_ERR_SHAPE;
  if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f) return B2B_ERR_SHAPE;
  const int64_t rows = static_cast<int64_t>(c->max_new) * q_heads;
  if (q_heads > 65536 || rows > kMostRows || rows * (c->batch > 0 ? c->batch : 1) > 0x7FFFFFFF)
    return B2B_ERR_UNSUPPORTED;
  // the split kernel numbers its work, (8 query rows, 64 tokens) at the finest, in 32 bits
  const double tiles = std::ceil(static_cast<double>(c->max_pages) * c->page_size / 64) *
                       std::ceil(static_cast<double>(rows) / c->heads / 8) * c->heads * c->batch;
  if (tiles > 2.0e9) return B2B_ERR_UNSUPPORTED;
  return B2B_OK;
}

}  // namespace
}  // namespace b2b

using namespace b2b;

extern "C" {

b2b_status b2b_rotary_table(int64_t positions, int32_t rot, double base, b2b_rotary_scaling scaling,
                            double factor, int64_t original, double low, double high, double gain,
                            float* table, void* stream) {
  if (scaling < B2B_ROTARY_PLAIN || scaling > B2B_ROTARY_BLEND) return B2B_ERR_UNSUPPORTED;
  if (positions < 0 || rot <= 0) return B2B_ERR_SHAPE;
  if (rot % 16 != 0) return B2B_ERR_ALIGN;
  if (!(base > 0) || !std::isfinite(base) || !(factor > 0) || !std::isfinite(factor) ||
      !std::isfinite(gain))
    return B2B_ERR_SHAPE;
  if (scaling == B2B_ROTARY_BLEND &&
      (original <= 0 || !std::isfinite(low) || !std::isfinite(high) || !(high > low)))
    return B2B_ERR_SHAPE;
  if (positions > (int64_t{1} << 38) / rot) return B2B_ERR_UNSUPPORTED;
  if (positions == 0) return B2B_OK;
  if (!table) return B2B_ERR_NULL;
  if (!aligned(table, 16)) return B2B_ERR_ALIGN;
  if (decoder_device() == nullptr) return B2B_ERR_CUDA;
  const double v[8] = {base, static_cast<double>(rot), static_cast<double>(scaling), factor,
                       low,  high, gain, static_cast<double>(original)};
  return launched(launch_rotary_table(reinterpret_cast<float2*>(table), positions, rot / 2, v,
                                      static_cast<cudaStream_t>(stream)));
}

b2b_status b2b_rotary(b2b_dtype dt, int64_t T, int32_t H, int32_t D, int32_t rot,
                      b2b_rotary_layout layout, int32_t inverse, const void* x, int64_t ldx,
                      const float* table, int64_t positions_in_table, const int32_t* positions,
                      void* out, int64_t ldo, void* stream) {
  if ((dt != B2B_F16 && dt != B2B_BF16) || (inverse != 0 && inverse != 1)) return B2B_ERR_UNSUPPORTED;
  if (T < 0 || H <= 0 || D <= 0 || positions_in_table < 0) return B2B_ERR_SHAPE;
  if (D % 8 != 0) return B2B_ERR_ALIGN;
  if (b2b_status st = check_rot(D, rot, layout); st != B2B_OK) return st;
  if (T > kMostRows || D > 2048 || static_cast<int64_t>(H) * D > (int64_t{1} << 27))
    return B2B_ERR_UNSUPPORTED;
  if (b2b_status st = check_ld(ldx, static_cast<int64_t>(H) * D); st != B2B_OK) return st;
  if (b2b_status st = check_ld(ldo, static_cast<int64_t>(H) * D); st != B2B_OK) return st;
  if (T == 0) return B2B_OK;
  if (!x || !out || !table || !positions) return B2B_ERR_NULL;
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(table, 16) || !aligned(positions, 4))
    return B2B_ERR_ALIGN;
  DecoderDevice* d = decoder_device();
  if (d == nullptr) return B2B_ERR_CUDA;
  const RowSet in{x, ldx, static_cast<int64_t>(H) * D}, to{out, ldo, static_cast<int64_t>(H) * D};
  if (!same_rows(in, to, T) && overlap(in, to, T)) return B2B_ERR_UNSUPPORTED;
  RotaryParams p;
  p.x = static_cast<const uint16_t*>(x);
  p.out = static_cast<uint16_t*>(out);
  p.table = reinterpret_cast<const float2*>(table);
  p.positions = positions;
  p.T = T;
  p.ldx = ldx;
  p.ldo = ldo;
  p.table_len = positions_in_table;
  p.H = H;
  p.D = D;
  p.rot = rot;
  p.interleaved = layout == B2B_ROTARY_INTERLEAVED;
  p.inverse = inverse;
  p.err = d->err;
  return launched(launch_rotary(dt == B2B_BF16, p, d->num_sms, static_cast<cudaStream_t>(stream)));
}

b2b_status b2b_cache_append(b2b_dtype dt, const b2b_cache* cache, int64_t T, const void* k,
                            int64_t ldk, const void* v, int64_t ldv, const float* table,
                            int64_t positions_in_table, int32_t rot, b2b_rotary_layout layout,
                            const void* q, int64_t ldq, int32_t q_heads, void* q_out, int64_t ldqo,
                            void* stream) {
  if (dt != B2B_F16 && dt != B2B_BF16) return B2B_ERR_UNSUPPORTED;
  if (b2b_status st = check_cache(cache, T); st != B2B_OK) return st;
  const int64_t row = static_cast<int64_t>(cache->heads) * cache->head_dim;
  if (b2b_status st = check_ld(ldk, row); st != B2B_OK) return st;
  if (b2b_status st = check_ld(ldv, row); st != B2B_OK) return st;
  if (table != nullptr) {
    if (positions_in_table < 0) return B2B_ERR_SHAPE;
    if (b2b_status st = check_rot(cache->head_dim, rot, layout); st != B2B_OK) return st;
  }
  if (q != nullptr || q_out != nullptr) {
    if (q_heads <= 0 || q_heads > 65536) return B2B_ERR_SHAPE;
    const int64_t q_row = static_cast<int64_t>(q_heads) * cache->head_dim;
    if (b2b_status st = check_ld(ldq, q_row); st != B2B_OK) return st;
    if (b2b_status st = check_ld(ldqo, q_row); st != B2B_OK) return st;
    if (table == nullptr) return B2B_ERR_NULL;       // queries come along to be rotated only
    if (T > 0 && (!q || !q_out)) return B2B_ERR_NULL;
    if (!aligned(q, 16) || !aligned(q_out, 16)) return B2B_ERR_ALIGN;
  }
  if (T == 0) return B2B_OK;
  if (!k || !v) return B2B_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(table, 16)) return B2B_ERR_ALIGN;
  const int64_t per_seq = (cache->max_new - 1 + cache->page_size - 1) / cache->page_size + 1;
  if (per_seq * cache->batch * cache->heads * 2 + T > 0x7FFFFFFF) return B2B_ERR_UNSUPPORTED;
  DecoderDevice* d = decoder_device();
  if (d == nullptr) return B2B_ERR_CUDA;
  if (q != nullptr) {
    const int64_t q_row = static_cast<int64_t>(q_heads) * cache->head_dim;
    const RowSet from{q, ldq, q_row}, to{q_out, ldqo, q_row};
    if ((!same_rows(from, to, T) && overlap(from, to, T)) || overlap(to, RowSet{k, ldk, row}, T) ||
        overlap(to, RowSet{v, ldv, row}, T))
      return B2B_ERR_UNSUPPORTED;
  }
  AppendParams p;
  p.c = view_of(cache, T, d->err);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q = static_cast<const uint16_t*>(q);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.table = reinterpret_cast<const float2*>(table);
  p.ldk = ldk;
  p.ldv = ldv;
  p.ldq = ldq;
  p.ldqo = ldqo;
  p.table_len = positions_in_table;
  p.q_heads = q_heads;
  p.rot = rot;
  p.interleaved = layout == B2B_ROTARY_INTERLEAVED;
  return launched(launch_append(dt == B2B_BF16, p, d->num_sms, static_cast<cudaStream_t>(stream)));
}

b2b_status b2b_cache_attention_workspace(const b2b_cache* cache, int64_t T, int32_t q_heads,
                                         int64_t* bytes) {
  if (bytes == nullptr) return B2B_ERR_NULL;
  *bytes = 0;
  if (b2b_status st = check_attention(cache, T, q_heads, 1.f, 0.f); st != B2B_OK) return st;
  if (T == 0) return B2B_OK;
  DecoderDevice* d = decoder_device();
  if (d == nullptr) return B2B_ERR_CUDA;
  *bytes = split_of(cache, q_heads, d->num_sms).bytes;
  return B2B_OK;
}

b2b_status b2b_cache_attention(b2b_dtype dt, const b2b_cache* cache, int64_t T, const void* q,
                               int64_t ldq, int32_t q_heads, float scale, float softcap,
                               const float* slopes, void* out, void* workspace,
                               int64_t workspace_bytes, void* stream) {
  if (dt != B2B_F16 && dt != B2B_BF16) return B2B_ERR_UNSUPPORTED;
  if (b2b_status st = check_attention(cache, T, q_heads, scale, softcap); st != B2B_OK) return st;
  if (b2b_status st = check_ld(ldq, static_cast<int64_t>(q_heads) * cache->head_dim); st != B2B_OK)
    return st;
  if (T == 0) return B2B_OK;
  if (!q || !out) return B2B_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(slopes, 4) || !aligned(workspace, 16))
    return B2B_ERR_ALIGN;
  DecoderDevice* d = decoder_device();
  if (d == nullptr) return B2B_ERR_CUDA;
  const int64_t row = static_cast<int64_t>(q_heads) * cache->head_dim;
  if (overlap(RowSet{q, ldq, row}, RowSet{out, row, row}, T)) return B2B_ERR_UNSUPPORTED;
  const SplitChoice sc = split_of(cache, q_heads, d->num_sms);
  if (sc.bytes > 0 && workspace == nullptr) return B2B_ERR_NULL;
  if (workspace_bytes < sc.bytes) return B2B_ERR_SHAPE;
  AttendParams p;
  p.c = view_of(cache, T, d->err);
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.slopes = slopes;
  p.ldq = ldq;
  p.q_heads = q_heads;
  p.group = q_heads / cache->heads;
  p.is_bf16 = dt == B2B_BF16;
  p.scale = scale;
  // a cap below 2^-100 is nothing beside any other score's rounding, and its inverse stays finite
  p.softcap = softcap > 0.f && softcap < 7.8886091e-31f ? 7.8886091e-31f : softcap;
  p.inv_softcap = softcap > 0.f ? 1.f / p.softcap : 0.f;
  p.grid = sc.grid;
  p.min_tiles = kMinTiles;
  p.whole = sc.whole;
  p.meta = sc.bytes == 0 ? nullptr : static_cast<uint32_t*>(workspace);
  p.part = sc.bytes == 0 || sc.prompt ? nullptr
                    : reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                               16 * ((static_cast<int64_t>(cache->batch) + 4) / 4));
  p.wait_limit_ns = kDecoderWaitNs;
  auto s = static_cast<cudaStream_t>(stream);
  if (sc.prompt) return launched(launch_prompt(p, s));
  cudaError_t e = cudaErrorInvalidValue;
  switch (cache->head_dim) {
    case 64: e = launch_attend_64(sc.nt, p, s); break;
    case 96: e = launch_attend_96(sc.nt, p, s); break;
    case 128: e = launch_attend_128(sc.nt, p, s); break;
    case 192: e = launch_attend_192(sc.nt, p, s); break;
    case 256: e = launch_attend_256(sc.nt, p, s); break;
    default: break;
  }
  if (e != cudaSuccess || sc.whole) return launched(e);
  return launched(launch_attend_combine(p, sc.nt, d->num_sms, s));
}

b2b_status b2b_get_cache_error(uint32_t info[4]) {
  DecoderDevice* d = decoder_device();
  if (d == nullptr) return B2B_ERR_CUDA;
  uint32_t w[4] = {0, 0, 0, 0};
  if (cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(w, d->err, sizeof(w), cudaMemcpyDeviceToHost) != cudaSuccess) {
    cudaGetLastError();
    return B2B_ERR_CUDA;
  }
  if (info) std::memcpy(info, w, sizeof(w));
  if (w[0] == 0u) return B2B_OK;
  const uint32_t zero[4] = {0, 0, 0, 0};
  if (cudaMemcpy(d->err, zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess) {
    cudaGetLastError();
    return B2B_ERR_CUDA;
  }
  return w[0] == kCodeIndex ? B2B_ERR_SHAPE : w[0] == 6u ? B2B_ERR_TIMEOUT : B2B_ERR_CUDA;
}

}  // extern "C"
