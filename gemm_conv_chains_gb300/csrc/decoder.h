// decoder.h -- internal interface of the decoder-block operators (rotary positions, the
// append to a paged e4m3 cache, the attention over it): launch parameters and launchers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace b2b {

// Error word of these operators: {code, kernel, what, index}; the first error wins.
enum DecoderError : uint32_t {
  DEC_ERR_POSITION = 1,   // a position outside the rotary table
  DEC_ERR_PAGE = 2,       // a page number outside the pool
  DEC_ERR_LENGTH = 3,     // a length that is below its new tokens or above its page table
  DEC_ERR_STARTS = 4      // starts that decrease, leave the rows or exceed max_new
};
enum DecoderKernel : uint32_t { DK_ROTARY = 32, DK_APPEND = 33, DK_ATTEND = 34, DK_PROMPT = 35 };
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
  int64_t ldq;
  int32_t q_heads, group, is_bf16;
  float scale, softcap;       // softcap 0: none
  float inv_softcap;
  int32_t grid, min_tiles, whole;
  float* part;                // split workspace: see cache_attention.cuh
  uint32_t* meta;             // [0]: tiles per run, [1 + b]: sequence b's first tile
  uint64_t wait_limit_ns;
};

// Launches with programmatic stream serialisation, as the chain kernels: the kernel may be scheduled
// while the one before it in the stream finishes, and waits for that (griddepcontrol.wait) before
// it touches global memory.
template <class... P, class... A>
cudaError_t launch_early(void (*fn)(P...), int64_t grid, int block, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
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
// The split kernel with row tiles of 8 nt query rows, per head size.
cudaError_t launch_attend_64(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_96(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_128(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_192(int nt, const AttendParams& p, cudaStream_t s);
cudaError_t launch_attend_256(int nt, const AttendParams& p, cudaStream_t s);
// The tcgen05 kernel for prompts (head sizes 64, 96, 128).
cudaError_t launch_prompt(const AttendParams& p, cudaStream_t s);
// Bytes of workspace that it takes for `rows` query rows per sequence and kv head (p.meta).
int64_t prompt_workspace(int64_t rows, int32_t B);
// Joins what the split kernel left in parts.
cudaError_t launch_attend_combine(const AttendParams& p, int nt, int num_sms, cudaStream_t s);

}  // namespace b2b
