// decoder_device.cuh -- device helpers of the decoder-block operators.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "decoder.h"
#include "ptx.cuh"

namespace b2b {

__device__ __forceinline__ void index_error(uint32_t* err, uint32_t kernel, uint32_t what,
                                            uint32_t index) {
  record_error(err, kCodeIndex, kernel, what, index);
}

// One sequence of a call: its rows among the new tokens and its length in the cache.
// Values that leave the rows or the page table are cut down to what fits and recorded.
struct Sequence {
  int row;      // first new token's row
  int n;        // new tokens
  int len;      // cached tokens, the new ones included
};

__device__ __forceinline__ Sequence load_sequence(const CacheView& c, int b, uint32_t kernel) {
  Sequence s;
  int64_t end;
  if (c.starts != nullptr) {
    s.row = __ldg(c.starts + b);
    end = __ldg(c.starts + b + 1);
  } else {
    const int each = static_cast<int>(c.T / c.B);
    s.row = b * each;
    end = s.row + each;
  }
  const int64_t n = end - s.row;
  s.n = static_cast<int>(n);
  if (s.row < 0 || n < 0 || end > c.T || n > c.max_new) {
    index_error(c.err, kernel, DEC_ERR_STARTS, b);
    s.n = (s.row < 0 || n < 0 || end > c.T) ? 0 : c.max_new;
  }
  s.len = __ldg(c.lens + b);
  const int64_t most = static_cast<int64_t>(c.max_pages) << c.page_shift;
  if (s.len < s.n || s.len > most) {
    index_error(c.err, kernel, DEC_ERR_LENGTH, b);
    if (s.len < s.n) s.n = 0;
    if (s.len > most) s.n = s.len = 0;
  }
  return s;
}

template <bool BF16>
__device__ __forceinline__ float2 widen2(uint32_t v) {
  if constexpr (BF16) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = widen2<BF16>(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(narrow2<BF16>(f[0], f[1]), narrow2<BF16>(f[2], f[3]),
                    narrow2<BF16>(f[4], f[5]), narrow2<BF16>(f[6], f[7]));
}

// (a, b) turned by (cos, sin): a c - b s, b c + a s, each product and sum rounded to fp32
// on its own (no fused multiply-add), so that a rotated key has one value whichever
// kernel turns it.
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float x = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
  const float y = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
  a = x;
  b = y;
}

// Eight channels of one head's row split into units of work:
//   half layout         unit u < rot / 16: channels [8u, 8u + 8) with their partners at
//                       rot / 2 + 8u; later units copy 8 channels past rot
//   interleaved layout  unit u: channels [8u, 8u + 8), four pairs, copied past rot
__device__ __forceinline__ int row_units(int D, int rot, int interleaved) {
  return interleaved ? D / 8 : rot / 16 + (D - rot) / 8;
}

// The fp32 values of unit u after the rotation: lo (and hi in a half-layout pair unit).
// cs: the position's table row.  Returns the channel of lo, or of both through `pair`.
template <bool BF16>
__device__ __forceinline__ int load_unit(const uint16_t* row, const float2* cs, int u, int rot,
                                         int interleaved, bool inverse, float (&lo)[8],
                                         float (&hi)[8], bool& pair) {
  const float sign = inverse ? -1.f : 1.f;
  pair = false;
  if (interleaved) {
    const int d = 8 * u;
    widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(row + d)), lo);
    if (d < rot) {
      const float4* t = reinterpret_cast<const float4*>(cs + d / 2);
      const float4 c0 = __ldg(t), c1 = __ldg(t + 1);
      turn(lo[0], lo[1], make_float2(c0.x, sign * c0.y));
      turn(lo[2], lo[3], make_float2(c0.z, sign * c0.w));
      turn(lo[4], lo[5], make_float2(c1.x, sign * c1.y));
      turn(lo[6], lo[7], make_float2(c1.z, sign * c1.w));
    }
    return d;
  }
  const int pairs = rot / 16;
  if (u >= pairs) {
    const int d = rot + 8 * (u - pairs);
    widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(row + d)), lo);
    return d;
  }
  pair = true;
  const int d = 8 * u;
  widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(row + d)), lo);
  widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(row + d + rot / 2)), hi);
  const float4* t = reinterpret_cast<const float4*>(cs + d);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 c = __ldg(t + i);
    turn(lo[2 * i], hi[2 * i], make_float2(c.x, sign * c.y));
    turn(lo[2 * i + 1], hi[2 * i + 1], make_float2(c.z, sign * c.w));
  }
  return d;
}

// Two fp32 values to e4m3, nearest even, saturating; a NaN stays one.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The four e4m3 codes of a word as two pairs of fp16 (exact; a NaN code gives a NaN).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

}  // namespace b2b
