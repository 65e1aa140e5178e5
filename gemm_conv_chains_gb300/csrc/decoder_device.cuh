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

// The kernels read with plain loads, not __ldg: that promises data which stays the same for the
// whole kernel, and a kernel launched early starts while the one that writes its inputs still
// runs (and an in-place call writes what it reads).

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
    s.row = c.starts[b];
    end = c.starts[b + 1];
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
  s.len = c.lens[b];
  const int64_t most = static_cast<int64_t>(c.max_pages) << c.page_shift;
  if (s.len < s.n || s.len > most) {
    index_error(c.err, kernel, DEC_ERR_LENGTH, b);
    if (s.len < s.n) s.n = 0;
    if (s.len > most) s.n = s.len = 0;
  }
  return s;
}

// Which of the 16 tokens from the new token `off` on a row of a tree sees, as bits: its mask's, and
// every older token (off < 0, above -16).  Nothing at or past the n new ones (off < n).  The mask's words
// are `stride` apart.
__device__ __forceinline__ uint32_t tree_window(const uint32_t* mask, int stride, int words, int off, int n) {
  uint32_t w;
  if (off < 0) {
    w = (mask[0] << -off) | ((1u << -off) - 1u);
  } else {
    const int i = off >> 5, sh = off & 31;
    w = mask[i * stride] >> sh;
    if (sh > 16 && i + 1 < words) w |= mask[(i + 1) * stride] << (32 - sh);
  }
  const int left = n - off;
  return w & (left < 16 ? (1u << left) - 1u : 0xFFFFu);
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

// (a, b) turned by (cos, sin): a c - b s, b c + a s; one function, so that a key has one value
// whichever kernel turns it.
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float x = fmaf(a, cs.x, -(b * cs.y));
  const float y = fmaf(b, cs.x, a * cs.y);
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

// Where a thread's unit u lies in every row that it takes: channel d, and (a pair unit of the half
// layout) its partners at d + rot / 2.
struct UnitAt {
  int d;
  bool pair, turned;
};
__device__ __forceinline__ UnitAt unit_at(int u, int rot, int interleaved) {
  UnitAt a;
  if (interleaved) {
    a.d = 8 * u;
    a.pair = false;
    a.turned = a.d < rot;
  } else {
    const int pairs = rot / 16;
    a.pair = a.turned = u < pairs;
    a.d = a.pair ? 8 * u : rot + 8 * (u - pairs);
  }
  return a;
}

// A unit's raw vectors, to be asked for ahead of what their use waits for.
struct RawUnit {
  uint4 lo, hi;
};
__device__ __forceinline__ RawUnit load_raw(const uint16_t* row, const UnitAt& a, int rot) {
  RawUnit r;
  r.lo = *reinterpret_cast<const uint4*>(row + a.d);
  r.hi = r.lo;
  if (a.pair) r.hi = *reinterpret_cast<const uint4*>(row + a.d + rot / 2);
  return r;
}

// The (cos, sin) of a unit's pairs: kept in registers by a thread that turns several units with
// them, or read from a table row as they are used.
struct Angles {
  float4 v[4];
  __device__ __forceinline__ float4 operator[](int i) const { return v[i]; }
};
struct AngleRow {
  const float4* t;
  __device__ __forceinline__ float4 operator[](int i) const { return t[i]; }
};
__device__ __forceinline__ AngleRow angle_row(const float2* row, const UnitAt& a, int interleaved) {
  return AngleRow{reinterpret_cast<const float4*>(row + (interleaved ? a.d / 2 : a.d))};
}
__device__ __forceinline__ Angles load_angles(const float2* row, const UnitAt& a, int interleaved) {
  const AngleRow t = angle_row(row, a, interleaved);
  Angles g;
  if (a.turned) {
    g.v[0] = t[0];
    g.v[1] = t[1];
    if (!interleaved) {
      g.v[2] = t[2];
      g.v[3] = t[3];
    }
  }
  return g;
}

// The fp32 values of a unit after the rotation: lo, and hi of a pair unit.
template <bool BF16, class A>
__device__ __forceinline__ void turn_unit(const RawUnit& r, const UnitAt& a, const A& g,
                                          int interleaved, float sign, float (&lo)[8], float (&hi)[8]) {
  widen8<BF16>(r.lo, lo);
  if (!a.turned) return;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c = g[i];
      turn(lo[4 * i], lo[4 * i + 1], make_float2(c.x, sign * c.y));
      turn(lo[4 * i + 2], lo[4 * i + 3], make_float2(c.z, sign * c.w));
    }
  } else {
    widen8<BF16>(r.hi, hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 c = g[i];
      turn(lo[2 * i], hi[2 * i], make_float2(c.x, sign * c.y));
      turn(lo[2 * i + 1], hi[2 * i + 1], make_float2(c.z, sign * c.w));
    }
  }
}

// The unit stored in its rows' type; what is not turned is copied bit by bit.
template <bool BF16, class A>
__device__ __forceinline__ void store_turned(uint16_t* row, const RawUnit& r, const UnitAt& a,
                                             const A& g, int rot, int interleaved, float sign) {
  uint4* dst = reinterpret_cast<uint4*>(row + a.d);
  if (!a.turned) {
    *dst = r.lo;
    return;
  }
  float lo[8], hi[8];
  turn_unit<BF16>(r, a, g, interleaved, sign, lo, hi);
  *dst = narrow8<BF16>(lo);
  if (a.pair) *reinterpret_cast<uint4*>(row + a.d + rot / 2) = narrow8<BF16>(hi);
}

// A query row's fp16 form: fp16 rows are taken as they are; bf16 rows are multiplied by the power of
// two `inv` (at most 2^126) that brings their largest magnitude to 2^14 .. 2^15, and its inverse, which
// is returned, is put back into the scores in fp32.
template <bool BF16>
__device__ __forceinline__ float row_unit(float amax, float& inv) {
  inv = 1.f;
  if (!BF16) return 1.f;
  const uint32_t e = (__float_as_uint(amax) >> 23) & 0xFFu, u = e > 15u ? e - 14u : 1u;
  inv = __uint_as_float((254u - u) << 23);
  return __uint_as_float(u << 23);
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap tanh(z / cap).  tanh y = 1 - 2 / (e^2y + 1) cancels for small y, by 2^-23 of the cap whatever z
// is; below 1/4 it is y (1 - y^2 / 3 + 2 y^4 / 15 - 17 y^6 / 315), the start of its series, whose rest
// is below 2^-21 of y there.
__device__ __forceinline__ float capped(float z, float cap, float inv_cap) {
  const float y = z * inv_cap, yy = y * y;
  const float near = z * fmaf(yy, fmaf(yy, fmaf(yy, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  const float far = cap - 2.f * cap * rcp_fast(exp2_fast(y * (2.f * kLog2e)) + 1.f);
  return fabsf(y) < 0.25f ? near : far;
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
