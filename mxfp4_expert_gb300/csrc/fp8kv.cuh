// Helpers of the 8-bit key/value cache: codes are E4M3, a page and head share
// one E8M0 scale byte s worth 2^(s - 127).
#pragma once

#include "common.cuh"

namespace moe {

// Byte of the smallest power of two 2^e (e >= -127) with amax <= 448 * 2^e
// (448 = 0.875 * 2^9 is E4M3's largest value); 0 for amax 0.
__device__ __forceinline__ int kv_scale_byte(float amax) {
  if (!(amax > 0.0f)) return 0;
  int e;
  const float m = frexpf(amax, &e);
  e += (m > 0.875f ? 1 : 0) - 9 + 127;
  return e < 0 ? 0 : (e > 254 ? 254 : e);
}

// The same for a code of finite magnitude c (7 bits) and scale byte s, whose
// value may be more than fp32 holds. A normal code is (8 + m) 2^(e - 10), of
// which 448 = 14 * 2^5 goes to byte s at e = 15, m <= 6; m = 7 needs one more. A
// subnormal one is m 2^-9 = m 2^-(floor log2 m) 2^(floor log2 m - 9).
__device__ __forceinline__ int kv_code_byte(uint32_t c, int s) {
  const int e = int(c >> 3), m = int(c & 7u);
  const int b = e ? s + e - 15 + (m == 7) : (m ? s - 17 + (m >= 2) + (m >= 4) : 0);
  return max(b, 0);
}

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }
// Does one of the word's four codes stand for NaN?
__device__ __forceinline__ bool any_nan4(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Four codes in a word times f, a power of two: rounded to nearest even, NaN
// stays NaN. |values| * f <= 448 is up to the caller.
__device__ __forceinline__ uint32_t kv_rescale4(uint32_t w, float f) {
  uint32_t h0, h1;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(h0), "=r"(h1)
      : "r"(w));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  return uint32_t(f32x2_to_e4m3x2(a.x * f, a.y * f)) | uint32_t(f32x2_to_e4m3x2(b.x * f, b.y * f)) << 16;
}
// The factor that turns codes of scale byte `from` into units of `to`; below
// 2^-126 every code becomes zero.
__device__ __forceinline__ float kv_factor(int from, int to) { return pow2(max(from - to, -126)); }

// Sequence b's rows [c0, c1) of `total` packed rows, cut to what fits;
// *bad if cu leaves [0, total] or falls.
__device__ __forceinline__ void packed_range(const int32_t* cu, int b, int total, int* c0, int* c1, bool* bad) {
  const int x = __ldg(cu + b), y = __ldg(cu + b + 1);
  const int lo = min(max(x, 0), total), hi = min(max(y, lo), total);
  if (lo != x || hi != y) *bad = true;
  *c0 = lo;
  *c1 = hi;
}

}  // namespace moe
