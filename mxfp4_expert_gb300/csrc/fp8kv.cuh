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
__device__ __forceinline__ bool e4m3_is_nan(uint32_t c) { return (c & 0x7Fu) == 0x7Fu; }

// Four codes in a word, worth 2^sh of what they were (sh < 0: rounded to
// nearest even; NaN stays NaN).
__device__ __forceinline__ uint32_t kv_rescale4(uint32_t w, int sh) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t c0 = (w >> (8 * i)) & 0xFFu, c1 = (w >> (8 * i + 8)) & 0xFFu;
    const float v0 = e4m3_is_nan(c0) ? __int_as_float(0x7FC00000) : scale2(e4m3_to_f32(c0), sh);
    const float v1 = e4m3_is_nan(c1) ? __int_as_float(0x7FC00000) : scale2(e4m3_to_f32(c1), sh);
    r |= uint32_t(f32x2_to_e4m3x2(v0, v1)) << (8 * i);
  }
  return r;
}

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
