// Append to the 8-bit cache with the position rotation on the way, and the
// queries' rotation beside it.
//
// Pair j of a head is turned by the angle p f_j, p the token's position. The
// angle is taken in turns and in integers: F_j = f_j / 2 pi (without its whole
// part) times 2^64, and p F_j modulo 2^64 is the angle's fraction of a turn. F_j is
// cut, so that errs by p 2^-64; the top 32 bits, which do for fp32, give quadrant and
// remainder, cosine and sine of the remainder are their Taylor series. Keys in doubt
// take the angle from p f_j as a whole, to 2^-63 of a turn.
//
// A CTA takes one page's new tokens and a few heads, of keys, values or queries: the
// cosines and sines of all the tokens into shared memory once, then head after head,
// the next one's channels on their way meanwhile. A thread holds both halves of its
// pairs. Of a key or value head the maximum, the page's scale and the codes as
// append_kernel makes them, which has no rotation. Bound by HBM: 3 bytes a key or
// value, 4 a query's channel; 12,345 tokens of 16 heads over 8 of 128 take 46 us (3.8
// TB/s), a token of each of 64 sequences 8.8 where a key is in doubt, which costs about 2.
#include <algorithm>

#include "attn.h"
#include "fp8kv.cuh"
#include "kvblock.cuh"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 6;        // CTAs an SM before heads share one

// cos and sin of s 2^-32 turns.
__device__ __forceinline__ float2 turn(uint32_t s) {
  const uint32_t quad = (s + 0x20000000u) >> 30;
  const float x = float(int32_t(s - (quad << 30))) * 1.4629180792671596e-9f;   // 2 pi 2^-32; |x| <= pi / 4
  const float z = x * x;
  const float sn = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
  const float cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const float a = (quad & 1) ? sn : cs, b = (quad & 1) ? cs : sn;
  return make_float2(((quad + 1) & 2) ? -a : a, (quad & 2) ? -b : b);
}

// Sixteen channels of a row, of eight pairs that t turns; kind 0: not turned, 1:
// pair i is channel i of both vectors, 2: neighbours.
__device__ __forceinline__ void turn16(const uint4& w0, const uint4& w1, const float2* t, int kind, float (&y)[16]) {
  const uint32_t u[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  if (kind == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = bf16_lo(u[i]);
      y[2 * i + 1] = bf16_hi(u[i]);
    }
    return;
  }
  const float4* t4 = reinterpret_cast<const float4*>(t);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 c = t4[i];          // pairs 2 i and 2 i + 1
    if (kind == 1) {
      const float a0 = bf16_lo(u[i]), a1 = bf16_hi(u[i]), b0 = bf16_lo(u[4 + i]), b1 = bf16_hi(u[4 + i]);
      y[2 * i] = a0 * c.x - b0 * c.y;
      y[2 * i + 1] = a1 * c.z - b1 * c.w;
      y[8 + 2 * i] = b0 * c.x + a0 * c.y;
      y[8 + 2 * i + 1] = b1 * c.z + a1 * c.w;
    } else {
      const float a0 = bf16_lo(u[2 * i]), b0 = bf16_hi(u[2 * i]), a1 = bf16_lo(u[2 * i + 1]), b1 = bf16_hi(u[2 * i + 1]);
      y[4 * i] = a0 * c.x - b0 * c.y;
      y[4 * i + 1] = b0 * c.x + a0 * c.y;
      y[4 * i + 2] = a1 * c.z - b1 * c.w;
      y[4 * i + 3] = b1 * c.z + a1 * c.w;
    }
  }
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// find_block by the whole CTA: a sequence a thread, so one round of loads for up to
// kRopeThreads of them. Ends with a barrier.
__device__ __forceinline__ Block find_block_cta(const AppendArgs& a, int x, bool* bad) {
  __shared__ int s_warp[kRopeThreads / 32];
  __shared__ Block s_blk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = a.c.page_size;
  if (tid == 0) s_blk.b = -1;
  int before = 0;
  for (int b0 = 0; b0 < a.n_seq; b0 += kRopeThreads) {
    const int b = b0 + tid;
    int c0 = 0, c1 = 0, start = 0, n = 0;
    if (b < a.n_seq) {
      start = __ldg(a.start + b);
      packed_range(a.cu, b, a.total, &c0, &c1, bad);
      if (start < 0 || start > 0x7FFFFFFF - (c1 - c0)) {
        *bad = true;
        c1 = c0;
      }
      if (c1 > c0) n = (start + (c1 - c0) - 1) / P - start / P + 1;
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int lo = before + incl - n, all = before;
#pragma unroll
    for (int i = 0; i < kRopeThreads / 32; ++i) {
      lo += i < warp ? s_warp[i] : 0;
      all += s_warp[i];
    }
    if (x >= lo && x < lo + n) {
      const int blk = start / P + (x - lo);
      const int64_t p0 = (int64_t)blk * P, end = (int64_t)start + (c1 - c0);
      const int s0 = start > p0 ? int(start - p0) : 0;
      s_blk = Block{b, blk, s0, end < p0 + P ? int(end - p0) : P, c0 + int(p0 + s0 - start)};
    }
    before = all;
    __syncthreads();
    if (x < before) break;       // found; the last CTA looks at every sequence
  }
  return s_blk;
}
// n f / 2 pi for a frequency of magnitude f = mantissa 2^e, n times the mantissa below 2^57: its
// fraction of a turn in units of 2^-64, cut. 1 / 2 pi to 2^-128, and shifts: what the last words
// leave out is less than 2^-64 of a turn for f up to 2^30.
struct Frequency {
  uint32_t mantissa;
  int e, negative;
};
__device__ __forceinline__ Frequency parts_of(float inv_freq) {
  const uint32_t b = __float_as_uint(inv_freq) & 0x7FFFFFFFu, ex = b >> 23;
  return {(b & 0x7FFFFFu) | (ex ? 0x800000u : 0u), min(int(ex ? ex : 1u) - 150, 63), inv_freq < 0.0f};
}
__device__ __forceinline__ uint64_t turns_of(uint64_t n, const Frequency& f) {
  constexpr uint64_t kHigh = 0x28BE60DB9391054Aull, kLow = 0x7F09D5F47D4D3770ull;
  n *= f.mantissa;
  const uint64_t w0 = n * kLow, c = __umul64hi(n, kLow), w1 = n * kHigh + c, w2 = __umul64hi(n, kHigh) + (w1 < c);
  if (f.e >= 0) return f.e ? w1 << f.e | w0 >> (64 - f.e) : w1;
  const int s = -f.e;
  return s < 64 ? w1 >> s | w2 << (64 - s) : s < 128 ? w2 >> (s - 64) : 0;
}
// Beyond this a frequency is no angle per position; it turns to NaN, as does one that is not finite.
constexpr float kMostFreq = 1099511627776.0f;       // 2^40
// Phase per position of a pair, in 2^-64 turns; false for NaN.
__device__ __forceinline__ bool phase_of_pair(const RopeArgs& a, int j, uint64_t* F) {
  const float inv_freq = __ldg(a.inv_freq + j);
  const Frequency f = parts_of(inv_freq);
  const uint64_t x = turns_of(1, f);
  *F = f.negative ? 0 - x : x;
  return fabsf(inv_freq) <= kMostFreq;
}
// Position of a page's first new token.
__device__ __forceinline__ int64_t first_position(const RopeArgs& a, const Block& f) {
  return (int64_t)__ldg(a.rope_start + f.b) + ((int64_t)f.blk * a.ap.c.page_size + f.s0 - __ldg(a.ap.start + f.b));
}
// Cosines and sines of a page's new tokens, for the caller's barrier; NaN without an `angle`.
__device__ __forceinline__ void fill_angles(const RopeArgs& a, const Block& f, uint64_t F, bool angle, float2* cs) {
  const int half = a.rot / 2, j = threadIdx.x % half, first = threadIdx.x / half, step = kRopeThreads / half;
  if (first >= step) return;
  const int64_t p0 = first_position(a, f);
  uint64_t at = uint64_t(p0 + first) * F;
  const uint64_t by = uint64_t(step) * F;
  for (int t = first; t < f.s1 - f.s0; t += step, at += by)
    cs[t * half + j] = angle ? turn(uint32_t(at >> 32)) : make_float2(__int_as_float(0x7FC00000), __int_as_float(0x7FC00000));
}
__device__ __forceinline__ void store_bf16(__nv_bfloat16* o, int c0, int c1, const float (&y)[16]) {
  *reinterpret_cast<uint4*>(o + c0) = make_uint4(bf16x2(y[0], y[1]), bf16x2(y[2], y[3]), bf16x2(y[4], y[5]), bf16x2(y[6], y[7]));
  *reinterpret_cast<uint4*>(o + c1) =
      make_uint4(bf16x2(y[8], y[9]), bf16x2(y[10], y[11]), bf16x2(y[12], y[13]), bf16x2(y[14], y[15]));
}
// Largest finite magnitude's bits; *nonfinite if some are not.
__device__ __forceinline__ uint32_t largest(const float (&y)[16], bool* nonfinite) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(y[e]) & 0x7FFFFFFFu);
  if (top >= 0x7F800000u) {
    *nonfinite = true;
    top = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t m = __float_as_uint(y[e]) & 0x7FFFFFFFu;
      if (m < 0x7F800000u) top = max(top, m);
    }
  }
  return top;
}
// 2^(127 - byte); 2^-127 and 2^-128 are subnormal
__device__ __forceinline__ float code_factor(int byte) {
  return byte <= 253 ? pow2(127 - byte) : __uint_as_float(0x00800000u >> (byte - 253));
}
__device__ __forceinline__ void store_codes(uint8_t* o, int c0, int c1, const float (&y)[16], float f, bool nonfinite) {
  uint32_t q[4];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float lo = y[2 * j] * f, hi = y[2 * j + 1] * f;
    if (nonfinite) {   // inf takes the code of NaN: there is none for it
      if (!(fabsf(y[2 * j]) <= 3.4028235e38f)) lo = __int_as_float(0x7FC00000);
      if (!(fabsf(y[2 * j + 1]) <= 3.4028235e38f)) hi = __int_as_float(0x7FC00000);
    }
    const uint32_t c = f32x2_to_e4m3x2(lo, hi);
    q[j >> 1] = j & 1 ? q[j >> 1] | c << 16 : c;
  }
  *reinterpret_cast<uint2*>(o + c0) = make_uint2(q[0], q[1]);
  *reinterpret_cast<uint2*>(o + c1) = make_uint2(q[2], q[3]);
}
// A turned channel errs by less than kKeyError times the sizes of its pair: cosine and
// sine by 2^-23 each (an angle of 24 bits, its factor, a series), two products and
// their sum by 2^-24 each, so 2^-22 (|a| + |b|), and |a| + |b| is at most 1.4143 times
// that of the turned pair. Where that could change a code, which is a step of 2^-3, or
// a scale, the pair is turned once more in fp64, so that codes and scales are those of
// the exact values: one value in 2^16, and 10 % of the time for 12,345 tokens.
constexpr float kKeyError = 3.4e-7f;    // 1.4143 * 2^-22 = 3.372e-7
constexpr float kLargest = 3.4028235e38f;

// A key's pair turned in fp64, times f; rounded to fp32 by truncation with the last bit set where
// that leaves something out, so that a further rounding is right. What is not finite, or would not be
// in fp32 before the product with f, is NaN.
__device__ __noinline__ float2 turn_exact(float a0, float b0, const float* inv_freq, int64_t pos, float f) {
  const double a = a0, b = b0;
  const float fr = __ldg(inv_freq), nan = __int_as_float(0x7FC00000);
  if (!(fabsf(fr) <= kMostFreq && fabsf(a0) <= kLargest && fabsf(b0) <= kLargest)) return make_float2(nan, nan);
  const Frequency freq = parts_of(fr);
  const uint64_t x = turns_of(uint64_t(pos < 0 ? -pos : pos), freq);
  const int64_t at = int64_t((pos < 0) != (freq.negative != 0) ? 0 - x : x);
  double sn = 0.0, cs = 1.0;
  if (at != 0) sincospi(double(at) * 1.0842021724855044e-19, &sn, &cs);      // half turns: 2^-63
  auto odd = [f, nan](double v) {
    if (fabs(v) >= 3.4028235677973366e38) return nan;     // 2^128 - 2^103: half a step above fp32's largest
    v *= f;
    const uint32_t r = __float_as_uint(__double2float_rz(v));
    return __uint_as_float(double(__uint_as_float(r)) != v ? r | 1u : r);
  };
  return make_float2(odd(a * cs - b * sn), odd(b * cs + a * sn));
}
// The CTA: a part-filled page's older codes, in units of the new scale.
__device__ __forceinline__ void rescale_codes(uint8_t* codes, int n, float f) {
  for (int v = threadIdx.x; v < n / 16; v += kRopeThreads) {
    uint4* p = reinterpret_cast<uint4*>(codes) + v;
    uint4 c = *p;
    c.x = kv_rescale4(c.x, f);
    c.y = kv_rescale4(c.y, f);
    c.z = kv_rescale4(c.z, f);
    c.w = kv_rescale4(c.w, f);
    *p = c;
  }
}

// Could codes of y, times f, be others within the error of y?
__device__ __forceinline__ bool in_doubt(const float (&y)[16], float f, int kind) {
  uint32_t differ = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = (kind == 1 ? y[i] : y[2 * i]) * f, b = (kind == 1 ? y[8 + i] : y[2 * i + 1]) * f;
    const float e = (fabsf(a) + fabsf(b)) * kKeyError;
    differ |= uint32_t(f32x2_to_e4m3x2(a - e, b - e)) ^ uint32_t(f32x2_to_e4m3x2(a + e, b + e));
  }
  return (differ & 0x7F7Fu) != 0;        // the sign of a zero does not count
}
// Bounds of a largest magnitude: of turned channels on both sides of it, others are exact.
__device__ __forceinline__ float largest_most(float top, int kind) {
  return kind ? fminf(fmaf(top, 2.0f * kKeyError, top), kLargest) : top;
}
__device__ __forceinline__ float largest_least(float top, int kind) { return kind ? fmaf(top, -2.0f * kKeyError, top) : top; }

// What a CTA turns exactly when it has stored everything else: groups of eight pairs (head, row of the page's new tokens,
// group; beyond the list's room all groups), and heads of which nothing is stored yet: those whose scale is in doubt, and
// those with values that are not finite or may be beyond fp32.
constexpr int kDoubts = 256;
struct Doubts {
  int n, any_head;
  uint32_t at[kDoubts], heads[32];
};
__device__ __forceinline__ void clear_doubts(Doubts* d) {
  if (threadIdx.x < 32) d->heads[threadIdx.x] = 0;
  if (threadIdx.x == 0) d->n = d->any_head = 0;
}
__device__ __forceinline__ void note_doubt(Doubts* d, int h, int row, int u) {
  const int i = atomicAdd(&d->n, 1);
  if (i < kDoubts) d->at[i] = uint32_t(h) << 16 | uint32_t(row) << 3 | uint32_t(u);
}
__device__ __forceinline__ void note_head(Doubts* d, int h) {
  atomicOr(&d->heads[h >> 5], 1u << (h & 31));
  d->any_head = 1;
}
// Whole CTA, behind a barrier: heads h0 .. h1 of its keys.
__device__ __noinline__ void settle_doubts(const RopeArgs& a, const Block& f, int page, int h0, int h1, const Doubts* d) {
  __shared__ uint32_t s_top;
  const AppendArgs& ap = a.ap;
  const int P = ap.c.page_size, D = ap.c.head_dim, H = ap.c.n_kv_heads, half = a.rot / 2, tokens = f.s1 - f.s0;
  const int64_t p0 = first_position(a, f);
  uint8_t* scales = static_cast<uint8_t*>(ap.c.k_scales) + (size_t)page * H;
  // pair `pair` of the head in row `row`, turned exactly and times 2^(127 - byte)
  auto exact = [&](int h, int row, int pair, int byte, int* c0, int* c1) {
    *c0 = a.interleaved ? 2 * pair : pair;
    *c1 = a.interleaved ? 2 * pair + 1 : pair + half;
    const __nv_bfloat16* src = ap.k + (int64_t)(f.t0 + row) * ap.k_ts + h * ap.k_hs;
    return turn_exact(__bfloat162float(src[*c0]), __bfloat162float(src[*c1]), a.inv_freq + pair, p0 + row, code_factor(byte));
  };
  auto codes = [&](int h) { return static_cast<uint8_t*>(ap.c.k_codes) + ((size_t)page * H + h) * P * D; };
  auto in_heads = [&](int h) { return (d->heads[h >> 5] >> (h & 31)) & 1u; };

  const bool all = d->n > kDoubts;
  const int n = (all ? (h1 - h0) * tokens * (half / 8) : d->n) * 8;
  for (int i = threadIdx.x; i < n; i += kRopeThreads) {
    const int x = i >> 3;
    const int h = all ? h0 + x / (tokens * (half / 8)) : int(d->at[x] >> 16);
    const int row = all ? x / (half / 8) % tokens : int(d->at[x] >> 3) & 0x1FFF, u = all ? x % (half / 8) : int(d->at[x]) & 7;
    if (in_heads(h)) continue;
    int c0, c1;
    const float2 v = exact(h, row, 8 * u + (i & 7), scales[h], &c0, &c1);
    uint8_t* o = codes(h) + (f.s0 + row) * D;
    const uint32_t c = f32x2_to_e4m3x2(v.x, v.y);
    o[c0] = uint8_t(c);
    o[c1] = uint8_t(c >> 8);
  }
  for (int h = h0; d->any_head && h < h1; ++h) {
    if (!in_heads(h)) continue;
    // the exact largest value decides between a byte and the next
    const int had = f.s0 > 0 ? int(scales[h]) : 0;
    auto value = [&](int i, int byte, int* c0, int* c1) {       // pair i of the rows' D / 2, those of the rest as they are
      const int row = i / (D / 2), pair = i % (D / 2);
      if (pair < half) return exact(h, row, pair, byte, c0, c1);
      *c0 = 2 * pair;
      *c1 = 2 * pair + 1;
      const __nv_bfloat16* src = ap.k + (int64_t)(f.t0 + row) * ap.k_ts + h * ap.k_hs;
      auto times = [byte](float v) { return fabsf(v) <= kLargest ? v * code_factor(byte) : __int_as_float(0x7FC00000); };
      return make_float2(times(__bfloat162float(src[*c0])), times(__bfloat162float(src[*c1])));
    };
    int c0, c1;
    float top = 0.0f;                 // truncated values, but what they leave out is in their last bit
    bool odd = false;
    for (int i = threadIdx.x; i < tokens * (D / 2); i += kRopeThreads) {
      const float2 v = value(i, 127, &c0, &c1);
      top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));        // of numbers
      odd |= isnan(v.x) || isnan(v.y);
    }
    odd = __syncthreads_or(odd);
    if (threadIdx.x == 0 && odd && ap.status) atomicOr(ap.status, MOE_DEV_NONFINITE_INPUT);
    if (threadIdx.x == 0) s_top = 0;
    __syncthreads();
    atomicMax(&s_top, __float_as_uint(top));
    __syncthreads();
    const int byte = max(kv_scale_byte(__uint_as_float(s_top)), had);
    for (int i = threadIdx.x; i < tokens * (D / 2); i += kRopeThreads) {
      const float2 v = value(i, byte, &c0, &c1);
      uint8_t* o = codes(h) + (f.s0 + i / (D / 2)) * D;
      const uint32_t c = f32x2_to_e4m3x2(v.x, v.y);
      o[c0] = uint8_t(c);
      o[c1] = uint8_t(c >> 8);
    }
    __syncthreads();                  // everyone has read the old scale
    if (threadIdx.x == 0) scales[h] = uint8_t(byte);
    if (byte > had && f.s0 > 0) rescale_codes(codes(h), f.s0 * D, kv_factor(had, byte));
  }
}

// Few new tokens a page, one mostly (a decode step): a CTA takes all heads of a
// page's tokens, D / 16 neighbouring lanes a head. Right for any number of tokens,
// which are read once more where there are several. A token of each of 64 sequences:
// 6.1 us, by the other kernel, which gives a page's every head a CTA, 13.0 (both before
// keys in doubt were turned again).
__global__ void __launch_bounds__(kRopeThreads) append_rope_few_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) float2 s_cs[];        // [tokens][rot / 2]
  __shared__ uint8_t s_grown[2][1024];                  // of a key or value head whose scale has grown: the bytes before
  __shared__ int s_any;
  __shared__ Doubts s_doubts;
  const AppendArgs& ap = a.ap;
  const int tid = threadIdx.x;
  const int P = ap.c.page_size, D = ap.c.head_dim, H = ap.c.n_kv_heads, half = a.rot / 2;
  if (tid == 0) s_any = 0;
  clear_doubts(&s_doubts);             // find_block_cta has barriers
  uint64_t F = 0;
  const bool angle = tid / half >= kRopeThreads / half || phase_of_pair(a, tid % half, &F);
  bool bad = false;
  const Block f = find_block_cta(ap, int(blockIdx.x), &bad);
  if (bad && ap.status) atomicOr(ap.status, MOE_DEV_INDEX_OOB);
  if (f.b < 0) return;
  const int tokens = f.s1 - f.s0, upr = D / 16, u = tid % upr, step = kRopeThreads / upr, all = 2 * H + (a.q ? a.n_heads : 0);
  int page = f.blk < ap.width ? __ldg(ap.table + (size_t)f.b * ap.width + f.blk) : -1;
  fill_angles(a, f, F, angle, s_cs);
  __syncthreads();
  if (page < 0 || page >= ap.c.n_pages) {
    if (tid == 0 && ap.status) atomicOr(ap.status, MOE_DEV_INDEX_OOB);
    page = -1;
  }
  for (int g0 = 0; g0 < all; g0 += step) {
    const int g = g0 + tid / upr, role = g < H ? 0 : g < 2 * H ? 1 : 2, h = g - role * H;
    const bool in = g < all && (role == 2 || page >= 0);
    const int rot = role == 1 ? 0 : a.rot, kind = 16 * u >= rot ? 0 : a.interleaved ? 2 : 1;
    const int c0 = kind == 1 ? 8 * u : 16 * u, c1 = c0 + (kind == 1 ? half : 8);
    const __nv_bfloat16* src = role == 0 ? ap.k + h * ap.k_hs : role == 1 ? ap.v + h * ap.v_hs : a.q + h * a.q_hs;
    const int64_t ts = role == 0 ? ap.k_ts : role == 1 ? ap.v_ts : a.q_ts;
    float y[16];
    auto load = [&](int t) {
      const __nv_bfloat16* p = src + (int64_t)(f.t0 + t) * ts;
      turn16(*reinterpret_cast<const uint4*>(p + c0), *reinterpret_cast<const uint4*>(p + c1), s_cs + t * half + 8 * u, kind, y);
    };
    uint32_t top = 0;
    bool nonfinite = false;
    if (in)
      for (int t = 0; t < tokens; ++t) {
        load(t);
        if (role == 2) store_bf16(a.q_out + ((int64_t)(f.t0 + t) * a.n_heads + h) * D, c0, c1, y);
        else top = max(top, largest(y, &nonfinite));
      }
    float most = largest_most(__uint_as_float(top), kind), least = largest_least(__uint_as_float(top), kind);
    for (int o = 1; o < upr; o <<= 1) {
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      least = fmaxf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
      nonfinite |= __shfl_xor_sync(0xFFFFFFFFu, int(nonfinite), o) != 0;
    }
    if (!in || role == 2) continue;
    uint8_t* codes = static_cast<uint8_t*>(role ? ap.c.v_codes : ap.c.k_codes) + ((size_t)page * H + h) * P * D;
    uint8_t* scale = (role ? ap.c.v_scales : ap.c.k_scales) + (size_t)page * H + h;
    const int had = f.s0 > 0 ? int(*scale) : 0;
    int byte = kv_scale_byte(most);
    const bool turned = role == 0;
    if (turned && (nonfinite || most >= kLargest || (byte > had && kv_scale_byte(least) != byte))) {
      if (u == 0) {
        note_head(&s_doubts, h);
        s_grown[0][h] = 255;          // nothing below has to be done for it
      }
      continue;
    }
    byte = max(byte, had);
    for (int t = 0; t < tokens; ++t) {
      if (tokens > 1) load(t);
      store_codes(codes + (f.s0 + t) * D, c0, c1, y, code_factor(byte), nonfinite);
      if (turned && kind && in_doubt(y, code_factor(byte), kind)) note_doubt(&s_doubts, h, t, u);
    }
    __syncwarp(((1u << upr) - 1) << ((tid & 31) & ~(upr - 1)));     // the head's lanes have read the old scale
    if (u == 0) {
      *scale = uint8_t(byte);
      if (nonfinite && ap.status) atomicOr(ap.status, MOE_DEV_NONFINITE_INPUT);
      if (f.s0 > 0) s_grown[role][h] = uint8_t(had);
      if (f.s0 > 0 && byte > had) s_any = 1;
    }
  }
  __syncthreads();
  if (s_doubts.n || s_doubts.any_head) settle_doubts(a, f, page, 0, H, &s_doubts);
  if (f.s0 == 0 || page < 0 || !s_any) return;
  for (int g = 0; g < 2 * H; ++g) {
    const int role = g >= H, h = g - role * H, had = s_grown[role][h];
    const int byte = (role ? ap.c.v_scales : ap.c.k_scales)[(size_t)page * H + h];
    if (byte > had)
      rescale_codes(static_cast<uint8_t*>(role ? ap.c.v_codes : ap.c.k_codes) + ((size_t)page * H + h) * P * D, f.s0 * D,
                    kv_factor(had, byte));
  }
}

// NU = units of 16 channels a thread holds: page_size * head_dim / 16 / kRopeThreads,
// at least 1. gridDim.y counts groups of `heads` heads: k_groups of keys, as many of
// values, then the queries'.
template <int NU>
__global__ void __launch_bounds__(kRopeThreads, NU == 4 ? 2 : NU == 2 ? 3 : 4) append_rope_kernel(const RopeArgs a, int heads, int k_groups) {
  extern __shared__ __align__(16) float2 s_cs[];        // [tokens][rot / 2]
  __shared__ int smax[2][kRopeThreads / 32], smin[2][kRopeThreads / 32], sbad[2][kRopeThreads / 32];
  __shared__ Doubts s_doubts;
  const AppendArgs& ap = a.ap;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = ap.c.page_size, D = ap.c.head_dim, H = ap.c.n_kv_heads;
  const int group = blockIdx.y, role = group < k_groups ? 0 : group < 2 * k_groups ? 1 : 2;
  const int rot = role == 1 ? 0 : a.rot, half = rot / 2;
  uint64_t F = 0;
  const bool angle = !rot || tid / half >= kRopeThreads / half || phase_of_pair(a, tid % half, &F);
  clear_doubts(&s_doubts);             // find_block_cta has barriers
  bool bad = false;
  const Block f = find_block_cta(ap, int(blockIdx.x), &bad);
  if (bad && ap.status) atomicOr(ap.status, MOE_DEV_INDEX_OOB);
  if (f.b < 0) return;
  const int tokens = f.s1 - f.s0, upr = D / 16, n = tokens * upr;   // units per row; of the new rows
  const int row0 = tid / upr, u = tid % upr, rows = kRopeThreads / upr;
  const int kind = 16 * u >= rot ? 0 : a.interleaved ? 2 : 1;
  const int c0 = kind == 1 ? 8 * u : 16 * u, c1 = c0 + (kind == 1 ? half : 8);
  int h = (group - role * k_groups) * heads;
  const int h1 = min(h + heads, role == 2 ? a.n_heads : H);
  const __nv_bfloat16* src = role == 0 ? ap.k : role == 1 ? ap.v : a.q;
  const int64_t ts = role == 0 ? ap.k_ts : role == 1 ? ap.v_ts : a.q_ts, hs = role == 0 ? ap.k_hs : role == 1 ? ap.v_hs : a.q_hs;

  uint4 x[NU][2];
  auto fetch = [&](int head) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      if (i * kRopeThreads + tid < n) {
        const __nv_bfloat16* p = src + (int64_t)(f.t0 + row0 + i * rows) * ts + head * hs;
        x[i][0] = *reinterpret_cast<const uint4*>(p + c0);
        x[i][1] = *reinterpret_cast<const uint4*>(p + c1);
      }
    }
  };
  fetch(h);
  const int page = role < 2 && f.blk < ap.width ? __ldg(ap.table + (size_t)f.b * ap.width + f.blk) : -1;
  if (rot) {
    fill_angles(a, f, F, angle, s_cs);
    __syncthreads();
  }
  if (role < 2 && (page < 0 || page >= ap.c.n_pages)) {
    if (tid == 0 && ap.status) atomicOr(ap.status, MOE_DEV_INDEX_OOB);
    return;
  }

  const int h0 = h;
  for (int k = 0; h < h1; ++h, k ^= 1) {
    float y[NU][16];
#pragma unroll
    for (int i = 0; i < NU; ++i)     // a thread without a unit has zeros, and no angles of its own
      turn16(x[i][0], x[i][1], s_cs + (row0 + i * rows) * half + 8 * u, i * kRopeThreads + tid < n ? kind : 0, y[i]);
    if (h + 1 < h1) fetch(h + 1);
    if (role == 2) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (i * kRopeThreads + tid >= n) break;
        store_bf16(a.q_out + ((int64_t)(f.t0 + row0 + i * rows) * a.n_heads + h) * D, c0, c1, y[i]);
      }
      continue;
    }
    uint8_t* codes = static_cast<uint8_t*>(role ? ap.c.v_codes : ap.c.k_codes) + ((size_t)page * H + h) * P * D;
    uint8_t* scale = (role ? ap.c.v_scales : ap.c.k_scales) + (size_t)page * H + h;
    const int had = f.s0 > 0 ? int(*scale) : 0;
    uint32_t top = 0;
    bool nonfinite = false;
#pragma unroll
    for (int i = 0; i < NU; ++i) top = max(top, largest(y[i], &nonfinite));
    nonfinite = __any_sync(0xFFFFFFFFu, nonfinite);
    uint32_t least = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(largest_least(__uint_as_float(top), kind)));
    top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(largest_most(__uint_as_float(top), kind)));
    if (lane == 0) {
      smax[k][warp] = int(top);
      smin[k][warp] = int(least);
      sbad[k][warp] = nonfinite;
    }
    __syncthreads();   // also: everyone has read the old scale
#pragma unroll
    for (int i = 0; i < kRopeThreads / 32; ++i) {
      top = max(top, uint32_t(smax[k][i]));
      least = max(least, uint32_t(smin[k][i]));
      nonfinite |= sbad[k][i] != 0;
    }
    int byte = kv_scale_byte(__uint_as_float(top));
    const bool turned = rot != 0;      // the branch is the same for all threads
    if (turned && (nonfinite || __uint_as_float(top) >= kLargest || (byte > had && kv_scale_byte(__uint_as_float(least)) != byte))) {
      if (tid == 0) note_head(&s_doubts, h);
      continue;
    }
    byte = max(byte, had);
    if (tid == 0) {
      *scale = uint8_t(byte);
      if (nonfinite && ap.status) atomicOr(ap.status, MOE_DEV_NONFINITE_INPUT);
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      if (i * kRopeThreads + tid >= n) break;
      store_codes(codes + (f.s0 + row0 + i * rows) * D, c0, c1, y[i], code_factor(byte), nonfinite);
      if (turned && kind && in_doubt(y[i], code_factor(byte), kind)) note_doubt(&s_doubts, h, row0 + i * rows, u);
    }
    if (byte > had && f.s0 > 0) rescale_codes(codes, f.s0 * D, kv_factor(had, byte));
  }
  if (!rot || role == 2) return;
  __syncthreads();
  if (s_doubts.n || s_doubts.any_head) settle_doubts(a, f, page, h0, h1, &s_doubts);
}

}  // namespace

int launch_kv_append_rope(const RopeArgs& a, const DeviceInfo& di, cudaStream_t s) {
  const int P = a.ap.c.page_size, D = a.ap.c.head_dim;
  // every sequence touches at most len / P + 2 pages, and no more than its tokens
  const int64_t most = (int64_t)a.ap.total / P + 2 * (int64_t)a.ap.n_seq;
  const int nb = int(std::min(most, (int64_t)a.ap.total)) + 1;   // the last one looks at every sequence
  // Heads a CTA: more share one table of angles, while there are CTAs for every SM several times over (12,345 tokens:
  // one 64.1 us, two 47.9, four 42.9, before keys in doubt were turned again).
  const int H = a.ap.c.n_kv_heads, n_q = a.q ? a.n_heads : 0;
  int heads = 1;
  while (heads < 4 && (int64_t)nb * (2 * H + n_q) >= (int64_t)kRopeCtas * di.sm_count * 2 * heads) heads *= 2;
  const int k_groups = (H + heads - 1) / heads;
  const dim3 grid(nb, 2 * k_groups + (n_q + heads - 1) / heads);
  const uint32_t smem = uint32_t(P) * (a.rot / 2) * sizeof(float2);
  auto room = [&](auto kernel) -> int {
    if (smem <= 48 * 1024 - 4096) return MOE_OK;         // what a kernel may have without asking
    MOE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
    return MOE_OK;
  };
  auto go = [&](auto kernel) -> int {
    const int st = room(kernel);
    if (st != MOE_OK) return st;
    kernel<<<grid, kRopeThreads, smem, s>>>(a, heads, k_groups);
    return launch_status();
  };
  // A token or two a sequence: a CTA for all their heads. The host knows the mean alone: 64 sequences of two tokens take
  // 9.9 us here, but 64 single tokens beside a chunk of 64 (128 tokens of 65 sequences) take 77, since one CTA has the
  // chunk's page; with 67 in the chunk the other kernel has them all, 15.0.
  if (a.ap.total <= 2 * (int64_t)a.ap.n_seq) {
    const int st = room(append_rope_few_kernel);
    if (st != MOE_OK) return st;
    append_rope_few_kernel<<<nb, kRopeThreads, smem, s>>>(a);
    return launch_status();
  }
  switch (P * D / 16 / kRopeThreads) {
    case 0:
    case 1: return go(append_rope_kernel<1>);
    case 2: return go(append_rope_kernel<2>);
    default: return go(append_rope_kernel<4>);
  }
}

}  // namespace moe
