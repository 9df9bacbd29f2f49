// Append to the 8-bit cache with the position rotation on the way, and the
// queries' rotation beside it.
//
// Pair j of a head is turned by the angle p f_j, p the token's position. The
// angle is taken in turns and in integers: F_j = f_j / 2 pi (without its whole
// part) times 2^64, and p F_j modulo 2^64 is the angle's fraction of a turn, to
// p 2^-64 whatever p is. Its top 32 bits give quadrant and remainder, cosine and
// sine of the remainder are their Taylor series.
//
// A CTA takes one page's new tokens: the cosines and sines of all of them into
// shared memory, then of one key or value head the values into registers, their
// maximum, the page's scale and the codes (as append_kernel, which has no
// rotation), or several query heads one after another. Bound by HBM: 3 bytes a
// key or value, 4 a query's channel.
#include <algorithm>

#include "attn.h"
#include "fp8kv.cuh"
#include "kvblock.cuh"

namespace moe {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeQHeads = 4;      // query heads a CTA rotates

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

// Eight rotated channels at column col of a row: w, and where pairs lie r / 2
// apart the other halves' channels o; cs: the row's cosines and sines.
__device__ __forceinline__ void rotate8(const uint4& w, const uint4& o, const float2* cs, int col, int rot,
                                        bool interleaved, float (&y)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w}, p[4] = {o.x, o.y, o.z, o.w};
  if (col >= rot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = bf16_lo(u[i]);
      y[2 * i + 1] = bf16_hi(u[i]);
    }
  } else if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = cs[col / 2 + i];
      const float a = bf16_lo(u[i]), b = bf16_hi(u[i]);
      y[2 * i] = a * t.x - b * t.y;
      y[2 * i + 1] = b * t.x + a * t.y;
    }
  } else {
    const bool second = col >= rot / 2;
    const float2* c = cs + (second ? col - rot / 2 : col);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = c[2 * i], t2 = c[2 * i + 1];
      y[2 * i] = bf16_lo(u[i]) * t.x + (second ? bf16_lo(p[i]) : -bf16_lo(p[i])) * t.y;
      y[2 * i + 1] = bf16_hi(u[i]) * t2.x + (second ? bf16_hi(p[i]) : -bf16_hi(p[i])) * t2.y;
    }
  }
}

// NV = vectors of 8 channels a thread holds: page_size * head_dim / 8 / kRopeThreads, at least 1.
template <int NV>
__global__ void __launch_bounds__(kRopeThreads) append_rope_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) float2 s_cs[];        // [tokens][rot / 2]
  __shared__ Block sblk;
  __shared__ int smax[kRopeThreads / 32], sbad[kRopeThreads / 32];
  const AppendArgs& ap = a.ap;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) {
    bool bad = false;
    const Block f = find_block(ap, int(blockIdx.x), &bad);
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      sblk = f;
      if (bad && ap.status) atomicOr(ap.status, MOE_DEV_INDEX_OOB);
    }
  }
  __syncthreads();
  const Block f = sblk;
  if (f.b < 0) return;
  const int P = ap.c.page_size, D = ap.c.head_dim, H = ap.c.n_kv_heads, role = blockIdx.y;
  const bool is_q = role >= 2 * H, is_v = !is_q && role >= H;
  const int rot = is_v ? 0 : a.rot, half = rot / 2, tokens = f.s1 - f.s0;
  const int cpr = D / 8, n = tokens * cpr;              // vectors per row; of the new rows
  const int row = tid / cpr, col = (tid % cpr) * 8, rows = kRopeThreads / cpr;
  // where the other halves of the pairs are
  const int other = a.interleaved || col >= rot ? 0 : col >= half ? -half : half;
  const __nv_bfloat16* src;
  int64_t ts;
  int h = is_q ? (role - 2 * H) * kRopeQHeads : is_v ? role - H : role;
  if (is_q) src = a.q, ts = a.q_ts;
  else if (is_v) src = ap.v + h * ap.v_hs, ts = ap.v_ts;
  else src = ap.k + h * ap.k_hs, ts = ap.k_ts;

  if (rot) {   // cosines and sines of the page's new tokens; a thread keeps its frequency
    const int j = tid % half, first = tid / half, step = kRopeThreads / half;
    if (first < step) {
      const int64_t p0 = (int64_t)__ldg(a.rope_start + f.b) + ((int64_t)f.blk * P + f.s0 - __ldg(ap.start + f.b));
      double turns = double(__ldg(a.inv_freq + j)) * 0.15915494309189533577;
      turns -= floor(turns);
      const uint64_t F = uint64_t(turns * 18446744073709551616.0);
      for (int t = first; t < tokens; t += step) s_cs[t * half + j] = turn(uint32_t((uint64_t(p0 + t) * F) >> 32));
    }
    __syncthreads();
  }

  if (is_q) {
    const int h1 = min(h + kRopeQHeads, a.n_heads);
    for (; h < h1; ++h) {
      const __nv_bfloat16* s = src + h * a.q_hs;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int r = row + i * rows;
        if (i * kRopeThreads + tid >= n) break;
        const __nv_bfloat16* p = s + (int64_t)(f.t0 + r) * ts + col;
        const uint4 w = *reinterpret_cast<const uint4*>(p), o = *reinterpret_cast<const uint4*>(p + other);
        float y[8];
        rotate8(w, o, s_cs + r * half, col, rot, a.interleaved, y);
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b[e]) : "f"(y[2 * e + 1]), "f"(y[2 * e]));
        *reinterpret_cast<uint4*>(a.q_out + ((int64_t)(f.t0 + r) * a.n_heads + h) * D + col) =
            make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
    return;
  }

  const int page = f.blk < ap.width ? __ldg(ap.table + (size_t)f.b * ap.width + f.blk) : -1;
  float y[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int r = row + i * rows;
    if (i * kRopeThreads + tid < n) {
      const __nv_bfloat16* p = src + (int64_t)(f.t0 + r) * ts + col;
      const uint4 w = *reinterpret_cast<const uint4*>(p), o = *reinterpret_cast<const uint4*>(p + other);
      rotate8(w, o, s_cs + r * half, col, rot, a.interleaved, y[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] = 0.0f;
    }
  }
  if (page < 0 || page >= ap.c.n_pages) {
    if (tid == 0 && ap.status) atomicOr(ap.status, MOE_DEV_INDEX_OOB);
    return;
  }
  uint8_t* codes = static_cast<uint8_t*>(is_v ? ap.c.v_codes : ap.c.k_codes) + ((size_t)page * H + h) * P * D;
  uint8_t* scale = (is_v ? ap.c.v_scales : ap.c.k_scales) + (size_t)page * H + h;
  const int had = f.s0 > 0 ? int(*scale) : 0;
  uint32_t top = 0;            // the largest finite magnitude's bits
  bool nonfinite = false;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t m = __float_as_uint(y[i][e]) & 0x7FFFFFFFu;
      const bool inf = m >= 0x7F800000u;
      nonfinite |= inf;
      top = max(top, inf ? 0u : m);
    }
  nonfinite = __any_sync(0xFFFFFFFFu, nonfinite);
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) {
    smax[warp] = int(top);
    sbad[warp] = nonfinite;
  }
  __syncthreads();   // also: everyone has read the old scale
#pragma unroll
  for (int i = 0; i < kRopeThreads / 32; ++i) {
    top = max(top, uint32_t(smax[i]));
    nonfinite |= sbad[i] != 0;
  }
  const int byte = max(kv_scale_byte(__uint_as_float(top)), had);
  if (tid == 0) {
    *scale = uint8_t(byte);
    if (nonfinite && ap.status) atomicOr(ap.status, MOE_DEV_NONFINITE_INPUT);
  }
  // 2^(127 - byte); 2^-127 and 2^-128 are subnormal
  const float f1 = byte <= 253 ? pow2(127 - byte) : __uint_as_float(0x00800000u >> (byte - 253));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * kRopeThreads + tid >= n) break;
    uint32_t q[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo = y[i][2 * j] * f1, hi = y[i][2 * j + 1] * f1;
      if (nonfinite) {   // inf takes the code of NaN: there is none for it
        if (!(fabsf(y[i][2 * j]) <= 3.4028235e38f)) lo = __int_as_float(0x7FC00000);
        if (!(fabsf(y[i][2 * j + 1]) <= 3.4028235e38f)) hi = __int_as_float(0x7FC00000);
      }
      q[j >> 1] |= uint32_t(f32x2_to_e4m3x2(lo, hi)) << (16 * (j & 1));
    }
    *reinterpret_cast<uint2*>(codes + (f.s0 + row + i * rows) * D + col) = make_uint2(q[0], q[1]);
  }
  if (byte > had && f.s0 > 0) {   // older codes, in units of the new scale
    const float fo = kv_factor(had, byte);
    for (int v = tid; v < f.s0 * D / 16; v += kRopeThreads) {
      uint4* p = reinterpret_cast<uint4*>(codes) + v;
      uint4 c = *p;
      c.x = kv_rescale4(c.x, fo);
      c.y = kv_rescale4(c.y, fo);
      c.z = kv_rescale4(c.z, fo);
      c.w = kv_rescale4(c.w, fo);
      *p = c;
    }
  }
}

}  // namespace

int launch_kv_append_rope(const RopeArgs& a, cudaStream_t s) {
  const int P = a.ap.c.page_size, D = a.ap.c.head_dim;
  // every sequence touches at most len / P + 2 pages, and no more than its tokens
  const int64_t most = (int64_t)a.ap.total / P + 2 * (int64_t)a.ap.n_seq;
  const int nb = int(std::min(most, (int64_t)a.ap.total)) + 1;   // the last one looks at every sequence
  const dim3 grid(nb, 2 * a.ap.c.n_kv_heads + (a.q ? (a.n_heads + kRopeQHeads - 1) / kRopeQHeads : 0));
  const uint32_t smem = uint32_t(P) * (a.rot / 2) * sizeof(float2);
  auto go = [&](auto kernel) -> int {
    MOE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
    kernel<<<grid, kRopeThreads, smem, s>>>(a);
    return launch_status();
  };
  switch (P * D / 8 / kRopeThreads) {
    case 0:
    case 1: return go(append_rope_kernel<1>);
    case 2: return go(append_rope_kernel<2>);
    case 4: return go(append_rope_kernel<4>);
    default: return go(append_rope_kernel<8>);
  }
}

}  // namespace moe
