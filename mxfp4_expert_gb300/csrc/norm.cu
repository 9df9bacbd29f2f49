// The norms on both sides of a block's half, with its gate and residual.
//
//   n = a * rsqrt(mean a^2 + eps) * (offset + wp)      (n = a without wp)
//   y = x + scale * gate * n
//   h = y * rsqrt(mean y^2 + eps) * (offset + wn)
//
// One CTA per row: the row stays in registers from the read of a and x to the
// writes of y and h, so every element crosses memory once. Bound by HBM (8 bytes
// an element with a bf16 stream); a single row by the launch and its chain of a
// read and two sums over the CTA. h comes from y before its rounding.
#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kNormMaxThreads = 1024;

// Sum over the CTA; s: one float a warp, not used by the sum before.
__device__ __forceinline__ float cta_sum(float v, float* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = int(blockDim.x) >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (lane == 0) s[warp] = v;
  __syncthreads();
  v = lane < n ? s[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float cta_max(float v, float* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = int(blockDim.x) >> 5;
  v = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v)));   // v >= 0
  __syncthreads();
  if (lane == 0) s[warp] = v;
  __syncthreads();
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, lane < n ? __float_as_uint(s[lane]) : 0u));
}

// 1 / sqrt(mean v^2 + eps) of the row. Where the squares' sum leaves what fp32
// holds well, they are summed once more in units of the row's largest value.
template <int V>
__device__ __forceinline__ float row_rstd(const float (&v)[V][8], float d, float eps, float* s) {
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(v[i][e], v[i][e], q);
  q = cta_sum(q, s);
  if (q >= 1e-30f && q <= 1e37f) return rsqrtf(q / d + eps);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[i][e]));
  m = cta_max(m, s);
  if (!(m > 0.0f && m <= 3.4028235e38f) || q != q) return rsqrtf(q / d + eps);
  const int ex = min(max(int(__float_as_uint(m) >> 23) - 127, -125), 126);
  const float f = __uint_as_float(uint32_t(127 - ex) << 23);   // 2^-ex
  q = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(v[i][e] * f, v[i][e] * f, q);
  __syncthreads();
  q = cta_sum(q, s);
  const float e2 = eps * f * f;
  return e2 <= 3.4028235e38f ? f * rsqrtf(q / d + e2) : rsqrtf(eps);
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(u[i]);
    v[2 * i + 1] = bf16_hi(u[i]);
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
// Eight elements at column c of a row; kF32: of fp32.
template <bool kF32>
__device__ __forceinline__ void load8(const void* row, int c, float (&v)[8]) {
  if constexpr (kF32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + c);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(row) + c), v);
  }
}
template <bool kF32>
__device__ __forceinline__ void store8(void* row, int c, const float (&v)[8]) {
  if constexpr (kF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + c);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(row) + c) = pack8(v);
  }
}

// V: 8-element vectors a thread holds.
template <int V, bool kF32>
__global__ void __launch_bounds__(kNormMaxThreads) block_norm_kernel(const NormArgs a) {
  __shared__ float s[2][32];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, nt = blockDim.x;
  constexpr int kBytes = kF32 ? 4 : 2;
  const void* xr = static_cast<const char*>(a.x) + t * a.x_rs * kBytes;
  float y[V][8], n[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (tid + i * nt) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[i][e] = n[i][e] = 0.0f;
    if (c < a.d) {
      load8<kF32>(xr, c, y[i]);
      if (a.a) load8<false>(a.a + t * a.a_rs, c, n[i]);
    }
  }
  if (a.a) {
    const float r = a.wp ? row_rstd<V>(n, float(a.d), a.eps, s[0]) : 1.0f;
    void* yr = static_cast<char*>(a.y) + t * a.y_rs * kBytes;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (tid + i * nt) * 8;
      if (c >= a.d) break;
      float w[8];
      if (a.wp) {
        load8<false>(a.wp, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[i][e] = n[i][e] * r * (a.offset + w[e]);
      }
      if (a.gate) {
        load8<false>(a.gate + t * a.g_rs, c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) n[i][e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] = fmaf(a.scale, n[i][e], y[i][e]);
      store8<kF32>(yr, c, y[i]);
    }
  }
  if (a.h) {
    const float r = row_rstd<V>(y, float(a.d), a.eps, s[1]);
    __nv_bfloat16* hr = a.h + t * a.h_rs;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (tid + i * nt) * 8;
      if (c >= a.d) break;
      float w[8];
      if (a.wn) load8<false>(a.wn, c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] = y[i][e] * r * (a.wn ? a.offset + w[e] : 1.0f);
      store8<false>(hr, c, y[i]);
    }
  }
}

template <int V>
void launch_v(const NormArgs& a, int threads, cudaStream_t s) {
  if (a.fp32) block_norm_kernel<V, true><<<a.T, threads, 0, s>>>(a);
  else block_norm_kernel<V, false><<<a.T, threads, 0, s>>>(a);
}

}  // namespace

int launch_block_norm(const NormArgs& a, const DeviceInfo&, cudaStream_t s) {
  const int vecs = a.d / 8;
  const int v = vecs <= 256 ? 1 : vecs <= 2048 ? 2 : 4;
  const int threads = int(round_up((vecs + v - 1) / v, 32));
  if (v == 1) launch_v<1>(a, threads, s);
  else if (v == 2) launch_v<2>(a, threads, s);
  else launch_v<4>(a, threads, s);
  return launch_status();
}

}  // namespace moe
