// The norms on both sides of a block's half, with its gate and residual.
//
//   n = a * rsqrt(mean a^2 + eps) * (offset + wp)      (n = a without wp)
//   y = x + scale * gate * n
//   h = y * rsqrt(mean y^2 + eps) * (offset + wn)
//
// A CTA takes a row at a time, which stays in registers from the read of a and x to
// the writes of y and h, so every element crosses memory once; the next row's reads
// are on their way meanwhile, and the weights stay for all rows. h comes from y
// before its rounding.
//
// Bound by the reads in flight: 4,096 rows of 2,560 (8 bytes an element with a bf16
// stream) take 17.8 us, 0.69 of the copy rate, and three CTAs of 160 threads at 128
// registers are all an SM holds, some 30 KB on their way; DRAM carries 2.6 TB/s where the
// writes stay in L2, and the time is the same where they do not. 1,001 of 7,168 with an
// fp32 stream and a gate per token: 20.6 us (0.72). A ring of bulk copies in place of the
// reads into registers took 21.2 to 23.8 and 21.9 us. One row of 2,560: 3.4 us, the
// launch and a chain of a read and two sums over the CTA.
#include "block.h"
#include "common.cuh"
#include "f32x2.cuh"

namespace moe {
namespace {

constexpr int kNormThreads = 512;    // at most: a thread may then have 128 registers

// Sum over the CTA; s: one float a warp, not used by the sum before.
__device__ __forceinline__ float cta_sum(float v, float* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = int(blockDim.x) >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (lane == 0) s[warp] = v;
  __syncthreads();
  if (n <= 8) {                       // fewer instructions than five more shuffles
    v = 0.0f;
    for (int i = 0; i < n; ++i) v += s[i];
    return v;
  }
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

// Eight elements, two to a 64-bit register: an instruction takes both.
struct Eight {
  uint64_t p[4];
};
__device__ __forceinline__ Eight widen(const uint4& w) {          // bf16
  return {{pack2(bf16_lo(w.x), bf16_hi(w.x)), pack2(bf16_lo(w.y), bf16_hi(w.y)), pack2(bf16_lo(w.z), bf16_hi(w.z)),
           pack2(bf16_lo(w.w), bf16_hi(w.w))}};
}
__device__ __forceinline__ uint32_t narrow(uint64_t v) {
  float lo, hi;
  unpack2(v, lo, hi);
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 narrow(const Eight& v) {
  return make_uint4(narrow(v.p[0]), narrow(v.p[1]), narrow(v.p[2]), narrow(v.p[3]));
}
// Eight elements as they lie in memory.
template <bool kF32>
struct Raw {
  uint4 w[kF32 ? 2 : 1];
};
template <bool kF32>
__device__ __forceinline__ Raw<kF32> load_raw(const void* row, int c) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + c * (kF32 ? 4 : 2));
  Raw<kF32> r;
  r.w[0] = p[0];
  if constexpr (kF32) r.w[1] = p[1];
  return r;
}
template <bool kF32>
__device__ __forceinline__ Eight widen(const Raw<kF32>& r) {
  if constexpr (kF32)
    return {{uint64_t(r.w[0].x) | uint64_t(r.w[0].y) << 32, uint64_t(r.w[0].z) | uint64_t(r.w[0].w) << 32,
             uint64_t(r.w[1].x) | uint64_t(r.w[1].y) << 32, uint64_t(r.w[1].z) | uint64_t(r.w[1].w) << 32}};
  else
    return widen(r.w[0]);
}
template <bool kF32>
__device__ __forceinline__ void store8(void* row, int c, const Eight& v) {
  if constexpr (kF32) {
    ulonglong2* p = reinterpret_cast<ulonglong2*>(static_cast<float*>(row) + c);
    p[0] = make_ulonglong2(v.p[0], v.p[1]);
    p[1] = make_ulonglong2(v.p[2], v.p[3]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(row) + c) = narrow(v);
  }
}

__device__ __forceinline__ Eight constant(float v) {
  const uint64_t p = pack2(v, v);
  return {{p, p, p, p}};
}
__device__ __forceinline__ Eight product(const Eight& a, const Eight& b) {
  return {{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1]), mul2(a.p[2], b.p[2]), mul2(a.p[3], b.p[3])}};
}

// 1 / sqrt(mean v^2 + eps) of the row. Where the squares' sum leaves what fp32
// holds well, v is brought to other units, in which the result then is: those of its
// largest value where that is small (of subnormal numbers the result would else be
// more than fp32 holds), 2^72 where it is large.
template <int V>
__device__ __forceinline__ float row_rstd(Eight (&v)[V], float d, float eps, float* s) {
  auto squares = [&]() {
    uint64_t q[2] = {0, 0};            // two zeros each
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e & 1] = fma2(v[i].p[e], v[i].p[e], q[e & 1]);
    float lo, hi;
    unpack2(add2(q[0], q[1]), lo, hi);
    return lo + hi;
  };
  float q = cta_sum(squares(), s);
  if (q >= 1e-30f && q <= 1e37f) return rsqrtf(q / d + eps);
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo, hi;
      unpack2(v[i].p[e], lo, hi);
      m = fmaxf(m, fmaxf(fabsf(lo), fabsf(hi)));
    }
  m = cta_max(m, s);
  if (!(m > 0.0f && m <= 3.4028235e38f) || q != q) return rsqrtf(q / d + eps);
  const int ex = m < 1.0f ? max(int(__float_as_uint(m) >> 23) - 127, -125) : 72;
  const float f = __uint_as_float(uint32_t(127 - ex) << 23), e2 = eps * f * f;   // 2^-ex
  if (e2 > 3.4028235e38f) return rsqrtf(eps);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = product(v[i], constant(f));
  __syncthreads();
  q = cta_sum(squares(), s);
  return rsqrtf(q / d + e2);
}

// What n (of the half's output) and y are multiplied with, beside their norms:
// scale (offset + wp) gate, the gate where all rows share it, and offset + wn.
template <int V>
struct Weights {
  Eight a[V], h[V];
};
__device__ __forceinline__ Eight plus(const Eight& a, const Eight& b) {
  return {{add2(a.p[0], b.p[0]), add2(a.p[1], b.p[1]), add2(a.p[2], b.p[2]), add2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ Eight weight_a(const NormArgs& a, int c) {
  Eight w = constant(a.scale);
  if (a.wp) w = product(w, plus(constant(a.offset), widen(*reinterpret_cast<const uint4*>(a.wp + c))));
  if (a.gate && a.g_rs == 0) w = product(w, widen(*reinterpret_cast<const uint4*>(a.gate + c)));
  return w;
}
__device__ __forceinline__ Eight weight_h(const NormArgs& a, int c) {
  return a.wn ? plus(constant(a.offset), widen(*reinterpret_cast<const uint4*>(a.wn + c))) : constant(1.0f);
}

// One row: y and h from x, the half's output n and the gate gt (if gate_row); weights
// w where KEEP, else read. `next` runs once the row is out of x, n and gt. s0, s1:
// room for both sums, not used for the row before.
template <int V, bool kF32, bool HAS_A, bool KEEP, class Next>
__device__ __forceinline__ void norm_row(const NormArgs& a, int64_t t, const Raw<kF32> (&x)[V], const uint4 (&n)[V],
                                         const uint4 (&gt)[V], bool gate_row, const Weights<V>& w, float* s0, float* s1,
                                         Next next) {
  const int tid = threadIdx.x, nt = blockDim.x;
  Eight y[V], z[V];
  uint4 g[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    y[i] = widen<kF32>(x[i]);
    if (HAS_A) z[i] = widen(n[i]);
    g[i] = gt[i];
  }
  next();
  if (HAS_A) {
    const float r = a.wp ? row_rstd<V>(z, float(a.d), a.eps, s0) : 1.0f;
    void* yr = static_cast<char*>(a.y) + t * a.y_rs * (kF32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (tid + i * nt) * 8;
      if (c >= a.d) break;
      z[i] = product(z[i], constant(r));
      if (gate_row) z[i] = product(z[i], widen(g[i]));
      const Eight f = KEEP ? w.a[i] : weight_a(a, c);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[i].p[e] = fma2(z[i].p[e], f.p[e], y[i].p[e]);
      store8<kF32>(yr, c, y[i]);
    }
  }
  if (a.h) {
    const float r = row_rstd<V>(y, float(a.d), a.eps, s1);
    __nv_bfloat16* hr = a.h + t * a.h_rs;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (tid + i * nt) * 8;
      if (c >= a.d) break;
      store8<false>(hr, c, product(product(y[i], constant(r)), KEEP ? w.h[i] : weight_h(a, c)));
    }
  }
}

// V: 8-element vectors a thread holds. HAS_A: not only a norm of x. AHEAD: weights
// stay in registers for all rows of the CTA, and the next row is read while one is
// worked on; for that rows must not be too long.
template <int V, bool kF32, bool HAS_A, bool AHEAD>
__global__ void __launch_bounds__(kNormThreads) block_norm_kernel(const NormArgs a) {
  __shared__ float s[4][32];
  const int tid = threadIdx.x, nt = blockDim.x;
  const bool gate_row = HAS_A && a.gate && a.g_rs != 0;
  Raw<kF32> x[V];
  uint4 n[V], gt[V];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (tid + i * nt) * 8;
      if (c < a.d) {
        x[i] = load_raw<kF32>(static_cast<const char*>(a.x) + t * a.x_rs * (kF32 ? 4 : 2), c);
        if (HAS_A) n[i] = *reinterpret_cast<const uint4*>(a.a + t * a.a_rs + c);
        if (gate_row) gt[i] = *reinterpret_cast<const uint4*>(a.gate + t * a.g_rs + c);
      }
    }
  };
  Weights<V> w;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = Raw<kF32>{};
    n[i] = gt[i] = make_uint4(0, 0, 0, 0);
    w.a[i] = w.h[i] = constant(0.0f);
  }
  fetch(blockIdx.x);
  if (AHEAD) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (tid + i * nt) * 8;
      if (c < a.d) {
        if (HAS_A) w.a[i] = weight_a(a, c);
        w.h[i] = weight_h(a, c);
      }
    }
  }
  int k = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, k ^= 2) {
    if (!AHEAD && t != blockIdx.x) fetch(t);
    norm_row<V, kF32, HAS_A, AHEAD>(a, t, x, n, gt, gate_row, w, s[k], s[k + 1], [&] {
      if (AHEAD && t + gridDim.x < a.T) fetch(t + gridDim.x);
    });
  }
}

template <int V, bool kF32, bool HAS_A>
int launch_norm(const NormArgs& a, int threads, const DeviceInfo& di, cudaStream_t s) {
  constexpr bool kAhead = V <= 3;
  int per_sm = 8;
  if (kAhead && a.T > di.sm_count)
    MOE_CUDA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, block_norm_kernel<V, kF32, HAS_A, kAhead>, threads, 0));
  const int64_t most = (int64_t)di.sm_count * (per_sm > 0 ? per_sm : 1);
  block_norm_kernel<V, kF32, HAS_A, kAhead><<<int(a.T < most ? a.T : most), threads, 0, s>>>(a);
  return launch_status();
}
template <int V>
int launch_v(const NormArgs& a, const DeviceInfo& di, cudaStream_t s) {
  const int threads = int(round_up((a.d / 8 + V - 1) / V, 32));
  if (a.fp32) return a.a ? launch_norm<V, true, true>(a, threads, di, s) : launch_norm<V, true, false>(a, threads, di, s);
  return a.a ? launch_norm<V, false, true>(a, threads, di, s) : launch_norm<V, false, false>(a, threads, di, s);
}

}  // namespace

// Vectors a thread. One up to 256 threads; with more of them a row's sums cost more than its channels, and two are
// better (4,096 rows of 2,560: 320 threads with one 20.5 us, 160 with two 17.8), more where 512 threads need them. Of
// those, parts leave registers for local memory: the weights of three vectors (128 and 232 bytes a thread with a bf16 and
// an fp32 stream), some of four (96, 128), most of eight (880, 928). Three with the next row ahead against four without,
// 1,000 rows of 12,288: 29 to 47.8 us; a row shared by a cluster of two CTAs 47.2. 1,000 rows of 16,384: 42 us, 500 of
// 32,768 with an fp32 stream 121.
int launch_block_norm(const NormArgs& a, const DeviceInfo& di, cudaStream_t s) {
  const int vecs = a.d / 8;
  if (vecs <= 256) return launch_v<1>(a, di, s);
  if (vecs <= 2 * kNormThreads) return launch_v<2>(a, di, s);
  if (vecs <= 3 * kNormThreads) return launch_v<3>(a, di, s);
  if (vecs <= 4 * kNormThreads) return launch_v<4>(a, di, s);
  return launch_v<8>(a, di, s);
}

}  // namespace moe
