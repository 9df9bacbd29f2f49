// Attention over whole prompts (packed sequences, grouped heads).
//
// Simple form: four threads per query row, each holding a quarter of the
// channels of q and of the output; 32 rows of one head per CTA, keys and
// values in tiles of 32 through shared memory, softmax with a running maximum
// and sum, everything in fp32. Keys that a row does not see are skipped.
#include "attn.h"
#include "fp8kv.cuh"

namespace moe {
namespace {

constexpr int kRowsPerCta = 32, kSplit = 4, kKeys = 32;
constexpr int kThreads = kRowsPerCta * kSplit;

template <int D>
__global__ void __launch_bounds__(kThreads) prefill_simple_kernel(const PrefillArgs a) {
  constexpr int DS = D / kSplit;
  __shared__ __align__(16) __nv_bfloat16 ks[kKeys][D], vs[kKeys][D];
  __shared__ int s_b, s_tile;
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {
    bool bad = false;
    int before = 0, fb = -1, ft = 0;
    for (int b0 = 0; b0 < a.n_seq && fb < 0; b0 += 32) {
      int c0 = 0, c1 = 0, k0, k1;
      if (b0 + lane < a.n_seq) {
        packed_range(a.cu_q, b0 + lane, a.total_q, &c0, &c1, &bad);
        packed_range(a.cu_k, b0 + lane, a.total_k, &k0, &k1, &bad);
      }
      const int n = (c1 - c0 + kRowsPerCta - 1) / kRowsPerCta;
      int incl = n;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
      }
      const int lo = before + incl - n, x = blockIdx.x;
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, x >= lo && x < lo + n);
      if (hit) {
        fb = b0 + __ffs(hit) - 1;
        ft = x - __shfl_sync(0xFFFFFFFFu, lo, __ffs(hit) - 1);
      }
      before += __shfl_sync(0xFFFFFFFFu, incl, 31);
    }
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      s_b = fb;
      s_tile = ft;
      if (bad && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    }
  }
  __syncthreads();
  if (s_b < 0) return;
  bool ignore = false;
  int q0, q1, k0, k1;
  packed_range(a.cu_q, s_b, a.total_q, &q0, &q1, &ignore);
  packed_range(a.cu_k, s_b, a.total_k, &k0, &k1, &ignore);
  const int nq = q1 - q0, nk = k1 - k0;
  const int r = s_tile * kRowsPerCta + tid / kSplit, part = tid % kSplit;
  const int hq = blockIdx.y, hk = hq / (a.n_heads / a.n_kv);
  const int vis = r < nq ? (a.causal ? min(max(r + nk - nq + 1, 0), nk) : nk) : 0;
  const int last = min(s_tile * kRowsPerCta + kRowsPerCta, nq) - 1;   // last row of the tile
  const int most = a.causal ? min(max(last + nk - nq + 1, 0), nk) : nk;
  float q[DS], o[DS];
#pragma unroll
  for (int i = 0; i < DS; ++i) {
    q[i] = r < nq ? __bfloat162float(a.q[(q0 + r) * a.q_ts + hq * a.q_hs + part * DS + i]) : 0.0f;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int t0 = 0; t0 < most; t0 += kKeys) {
    __syncthreads();
    for (int v = tid; v < kKeys * D / 8; v += kThreads) {
      const int row = v / (D / 8), ch = (v % (D / 8)) * 8;
      if (t0 + row < nk) {
        *reinterpret_cast<uint4*>(&ks[row][ch]) = *reinterpret_cast<const uint4*>(a.k + (k0 + t0 + row) * a.k_ts + hk * a.k_hs + ch);
        *reinterpret_cast<uint4*>(&vs[row][ch]) = *reinterpret_cast<const uint4*>(a.v + (k0 + t0 + row) * a.v_ts + hk * a.v_hs + ch);
      }
    }
    __syncthreads();
    for (int j = 0; j < kKeys && t0 + j < most; ++j) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < DS; ++i) s = fmaf(q[i], __bfloat162float(ks[j][part * DS + i]), s);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
      s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
      if (t0 + j >= vis) continue;
      s *= a.scale;
      if (s > m) {
        const float f = expf(m - s);
        m = s;
        l *= f;
#pragma unroll
        for (int i = 0; i < DS; ++i) o[i] *= f;
      }
      const float p = s == -INFINITY ? 0.0f : expf(s - m);
      l += p;
#pragma unroll
      for (int i = 0; i < DS; ++i) o[i] = fmaf(p, __bfloat162float(vs[j][part * DS + i]), o[i]);
    }
  }
  if (r >= nq) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < DS; ++i)
    a.out[((size_t)(q0 + r) * a.n_heads + hq) * D + part * DS + i] = __float2bfloat16_rn(o[i] * inv);
  if (a.lse && part == 0) a.lse[(size_t)(q0 + r) * a.n_heads + hq] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace

int launch_attn_prefill(const PrefillArgs& a, const DeviceInfo& di, cudaStream_t s) {
  (void)di;
  // tiles of all sequences, and one block more, which looks at every sequence
  const dim3 grid(unsigned(a.total_q / kRowsPerCta + a.n_seq + 1), a.n_heads);
  if (a.D == 128)
    prefill_simple_kernel<128><<<grid, kThreads, 0, s>>>(a);
  else
    prefill_simple_kernel<64><<<grid, kThreads, 0, s>>>(a);
  return launch_status();
}

}  // namespace moe
