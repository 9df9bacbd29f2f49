// Attention of chunks of new tokens over the 8-bit paged cache: one warp per
// (token, head), one pass over the positions with the running maximum and sum.
#include "attn.h"
#include "fp8kv.cuh"

namespace moe {
namespace {

constexpr float kLn2f = 0.6931471805599453f, kLog2ef = 1.4426950408889634f;

template <int D>
__global__ void __launch_bounds__(128) chunk_simple_kernel(const ChunkArgs a) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y, G = a.n_heads / a.c.n_kv_heads, hk = h / G, P = a.c.page_size;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (t >= a.total_q) return;
  // the token's sequence
  int b = -1, c0 = 0, c1 = 0;
  bool bad = false;
  if (t == 0 && h == 0)
    for (int i = lane; i < a.n_seq; i += 32) packed_range(a.cu_q, i, a.total_q, &c0, &c1, &bad);
  if (bad && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
  bad = false;
  for (int i = 0; i < a.n_seq && b < 0; ++i) {
    packed_range(a.cu_q, i, a.total_q, &c0, &c1, &bad);
    if (t >= c0 && t < c1) b = i;
  }
  if (b < 0) return;
  const int cap = a.width * P, L0 = __ldg(a.lengths + b), L = min(max(L0, 0), cap);
  if (a.status && lane == 0 && (bad || L != L0)) atomicOr(a.status, MOE_DEV_INDEX_OOB);
  const int vis = min(max(L - (c1 - c0) + (t - c0) + 1, 0), L);
  float q[C], o[C], m = -INFINITY, l = 0.0f;
  for (int i = 0; i < C; ++i) {
    q[i] = __bfloat162float(a.q[(int64_t)t * a.q_ts + (int64_t)h * a.q_hs + lane * C + i]);
    o[i] = 0.0f;
  }
  for (int p = 0; p < vis; ++p) {
    const int page = __ldg(a.table + (size_t)b * a.width + p / P);
    if (page < 0 || page >= a.c.n_pages) {
      if (a.status && lane == 0) atomicOr(a.status, MOE_DEV_INDEX_OOB);
      continue;
    }
    const size_t ph = (size_t)page * a.c.n_kv_heads + hk;
    const size_t at = (ph * P + p % P) * D + lane * C;
    const uint8_t *k = static_cast<const uint8_t*>(a.c.k_codes) + at, *v = static_cast<const uint8_t*>(a.c.v_codes) + at;
    float s = 0.0f;
    for (int i = 0; i < C; ++i) s += q[i] * e4m3_to_f32_hw(k[i]);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s = s * exp2i(int(a.c.k_scales[ph]) - 127) * (a.scale * kLog2ef);
    const float mn = fmaxf(m, s), f = exp2f(m - mn), e = exp2f(s - mn);
    const float vs = exp2i(int(a.c.v_scales[ph]) - 127);
    l = l * f + e;
    for (int i = 0; i < C; ++i) o[i] = o[i] * f + e * (e4m3_to_f32_hw(v[i]) * vs);
    m = mn;
  }
  const int64_t r = (int64_t)t * a.n_heads + h;
  for (int i = 0; i < C; ++i) a.out[r * D + lane * C + i] = __float2bfloat16(l == 0.0f ? 0.0f : o[i] / l);
  if (a.lse && lane == 0) a.lse[r] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2f;
}

}  // namespace

size_t attn_chunk_ws_bytes(const moe_kv_cache&, int, int, int, const DeviceInfo&) { return 256; }

int launch_attn_chunk(const ChunkArgs& a, const DeviceInfo&, cudaStream_t s) {
  const dim3 grid((a.total_q + 3) / 4, a.n_heads);
  if (a.c.head_dim == 128) chunk_simple_kernel<128><<<grid, 128, 0, s>>>(a);
  else chunk_simple_kernel<64><<<grid, 128, 0, s>>>(a);
  return launch_status();
}

}  // namespace moe
