// The 8-bit key/value cache: append and eviction.
//
// append: a page and head get the scale s = smallest 2^e with max |x| <= 448
// 2^e over the page's values, codes E4M3(x / s). One CTA per (touched page,
// head, K or V) holds the page's new values in registers between the maximum
// and the rounding, so each value is read once; a part-filled page whose scale
// grows has its older codes rounded once more by the same CTA. Bound by HBM:
// 2 bytes in and 1 out per value.
//
// evict: see the two kernels below.
#include "attn.h"
#include "fp8kv.cuh"

namespace moe {
namespace {

constexpr int kAppThreads = 128;

// Blocks of positions (page-sized, aligned) that a sequence's new tokens touch.
struct Block {
  int b;         // sequence, -1 for none
  int blk;       // page-table column
  int s0, s1;    // slots of new tokens
  int t0;        // row of the first of them
};

// Whole warp: which block is number x, counting over the sequences in order.
__device__ Block find_block(const AppendArgs& a, int x, bool* bad) {
  const int lane = threadIdx.x & 31, P = a.c.page_size;
  Block r{-1, 0, 0, 0, 0};
  int before = 0;
  for (int b0 = 0; b0 < a.n_seq; b0 += 32) {
    const int b = b0 + lane;
    int c0 = 0, c1 = 0, start = 0, n = 0;
    if (b < a.n_seq) {
      packed_range(a.cu, b, a.total, &c0, &c1, bad);
      start = __ldg(a.start + b);
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
    const int lo = before + incl - n;
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, x >= lo && x < lo + n);
    if (hit) {
      const int src = __ffs(hit) - 1;
      if (lane == src) {
        const int blk = start / P + (x - lo);
        const int64_t p0 = (int64_t)blk * P;
        const int64_t end = (int64_t)start + (c1 - c0);
        r.s0 = start > p0 ? int(start - p0) : 0;
        r.s1 = end < p0 + P ? int(end - p0) : P;
        r.t0 = c0 + int(p0 + r.s0 - start);
        r.blk = blk;
        r.b = b;
      }
      r.b = __shfl_sync(0xFFFFFFFFu, r.b, src);
      r.blk = __shfl_sync(0xFFFFFFFFu, r.blk, src);
      r.s0 = __shfl_sync(0xFFFFFFFFu, r.s0, src);
      r.s1 = __shfl_sync(0xFFFFFFFFu, r.s1, src);
      r.t0 = __shfl_sync(0xFFFFFFFFu, r.t0, src);
      return r;
    }
    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  return r;
}

// NV = 16-byte input vectors per thread: page_size * head_dim / 8 / kAppThreads.
template <int NV>
__global__ void __launch_bounds__(kAppThreads) append_kernel(const AppendArgs a) {
  __shared__ Block sblk;
  __shared__ int smax[kAppThreads / 32], sbad[kAppThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) {
    bool bad = false;
    const Block f = find_block(a, int(blockIdx.x), &bad);
    bad = __any_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      sblk = f;
      if (bad && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    }
  }
  __syncthreads();
  const Block f = sblk;
  if (f.b < 0) return;
  const int P = a.c.page_size, D = a.c.head_dim, H = a.c.n_kv_heads, h = blockIdx.y;
  const int page = f.blk < a.width ? __ldg(a.table + (size_t)f.b * a.width + f.blk) : -1;
  if (page < 0 || page >= a.c.n_pages) {
    if (tid == 0 && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    return;
  }
  const bool is_v = blockIdx.z != 0;
  const __nv_bfloat16* src = (is_v ? a.v : a.k) + h * (is_v ? a.v_hs : a.k_hs);
  const int64_t ts = is_v ? a.v_ts : a.k_ts;
  uint8_t* codes = static_cast<uint8_t*>(is_v ? a.c.v_codes : a.c.k_codes) + ((size_t)page * H + h) * P * D;
  uint8_t* scale = (is_v ? a.c.v_scales : a.c.k_scales) + (size_t)page * H + h;
  const int cpr = D / 8, n = (f.s1 - f.s0) * cpr;   // vectors per row; of the new rows

  uint4 x[NV];
  int top = 0, nonfinite = 0;   // largest finite magnitude, as bf16 bits
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * kAppThreads + tid;
    x[i] = make_uint4(0, 0, 0, 0);
    if (v < n) x[i] = *reinterpret_cast<const uint4*>(src + (f.t0 + v / cpr) * ts + (v % cpr) * 8);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int lo = w[j] & 0x7FFF, hi = (w[j] >> 16) & 0x7FFF;
      if (lo < 0x7F80) top = max(top, lo); else nonfinite = 1;
      if (hi < 0x7F80) top = max(top, hi); else nonfinite = 1;
    }
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  nonfinite = __any_sync(0xFFFFFFFFu, nonfinite);
  if (lane == 0) {
    smax[warp] = top;
    sbad[warp] = nonfinite;
  }
  const int had = f.s0 > 0 ? int(*scale) : 0;
  __syncthreads();   // also: everyone has read the old scale
#pragma unroll
  for (int i = 0; i < kAppThreads / 32; ++i) {
    top = max(top, smax[i]);
    nonfinite |= sbad[i];
  }
  const int byte = max(kv_scale_byte(__uint_as_float(uint32_t(top) << 16)), had);
  if (tid == 0) {
    *scale = uint8_t(byte);
    if (nonfinite && a.status) atomicOr(a.status, MOE_DEV_NONFINITE_INPUT);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * kAppThreads + tid;
    if (v >= n) break;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t q[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // inf takes the code of NaN: there is none for it
      const float lo = (w[j] & 0x7F80u) == 0x7F80u ? __int_as_float(0x7FC00000) : scale2(bf16_lo(w[j]), 127 - byte);
      const float hi = (w[j] & 0x7F800000u) == 0x7F800000u ? __int_as_float(0x7FC00000) : scale2(bf16_hi(w[j]), 127 - byte);
      q[j >> 1] |= uint32_t(f32x2_to_e4m3x2(lo, hi)) << (16 * (j & 1));
    }
    *reinterpret_cast<uint2*>(codes + (size_t)(f.s0 + v / cpr) * D + (v % cpr) * 8) = make_uint2(q[0], q[1]);
  }
  if (byte > had && f.s0 > 0) {   // older codes, in units of the new scale
    for (int v = tid; v < f.s0 * D / 16; v += kAppThreads) {
      uint4* p = reinterpret_cast<uint4*>(codes) + v;
      uint4 c = *p;
      c.x = kv_rescale4(c.x, had - byte);
      c.y = kv_rescale4(c.y, had - byte);
      c.z = kv_rescale4(c.z, had - byte);
      c.w = kv_rescale4(c.w, had - byte);
      *p = c;
    }
  }
}

// ---- eviction ----------------------------------------------------------------

constexpr int kSelThreads = 1024;
constexpr int kSelTile = 4 * kSelThreads;

// Order-preserving key: larger weight, larger key; -0 as +0, NaN as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) u = 0xFF800000u;
  if (u == 0x80000000u) u = 0;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Sequence length, cut to what the tables hold.
__device__ __forceinline__ int cut_length(const int32_t* lengths, int b, int width, int page, int64_t stride, bool* bad) {
  const int x = __ldg(lengths + b);
  const int64_t cap = min((int64_t)width * page, stride);
  const int l = x < 0 ? 0 : (x > cap ? int(cap) : x);
  if (l != x) *bad = true;
  return l;
}

// Which positions of (sequence blockIdx.y, head blockIdx.x) stay: the threshold
// weight by radix selection, 8 bits a pass, then one pass in order that takes
// what is above it, the first of what equals it, and the recent ones.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ unsigned hist[256];
  __shared__ unsigned s_bin, s_left;
  __shared__ unsigned long long s_warp[kSelThreads / 32];
  __shared__ unsigned long long s_base;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y, H = a.c.n_kv_heads;
  bool bad = false;
  const int L = cut_length(a.lengths, b, a.width, a.c.page_size, a.w_stride, &bad);
  const float* w = a.weights + ((size_t)b * H + h) * a.w_stride;
  int32_t* kept = a.kept + ((size_t)b * H + h) * a.keep;
  float* kw = a.kept_w ? a.kept_w + ((size_t)b * H + h) * a.keep : nullptr;
  const int m = min(L, a.keep);
  if (h == 0 && tid == 0) {
    a.new_lengths[b] = m;
    if (bad && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
  }
  for (int i = m + tid; i < a.keep; i += kSelThreads) {
    kept[i] = -1;
    if (kw) kw[i] = 0.0f;
  }
  if (L <= a.keep) {
    for (int i = tid; i < m; i += kSelThreads) {
      kept[i] = i;
      if (kw) kw[i] = w[i];
    }
    return;
  }
  const int n = L - a.recent;            // positions that compete
  unsigned left = a.keep - a.recent;     // for so many places (fewer than n)
  uint32_t thr = 0;
  if (left > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t k = weight_key(w[i]);
        if (shift == 24 || (k >> (shift + 8)) == (thr >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (warp == 0) {
        // lane l: bins 255 - 8 l down to 248 - 8 l
        unsigned c[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += (c[j] = hist[255 - 8 * lane - j]);
        unsigned incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (lane >= o) incl += v;
        }
        unsigned above = incl - sum;   // in the bins above this lane's
        if (above < left && incl >= left) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (above < left && above + c[j] >= left) {
              s_bin = 255 - 8 * lane - j;
              s_left = left - above;
              above = 0xFFFFFFFFu;   // found
            } else if (above != 0xFFFFFFFFu) {
              above += c[j];
            }
          }
        }
      }
      __syncthreads();
      thr |= s_bin << shift;
      left = s_left;
    }
  }
  // In order: (positions taken so far, ties seen so far) in one 64-bit sum.
  const bool any = a.keep > a.recent;
  if (tid == 0) s_base = 0;
  __syncthreads();
  for (int i0 = 0; i0 < n && any; i0 += kSelTile) {
    uint32_t k[4];
    float x[4];
    unsigned gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 4 * tid + j;
      x[j] = i < n ? w[i] : 0.0f;
      k[j] = weight_key(x[j]);
      gt += i < n && k[j] > thr;
      eq += i < n && k[j] == thr;
    }
    unsigned long long mine = (unsigned long long)gt << 32 | eq, incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    unsigned long long before = s_base + incl - mine;
    for (int j = 0; j < warp; ++j) before += s_warp[j];
    unsigned g = unsigned(before >> 32), e = unsigned(before);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 4 * tid + j;
      if (i >= n) break;
      const bool tie = k[j] == thr;
      if (k[j] > thr || (tie && e < left)) {
        const unsigned at = g + min(e, left);
        kept[at] = i;
        if (kw) kw[at] = x[j];
      }
      g += k[j] > thr;
      e += tie;
    }
    __syncthreads();
    if (tid == kSelThreads - 1) s_base = before + mine;
    __syncthreads();
  }
  for (int i = tid; i < a.recent; i += kSelThreads) {
    kept[a.keep - a.recent + i] = n + i;
    if (kw) kw[a.keep - a.recent + i] = w[n + i];
  }
}

constexpr int kGatThreads = 256;

// One destination page of one head: threads 0..127 its keys, 128..255 its
// values. The codes stay in registers between the maximum and the rounding.
// NV = 16-code vectors per thread: page_size * head_dim / 16 / 128.
template <int NV>
__global__ void __launch_bounds__(kGatThreads) evict_gather_kernel(const EvictArgs a) {
  __shared__ int s_page[128];        // source page of each slot, -1: none
  __shared__ uint8_t s_slot[128], s_scale[2][128];
  __shared__ float s_max[kGatThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blk = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int P = a.c.page_size, D = a.c.head_dim, H = a.c.n_kv_heads;
  bool bad = false;
  const int m = min(cut_length(a.lengths, b, a.width, P, a.w_stride, &bad), a.keep);
  if (blk * P >= m) return;
  const int page = __ldg(a.dst + (size_t)b * a.dst_width + blk);
  bool oob = page < 0 || page >= a.c.n_pages;
  if (oob) {
    if (tid == 0 && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    return;
  }
  const int slots = min(P, m - blk * P);
  if (tid < slots) {
    const int i = a.kept[((size_t)b * H + h) * a.keep + blk * P + tid];
    const int sp = __ldg(a.table + (size_t)b * a.width + i / P);
    uint8_t ks = 0, vs = 0;
    const bool in = sp >= 0 && sp < a.c.n_pages;
    if (!in) {
      if (a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    } else {
      ks = a.c.k_scales[(size_t)sp * H + h];
      vs = a.c.v_scales[(size_t)sp * H + h];
    }
    s_page[tid] = in ? sp : -1;
    s_slot[tid] = uint8_t(i % P);
    s_scale[0][tid] = ks;
    s_scale[1][tid] = vs;
  }
  __syncthreads();
  const int part = tid >> 7, pt = tid & 127;
  uint8_t* codes = static_cast<uint8_t*>(part ? a.c.v_codes : a.c.k_codes);
  const int cpr = D / 16, n = slots * cpr;
  uint4 x[NV];
  int sc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * 128 + pt;
    x[i] = make_uint4(0, 0, 0, 0);
    sc[i] = 0;
    if (v < n) {
      const int sp = s_page[v / cpr];
      if (sp >= 0) {
        const size_t row = ((size_t)sp * H + h) * P + s_slot[v / cpr];
        x[i] = *reinterpret_cast<const uint4*>(codes + row * D + (v % cpr) * 16);
        sc[i] = s_scale[part][v / cpr];
      }
    }
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t mag = 0;   // E4M3 magnitudes order as their codes do
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t c = (w[j >> 2] >> (8 * (j & 3))) & 0x7Fu;
      if (c != 0x7Fu) mag = max(mag, c);
    }
    if (mag) top = fmaxf(top, scale2(e4m3_to_f32(mag), sc[i] - 127));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) top = fmaxf(top, s_max[part * 4 + i]);
  const int byte = kv_scale_byte(top);
  if (pt == 0) (part ? a.c.v_scales : a.c.k_scales)[(size_t)page * H + h] = uint8_t(byte);
  uint8_t* to = codes + ((size_t)page * H + h) * P * D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * 128 + pt;
    if (v >= n) break;
    uint4 c = x[i];
    if (sc[i] != byte) {
      c.x = kv_rescale4(c.x, sc[i] - byte);
      c.y = kv_rescale4(c.y, sc[i] - byte);
      c.z = kv_rescale4(c.z, sc[i] - byte);
      c.w = kv_rescale4(c.w, sc[i] - byte);
    }
    *reinterpret_cast<uint4*>(to + (size_t)v * 16) = c;
  }
}

}  // namespace

int launch_kv_append(const AppendArgs& a, cudaStream_t s) {
  const int P = a.c.page_size;
  // every sequence touches at most len / P + 2 pages, and no more than its tokens
  const int64_t most = (int64_t)a.total / P + 2 * (int64_t)a.n_seq;
  const int nb = int(most < a.total ? most : a.total) + 1;   // the last one looks at every sequence
  const dim3 grid(nb, a.c.n_kv_heads, 2);
  switch (P * a.c.head_dim / 8 / kAppThreads) {
    case 1: append_kernel<1><<<grid, kAppThreads, 0, s>>>(a); break;
    case 2: append_kernel<2><<<grid, kAppThreads, 0, s>>>(a); break;
    case 4: append_kernel<4><<<grid, kAppThreads, 0, s>>>(a); break;
    case 8: append_kernel<8><<<grid, kAppThreads, 0, s>>>(a); break;
    default: append_kernel<16><<<grid, kAppThreads, 0, s>>>(a); break;
  }
  return launch_status();
}

int launch_kv_evict(const EvictArgs& a, const DeviceInfo& di, cudaStream_t s) {
  (void)di;
  const int P = a.c.page_size;
  evict_select_kernel<<<dim3(a.c.n_kv_heads, a.n_seq), kSelThreads, 0, s>>>(a);
  int st = launch_status();
  if (st != MOE_OK) return st;
  const int64_t most = (int64_t)a.width * P < a.keep ? (int64_t)a.width * P : a.keep;
  if (most == 0) return MOE_OK;
  const dim3 grid(unsigned((most + P - 1) / P), a.c.n_kv_heads, a.n_seq);
  switch (P * a.c.head_dim / 16 / 128) {
    case 0:   // 16 x 64: half of the threads hold a vector
    case 1: evict_gather_kernel<1><<<grid, kGatThreads, 0, s>>>(a); break;
    case 2: evict_gather_kernel<2><<<grid, kGatThreads, 0, s>>>(a); break;
    case 4: evict_gather_kernel<4><<<grid, kGatThreads, 0, s>>>(a); break;
    default: evict_gather_kernel<8><<<grid, kGatThreads, 0, s>>>(a); break;
  }
  return launch_status();
}

}  // namespace moe
