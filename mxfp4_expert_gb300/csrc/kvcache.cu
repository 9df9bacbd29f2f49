// The 8-bit key/value cache: append and eviction.
//
// append: a page and head get the scale s = smallest 2^e with max |x| <= 448
// 2^e over the page's values, codes E4M3(x / s). One CTA per (touched page,
// head, K or V) holds the page's new values in registers between the maximum
// and the rounding, so each value is read once; a part-filled page whose scale
// grows has its older codes rounded once more by the same CTA. Bound by HBM:
// 2 bytes in and 1 out per value. 12,345 tokens of 8 heads of 128 for 5
// sequences: 19.7 us, 3.8 TB/s: a CTA's chain (block, page, values, maximum,
// codes) overlaps with the other CTAs' on its SM, of which 2.4 rounds run. 64
// tokens for 64 sequences, 4 heads: 6.3 us, the launch and that chain.
//
// evict: see the two kernels below.
#include <algorithm>

#include "attn.h"
#include "fp8kv.cuh"
#include "kvblock.cuh"

namespace moe {
namespace {

constexpr int kAppThreads = 128;

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
  // the page, and meanwhile the values; then the page's scale, and meanwhile their maximum
  const int page = f.blk < a.width ? __ldg(a.table + (size_t)f.b * a.width + f.blk) : -1;
  const bool is_v = blockIdx.z != 0;
  const __nv_bfloat16* src = (is_v ? a.v : a.k) + h * (is_v ? a.v_hs : a.k_hs);
  const int64_t ts = is_v ? a.v_ts : a.k_ts;
  const int cpr = D / 8, n = (f.s1 - f.s0) * cpr;   // vectors per row; of the new rows
  const int row = tid / cpr, col = (tid % cpr) * 8, rows = kAppThreads / cpr;   // a thread's first vector; rows to its next

  uint4 x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    x[i] = i * kAppThreads + tid < n ? *reinterpret_cast<const uint4*>(src + (f.t0 + row + i * rows) * ts + col)
                                     : make_uint4(0, 0, 0, 0);
  if (page < 0 || page >= a.c.n_pages) {
    if (tid == 0 && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    return;
  }
  uint8_t* codes = static_cast<uint8_t*>(is_v ? a.c.v_codes : a.c.k_codes) + ((size_t)page * H + h) * P * D;
  uint8_t* scale = (is_v ? a.c.v_scales : a.c.k_scales) + (size_t)page * H + h;
  const int had = f.s0 > 0 ? int(*scale) : 0;
  uint32_t top2 = 0;   // largest magnitudes, as bf16 bits, of the even and the odd values
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) top2 = __vmaxu2(top2, w[j] & 0x7FFF7FFFu);
  }
  int top = max(top2 & 0xFFFFu, top2 >> 16);
  bool nonfinite = __any_sync(0xFFFFFFFFu, top >= 0x7F80);
  if (nonfinite) {     // the largest finite one then
    top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int lo = w[j] & 0x7FFF, hi = (w[j] >> 16) & 0x7FFF;
        if (lo < 0x7F80) top = max(top, lo);
        if (hi < 0x7F80) top = max(top, hi);
      }
    }
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) {
    smax[warp] = top;
    sbad[warp] = nonfinite;
  }
  __syncthreads();   // also: everyone has read the old scale
#pragma unroll
  for (int i = 0; i < kAppThreads / 32; ++i) {
    top = max(top, smax[i]);
    nonfinite |= sbad[i] != 0;
  }
  const int byte = max(kv_scale_byte(__uint_as_float(uint32_t(top) << 16)), had);
  if (tid == 0) {
    *scale = uint8_t(byte);
    if (nonfinite && a.status) atomicOr(a.status, MOE_DEV_NONFINITE_INPUT);
  }
  // 2^(127 - byte); 2^-127 and 2^-128 are subnormal (new values need 247 at most, but the page may hold more)
  const float f1 = byte <= 253 ? pow2(127 - byte) : __uint_as_float(0x00800000u >> (byte - 253));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * kAppThreads + tid >= n) break;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t q[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo = bf16_lo(w[j]) * f1, hi = bf16_hi(w[j]) * f1;
      if (nonfinite) {   // inf takes the code of NaN: there is none for it
        if ((w[j] & 0x7F80u) == 0x7F80u) lo = __int_as_float(0x7FC00000);
        if ((w[j] & 0x7F800000u) == 0x7F800000u) hi = __int_as_float(0x7FC00000);
      }
      q[j >> 1] |= uint32_t(f32x2_to_e4m3x2(lo, hi)) << (16 * (j & 1));
    }
    *reinterpret_cast<uint2*>(codes + (f.s0 + row + i * rows) * D + col) = make_uint2(q[0], q[1]);
  }
  if (byte > had && f.s0 > 0) {   // older codes, in units of the new scale
    const float fo = kv_factor(had, byte);
    for (int v = tid; v < f.s0 * D / 16; v += kAppThreads) {
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

// ---- eviction ----------------------------------------------------------------

constexpr int kSelThreads = 1024;
constexpr int kSelTile = 4 * kSelThreads;
constexpr int kSelBits = 11, kSelBins = 1 << kSelBits, kSelPasses = 3;
constexpr int kSelCluster = 4;          // CTAs per (sequence, head), at most
constexpr int kSelEach = 8192;          // positions that a CTA of several has at least
constexpr int kSelRegs = 16;            // keys that a thread keeps

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

// Which positions of (sequence, head) stay. A cluster of CTAs shares one pair,
// each a run of positions. The threshold weight comes from a radix selection, 11
// bits of the key a pass: every CTA counts its positions' digits in its own
// shared memory, then reads the others' counts through the cluster and finds the
// digit for itself, so a pass takes one cluster barrier. One more pass, in
// order, takes what is above the threshold, the first of what equals it, and
// the recent ones. Bound by latency: a few dependent passes over the keys, the
// first kSelRegs x 1024 of a CTA in registers, each with a shared-memory atomic a
// position, two barriers and a scan. 16 x 4 pairs of 32,768 positions, two CTAs
// a pair: 24 us (36 with one CTA and four passes of 8 bits); a read of the
// weights at the copy rate takes 1.3.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int csize) {
  __shared__ unsigned hist[kSelPasses][kSelBins];
  __shared__ unsigned s_bin, s_left;
  __shared__ unsigned s_sum[kSelThreads / 32];
  __shared__ unsigned s_cnt[2];                          // this CTA's positions above and at the threshold
  __shared__ unsigned s_gt[kSelThreads / 32], s_eq[kSelThreads / 32];
  __shared__ unsigned s_base[2];                         // positions above and at the threshold so far
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % csize, h = blockIdx.x / csize, b = blockIdx.y, H = a.c.n_kv_heads;
  bool bad = false;
  const int L = cut_length(a.lengths, b, a.width, a.c.page_size, a.w_stride, &bad);
  const float* w = a.weights + ((size_t)b * H + h) * a.w_stride;
  int32_t* kept = a.kept + ((size_t)b * H + h) * a.keep;
  float* kw = a.kept_w ? a.kept_w + ((size_t)b * H + h) * a.keep : nullptr;
  const int m = min(L, a.keep);
  const int me = rank * kSelThreads + tid, all = csize * kSelThreads;
  if (h == 0 && me == 0) {
    a.new_lengths[b] = m;
    if (bad && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
  }
  for (int i = m + me; i < a.keep; i += all) {
    kept[i] = -1;
    if (kw) kw[i] = 0.0f;
  }
  if (L <= a.keep) {
    for (int i = me; i < m; i += all) {
      kept[i] = i;
      if (kw) kw[i] = w[i];
    }
    return;
  }
  const int n = L - a.recent;            // positions that compete
  const int room = a.keep - a.recent;    // for so many places (fewer than n)
  for (int i = me; i < a.recent; i += all) {
    kept[room + i] = n + i;
    if (kw) kw[room + i] = w[n + i];
  }
  if (room == 0) return;                 // the same for the whole cluster
  // this CTA's run of positions
  const int each = ((n + csize - 1) / csize + 3) & ~3;
  const int i0 = min(n, rank * each), i1 = min(n, i0 + each);
  for (int i = tid; i < kSelPasses * kSelBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  __syncthreads();

  // the first kSelRegs x 1024 of them stay in registers, as keys
  uint32_t key[kSelRegs];
#pragma unroll
  for (int u = 0; u < kSelRegs; ++u) {
    const int i = i0 + tid + u * kSelThreads;
    key[u] = i < i1 ? weight_key(w[i]) : 0u;
  }
  const int i_more = i0 + tid + kSelRegs * kSelThreads;

  uint32_t thr = 0;
  unsigned left = room;
  // one address per lane and warp of any CTA's hist / s_cnt
  auto remote = [&](const void* p, int r) {
    uint32_t x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(x) : "r"(smem_addr(p)), "r"(r));
    return x;
  };
  auto ld_remote = [&](uint32_t x) {
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(x));
    return v;
  };
  // a value per warp: the sum over the warps before this one
  auto warps_before = [&](const unsigned* p) {
    return __reduce_add_sync(0xFFFFFFFFu, lane < warp ? p[lane] : 0u);
  };
  auto cluster_sync = [&]() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  // digits, from the top: bits [21, 32), [10, 21), [0, 10)
#pragma unroll
  for (int pass = 0; pass < kSelPasses; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    const uint32_t mask = (1u << bits) - 1;
#pragma unroll
    for (int u = 0; u < kSelRegs; ++u) {
      const uint32_t k = key[u];
      if (i0 + tid + u * kSelThreads < i1 && (pass == 0 || (k >> (shift + bits)) == (thr >> (shift + bits))))
        atomicAdd(&hist[pass][(k >> shift) & mask], 1u);
    }
#pragma unroll 4
    for (int i = i_more; i < i1; i += kSelThreads) {
      const uint32_t k = weight_key(w[i]);
      if (pass == 0 || (k >> (shift + bits)) == (thr >> (shift + bits))) atomicAdd(&hist[pass][(k >> shift) & mask], 1u);
    }
    if (csize > 1) cluster_sync(); else __syncthreads();
    // thread t: bins kSelBins - 1 - 2t and the one below
    const int hi = kSelBins - 1 - 2 * tid;
    unsigned c0 = 0, c1 = 0;
    if (csize == 1) {
      c0 = hist[pass][hi];
      c1 = hist[pass][hi - 1];
    } else {
      unsigned v0[kSelCluster], v1[kSelCluster];   // all on their way at once
#pragma unroll
      for (int r = 0; r < kSelCluster; ++r) {
        v0[r] = r < csize ? ld_remote(remote(&hist[pass][hi], r)) : 0;
        v1[r] = r < csize ? ld_remote(remote(&hist[pass][hi - 1], r)) : 0;
      }
#pragma unroll
      for (int r = 0; r < kSelCluster; ++r) c0 += v0[r], c1 += v1[r];
    }
    unsigned incl = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    const unsigned above = incl - c0 - c1 + warps_before(s_sum);   // in the bins above this thread's
    if (above < left && above + c0 + c1 >= left) {
      const bool first = above + c0 >= left;
      s_bin = first ? hi : hi - 1;
      s_left = left - above - (first ? 0 : c0);
    }
    __syncthreads();
    thr |= s_bin << shift;
    left = s_left;
  }

  // positions above and at the threshold in the CTAs before this one
  if (tid < 2) s_cnt[tid] = s_base[tid] = 0;
  __syncthreads();
  if (csize > 1) {
    unsigned gt = 0, eq = 0;
#pragma unroll
    for (int u = 0; u < kSelRegs; ++u) {
      const bool in = i0 + tid + u * kSelThreads < i1;
      gt += in && key[u] > thr;
      eq += in && key[u] == thr;
    }
#pragma unroll 4
    for (int i = i_more; i < i1; i += kSelThreads) {
      const uint32_t k = weight_key(w[i]);
      gt += k > thr;
      eq += k == thr;
    }
    gt = __reduce_add_sync(0xFFFFFFFFu, gt);
    eq = __reduce_add_sync(0xFFFFFFFFu, eq);
    if (lane == 0) {
      atomicAdd(&s_cnt[0], gt);
      atomicAdd(&s_cnt[1], eq);
    }
    cluster_sync();
    if (warp == 0) {
      const unsigned g = lane < rank ? ld_remote(remote(&s_cnt[0], lane)) : 0;
      const unsigned e = lane < rank ? ld_remote(remote(&s_cnt[1], lane)) : 0;
      const unsigned gs = __reduce_add_sync(0xFFFFFFFFu, g), es = __reduce_add_sync(0xFFFFFFFFu, e);
      if (lane == 0) {
        s_base[0] = gs;
        s_base[1] = es;
      }
    }
    __syncthreads();
  }
  for (int t0 = i0; t0 < i1; t0 += kSelTile) {
    uint32_t k[4];
    float x[4];
    unsigned gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = t0 + 4 * tid + j;
      x[j] = i < i1 ? w[i] : 0.0f;
      k[j] = weight_key(x[j]);
      gt += i < i1 && k[j] > thr;
      eq += i < i1 && k[j] == thr;
    }
    // (above, at) before this thread: at most 4 of each per thread, so both counts of a warp fit one word
    unsigned incl = gt << 16 | eq;
    const unsigned mine = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) {
      s_gt[warp] = incl >> 16;
      s_eq[warp] = incl & 0xFFFFu;
    }
    __syncthreads();
    unsigned g = s_base[0] + warps_before(s_gt) + ((incl - mine) >> 16);
    unsigned e = s_base[1] + warps_before(s_eq) + ((incl - mine) & 0xFFFFu);
    const unsigned g1 = g + gt, e1 = e + eq;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = t0 + 4 * tid + j;
      if (i >= i1) break;
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
    if (tid == kSelThreads - 1) {
      s_base[0] = g1;
      s_base[1] = e1;
    }
    __syncthreads();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (csize > 1) cluster_sync();     // no CTA leaves while another reads its counts
}

constexpr int kGatThreads = 256;

// One destination page of one head: threads 0..127 its keys, 128..255 its
// values. The codes stay in registers between the maximum and the rounding.
// NV = 16-code vectors per thread: page_size * head_dim / 16 / 128. Bound by
// HBM (a byte in and out per code); what costs is that a kept row is 128 bytes at
// a random place: 4.2 TB/s in all for such reads, 7.1 for long ones. Before it
// lies a chain of loads (kept position, its page, scale and codes), so many small
// CTAs per SM (with 4 instead of 8, 61.5 us instead of 56.2 for the call). 16 x
// 32,768 positions of 4 heads to 4,096 each: 32 us, 134 MB.
template <int NV>
__global__ void __launch_bounds__(kGatThreads, NV <= 4 ? 8 : 4) evict_gather_kernel(const EvictArgs a) {
  __shared__ int s_page[128];        // source page of each slot, -1: none
  __shared__ uint8_t s_slot[128], s_scale[2][128];
  __shared__ int s_top[kGatThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blk = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int P = a.c.page_size, D = a.c.head_dim, H = a.c.n_kv_heads;
  bool bad = false;
  const int page = __ldg(a.dst + (size_t)b * a.dst_width + blk);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the kept positions
  const int i = tid < P && blk * P + tid < a.keep ? a.kept[((size_t)b * H + h) * a.keep + blk * P + tid] : -1;
  const int m = min(cut_length(a.lengths, b, a.width, P, a.w_stride, &bad), a.keep);
  if (blk * P >= m) return;
  if (page < 0 || page >= a.c.n_pages) {
    if (tid == 0 && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    return;
  }
  const int slots = min(P, m - blk * P);
  if (tid < slots) {
    const int sp = __ldg(a.table + (size_t)b * a.width + i / P);
    const bool in = sp >= 0 && sp < a.c.n_pages;
    if (!in && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    s_page[tid] = in ? sp : -1;
    s_slot[tid] = uint8_t(i % P);
    s_scale[0][tid] = in ? a.c.k_scales[(size_t)sp * H + h] : 0;
    s_scale[1][tid] = in ? a.c.v_scales[(size_t)sp * H + h] : 0;
  }
  __syncthreads();
  const int part = tid >> 7, pt = tid & 127;
  uint8_t* codes = static_cast<uint8_t*>(part ? a.c.v_codes : a.c.k_codes);
  const int cpr = D / 16, row = pt / cpr, col = (pt % cpr) * 16, rows = 128 / cpr;   // first vector's slot; slots to the next
  uint4 x[NV];
  int sc[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int s = row + v * rows;
    x[v] = make_uint4(0, 0, 0, 0);
    sc[v] = 0;
    if (s < slots) {
      const int sp = s_page[s];
      if (sp >= 0) {
        x[v] = *reinterpret_cast<const uint4*>(codes + (((size_t)sp * H + h) * P + s_slot[s]) * D + col);
        sc[v] = s_scale[part][s];
      }
    }
  }
  int byte = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    // E4M3 magnitudes order as their codes do; NaN's is the largest
    const uint32_t w[4] = {x[v].x, x[v].y, x[v].z, x[v].w};
    uint32_t mag = 0;
    const bool nan = any_nan4(w[0]) || any_nan4(w[1]) || any_nan4(w[2]) || any_nan4(w[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) mag = __vmaxu2(mag, __vmaxu2(w[j] & 0x007F007Fu, (w[j] >> 8) & 0x007F007Fu));
    mag = max(mag & 0xFFFFu, mag >> 16);
    if (nan) {
      mag = 0;
#pragma unroll 1
      for (int j = 0; j < 16; ++j) {
        const uint32_t c = (w[j >> 2] >> (8 * (j & 3))) & 0x7Fu;
        if (c != 0x7Fu) mag = max(mag, c);
      }
    }
    // the byte that the largest value needs is the largest of the bytes that the vectors need
    byte = max(byte, kv_code_byte(mag, sc[v]));
  }
  byte = __reduce_max_sync(0xFFFFFFFFu, byte);
  if (lane == 0) s_top[warp] = byte;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) byte = max(byte, s_top[part * 4 + k]);
  if (pt == 0) (part ? a.c.v_scales : a.c.k_scales)[(size_t)page * H + h] = uint8_t(byte);
  uint8_t* to = codes + ((size_t)page * H + h) * P * D;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int s = row + v * rows;
    if (s >= slots) break;
    uint4 c = x[v];
    if (sc[v] != byte) {
      const float f = kv_factor(min(sc[v] - byte, 127), 0);   // a larger one than 2^127 meets zeros only
      c.x = kv_rescale4(c.x, f);
      c.y = kv_rescale4(c.y, f);
      c.z = kv_rescale4(c.z, f);
      c.w = kv_rescale4(c.w, f);
    }
    *reinterpret_cast<uint4*>(to + s * D + col) = c;
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
  const int P = a.c.page_size;
  const int64_t cap = std::min((int64_t)a.width * P, a.w_stride);
  // More CTAs per pair while each keeps enough positions and all run at once. The
  // whole call, us with 1, 2, 4 and 8 CTAs a pair: 4 pairs of 4,096 14.5, 18.5,
  // 20.6, 30.8; 16 of 9,000 18.6, 22.6, 24.6, 55.5; 4 of 32,768 29.6, 24.6, 22.7,
  // 30.9; 16 of 32,768 32.9, 28.7, 26.9, 59.5; 64 of 32,768 59.4, 51.5, 67.7, 163;
  // 8 of 100,000 77.3, 53.3, 36.6, 37.1.
  int csize = 1;
  while (csize < kSelCluster && 2 * (int64_t)csize * kSelEach <= cap &&
         2 * (int64_t)csize * a.c.n_kv_heads * a.n_seq <= di.sm_count)
    csize *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.c.n_kv_heads * csize, a.n_seq);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = csize;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, evict_select_kernel, a, csize));
  const int64_t most = std::min((int64_t)a.width * P, (int64_t)a.keep);
  if (most == 0) return MOE_OK;
  const dim3 grid(unsigned((most + P - 1) / P), a.c.n_kv_heads, a.n_seq);
  // starts while the selection ends (programmatic dependent launch): 57.5 -> 55.6 us for 16 x 32768
  cudaLaunchConfig_t gat{};
  gat.gridDim = grid;
  gat.blockDim = dim3(kGatThreads);
  gat.stream = s;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  gat.attrs = &pdl;
  gat.numAttrs = 1;
  switch (P * a.c.head_dim / 16 / 128) {
    case 0:   // 16 x 64: half of the threads hold a vector
    case 1: MOE_CUDA_TRY(cudaLaunchKernelEx(&gat, evict_gather_kernel<1>, a)); break;
    case 2: MOE_CUDA_TRY(cudaLaunchKernelEx(&gat, evict_gather_kernel<2>, a)); break;
    case 4: MOE_CUDA_TRY(cudaLaunchKernelEx(&gat, evict_gather_kernel<4>, a)); break;
    default: MOE_CUDA_TRY(cudaLaunchKernelEx(&gat, evict_gather_kernel<8>, a)); break;
  }
  return launch_status();
}

}  // namespace moe
