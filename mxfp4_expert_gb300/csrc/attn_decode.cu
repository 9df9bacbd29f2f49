// Attention of a few new tokens per sequence over the 8-bit paged cache.
//
// Bound by reading the cache once: 2 head_dim bytes per position and
// key/value head. What this asks of a kernel is many bytes in flight, few
// instructions per byte, and work cut evenly whatever the lengths are.
//
// Work. All (sequence, key/value head) pairs are laid end to end in units of
// kUnit positions; CTA c takes units [c W / N, (c + 1) W / N) of the W. Its
// range is one or more segments, each a run of positions of one pair. A
// segment that is a whole pair writes the output; any other writes its
// unnormalised output, maximum and sum to the workspace, and the last CTA of
// the pair to finish (a counter) joins them in order, so results do not depend
// on who finishes when.
//
// Inside a CTA the warps take groups of 16 positions (a group never leaves its
// page, so it has one scale for keys and one for values). A warp's next groups
// are on their way into shared memory by cp.async, every lane fetching what
// itself will use: no barrier, no bank conflict. Both products run on the f16
// warp MMA (m16n8k16) with positions or channels as its 16 rows and the query
// rows (token, head of the group) as its 8 columns: E4M3 converts to f16
// exactly, two codes an instruction, and up to 8 query rows cost one MMA
// column block instead of a 16-row one.
//   scores   S^T[pos][row] = K q^T: lane (g, c) holds 16-byte chunks of the
//            positions g and g + 8 and takes 4 consecutive codes of a chunk as
//            its k = 2c, 2c+1, 2c+8, 2c+9 of one MMA; q is loaded in the same
//            order, as f16 scaled by a power of two per row
//   softmax  running maximum that is raised only when a score passes it by
//            2^6 (probabilities up to 2^6 are exact enough in f16), sums in
//            fp32 kept per lane until the end
//   output   O^T[d][row] = V^T P^T: lane (g, c) holds a chunk of the positions
//            2c, 2c+1, 2c+8, 2c+9; a byte permute pairs the codes of two
//            positions; movmatrix turns the probabilities from S's layout
//            into the B operand
// The page's key scale multiplies the scores; O is held in units of the
// largest value scale so far, and a group of smaller scale is added with an
// fp32 factor, so no page's values are rounded for the sake of another's.
#include "attn.h"
#include "fp8kv.cuh"

namespace moe {
namespace {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kMaxSeqs = 4096;
constexpr float kRaise = 6.0f;     // log2 by which a score may pass the reference
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Workspace: counters [n_seq * n_kv], then partials, then (with weights) the
// rows' log2-sum-exp and the scores.
struct DecWs {
  size_t parts, lse2, scores, total;
  int n_cta, rows;    // CTAs; query rows padded to the row tiles
};

struct DecPlan {
  int nt, rt;         // column blocks of 8 rows per warp; row tiles
};
inline DecPlan dec_plan(int rows) {
  if (rows <= 8) return {1, 1};
  if (rows <= 16) return {2, 1};
  if (rows <= 32) return {2, 2};
  return {2, 4};
}

struct DecParams {
  DecodeArgs a;
  int G, rows;              // query heads per kv head; query rows n_new * G
  unsigned* counter;        // [n_seq * n_kv]
  float* parts;             // [n_cta][2][rows padded][D + 2]
  float* lse2;              // [n_seq * n_kv][rows padded] (weights)
  float* scores;            // [n_seq * n_kv][cap][rows padded] (weights)
  int64_t cap;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// codes in the low or high half of a word -> f16 pair
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Does one of the word's four codes stand for NaN?
__device__ __forceinline__ bool any_nan4(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// Length of sequence b, cut to what table, weights and workspace hold.
__device__ __forceinline__ int dec_length(const DecodeArgs& a, int b, bool* bad) {
  const int x = __ldg(a.lengths + b);
  int64_t cap = (int64_t)a.width * a.c.page_size;
  if (a.weights && a.w_stride < cap) cap = a.w_stride;
  const int l = x < 0 ? 0 : (x > cap ? int(cap) : x);
  if (l != x) *bad = true;
  return l;
}

// D: head_dim. NT: blocks of 8 query rows per warp. RT: row tiles (warps w, w
// + 1, .. RT work on the same positions). WT: scores are kept for the weights.
template <int D, int NT, int RT, bool WT>
struct DecCfg {
  static constexpr int kStages = 4;
  static constexpr int kGroups = kDecWarps / RT;         // position groups in flight per CTA step
  static constexpr int kUnit = 16 * kGroups;             // positions per unit
  static constexpr int kRows = 8 * NT * RT;              // padded query rows
  static constexpr int kVec = D / 16;                    // 16-byte vectors per lane and group (keys + values)
  static constexpr uint32_t kStageBytes = kVec * 32 * 16;
  static constexpr uint32_t kRing = kDecWarps * kStages * kStageBytes;
  static constexpr uint32_t kMerge = kDecWarps * 8 * NT * (D + 2) * 4;   // reuses the ring
  static constexpr uint32_t kSmem = (kRing > kMerge ? kRing : kMerge) + (kMaxSeqs + 1) * 4 + 64;
};

template <int D, int NT, int RT, bool WT>
__global__ void __launch_bounds__(kDecThreads) decode_attn_kernel(const DecParams p) {
  using C = DecCfg<D, NT, RT, WT>;
  constexpr int KS = D / 16;      // MMA steps over the channels
  constexpr int MT = D / 16;      // 16-channel blocks of the output
  constexpr int KC = D / 64;      // 16-byte key chunks per lane and position
  extern __shared__ __align__(128) uint8_t smem[];
  int* prefix = reinterpret_cast<int*>(smem + (C::kRing > C::kMerge ? C::kRing : C::kMerge));
  __shared__ int s_scan[kDecWarps];
  __shared__ int s_last;
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int H = a.c.n_kv_heads, P = a.c.page_size, B = a.n_seq, T = a.n_new;

  // units of the sequences before each one (per kv head)
  {
    bool bad = false;
    int before = 0;
    for (int b0 = 0; b0 < B; b0 += kDecThreads) {
      const int b = b0 + tid;
      int n = 0;
      if (b < B) {
        const int L = dec_length(a, b, &bad);
        n = L > 0 ? (L + C::kUnit - 1) / C::kUnit : 1;
      }
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) s_scan[warp] = incl;
      __syncthreads();
      int w0 = before, all = 0;
#pragma unroll
      for (int i = 0; i < kDecWarps; ++i) {
        w0 += i < warp ? s_scan[i] : 0;
        all += s_scan[i];
      }
      if (b < B) prefix[b] = w0 + incl - n;
      before += all;
      __syncthreads();
    }
    if (tid == 0) prefix[B] = before;
    if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    __syncthreads();
  }
  const int64_t W = (int64_t)prefix[B] * H, N = min((int64_t)gridDim.x, W);   // no CTA has an empty range
  if (blockIdx.x >= N) return;
  int64_t pos = blockIdx.x * W / N;
  const int64_t end = (blockIdx.x + 1) * W / N;

  const int rt = warp % RT, tg = warp / RT;
  uint8_t* ring = smem + (size_t)warp * C::kStages * C::kStageBytes;
  const uint32_t ring_s = smem_addr(ring) + lane * 16;

  while (pos < end) {
    // sequence of unit pos: the last b with prefix[b] H <= pos
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)prefix[mid] * H <= pos) lo = mid; else hi = mid - 1;
    }
    const int b = lo, nu = prefix[b + 1] - prefix[b];
    const int64_t pair0 = (int64_t)prefix[b] * H;
    const int h = int((pos - pair0) / nu), u0 = int((pos - pair0) % nu);
    const int u1 = int(min((int64_t)nu, u0 + (end - pos)));
    bool ignore = false;
    const int L = dec_length(a, b, &ignore);
    const int first = u0 * C::kUnit, last = min(L, u1 * C::kUnit);
    const int n_my = last > first + tg * 16 ? (last - first - tg * 16 + C::kUnit - 1) / C::kUnit : 0;
    const int32_t* table = a.table + (size_t)b * a.width;
    const size_t head_bytes = (size_t)P * D, page_bytes = head_bytes * H;
    const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k_codes) + h * head_bytes;
    const uint8_t* vbase = static_cast<const uint8_t*>(a.c.v_codes) + h * head_bytes;

    // position of this warp's group i; its page (-1: outside the cache)
    auto gpos = [&](int i) { return first + (i * C::kGroups + tg) * 16; };
    auto page_of = [&](int i) {
      if (i >= n_my) return -1;
      const int pg = __ldg(table + gpos(i) / P);
      return pg >= 0 && pg < a.c.n_pages ? pg : -1;
    };
    auto issue = [&](int i, int pg) {
      if (i < n_my && pg >= 0) {
        const size_t row = (size_t)pg * page_bytes + (size_t)(gpos(i) % P) * D;
        const uint32_t dst = ring_s + (i % C::kStages) * C::kStageBytes;
        const uint8_t* k0 = kbase + row + c * 16;
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          cp_async16(dst + (2 * j) * 512, k0 + (size_t)g * D + 64 * j);
          cp_async16(dst + (2 * j + 1) * 512, k0 + (size_t)(g + 8) * D + 64 * j);
        }
        // head_dim 128: chunk g of the positions 2c, 2c+1, 2c+8, 2c+9; head_dim
        // 64: a position has 4 chunks, lanes g and g ^ 1 fetch two positions' each
        const uint8_t* v0 = vbase + row;
        if (D == 128) {
          cp_async16(dst + (2 * KC) * 512, v0 + (size_t)(2 * c) * D + g * 16);
          cp_async16(dst + (2 * KC + 1) * 512, v0 + (size_t)(2 * c + 1) * D + g * 16);
          cp_async16(dst + (2 * KC + 2) * 512, v0 + (size_t)(2 * c + 8) * D + g * 16);
          cp_async16(dst + (2 * KC + 3) * 512, v0 + (size_t)(2 * c + 9) * D + g * 16);
        } else {
          const int o = g & 1;
          cp_async16(dst + (2 * KC) * 512, v0 + (size_t)(2 * c + o) * D + (g >> 1) * 16);
          cp_async16(dst + (2 * KC + 1) * 512, v0 + (size_t)(2 * c + 8 + o) * D + (g >> 1) * 16);
        }
      }
      cp_async_commit();
    };

    // query rows -> B fragments (f16, scaled by 2^-qe) and the factors that undo it
    uint32_t qf[KS][NT][2];
    float qs[NT][2];         // of rows 2c, 2c+1 of each block: 2^qe scale log2(e)
    int vis[NT][2];          // positions that those rows see
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = (rt * NT + n) * 8 + g;
      float x[KS * 4];
      float top = 0.0f;
      if (r < p.rows) {
        const __nv_bfloat16* q = a.q + ((int64_t)b * T + r / p.G) * a.q_ts + (int64_t)(h * p.G + r % p.G) * a.q_hs;
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          const uint4 v0 = *reinterpret_cast<const uint4*>(q + 64 * j + 16 * c);
          const uint4 v1 = *reinterpret_cast<const uint4*>(q + 64 * j + 16 * c + 8);
          const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[16 * j + 2 * i] = bf16_lo(w[i]);
            x[16 * j + 2 * i + 1] = bf16_hi(w[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < KS * 4; ++i) top = fmaxf(top, fabsf(x[i]));
      } else {
#pragma unroll
        for (int i = 0; i < KS * 4; ++i) x[i] = 0.0f;
      }
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      int e = 0;
      if (top > 0.0f && top < INFINITY) {
        frexpf(top, &e);
        e -= 12;             // the row's largest value in [2^11, 2^12)
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[k][n][0] = f16x2_bits(scale2(x[4 * k], -e), scale2(x[4 * k + 1], -e));
        qf[k][n][1] = f16x2_bits(scale2(x[4 * k + 2], -e), scale2(x[4 * k + 3], -e));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int er = __shfl_sync(0xFFFFFFFFu, e, (2 * c + j) * 4);
        const int rr = (rt * NT + n) * 8 + 2 * c + j;
        qs[n][j] = scale2(a.scale * kLog2e, er);
        vis[n][j] = rr < p.rows ? L - T + rr / p.G + 1 : 0;
      }
    }

    float o[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[t][n][j] = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) m[n][j] = -INFINITY, l[n][j] = 0.0f;
    int unit = 0;             // scale byte of o

    // pages and scales one step ahead of their use
    int pgs[C::kStages];      // pages of groups i .. i + kStages - 1
#pragma unroll
    for (int j = 0; j < C::kStages; ++j) pgs[j] = page_of(j);
#pragma unroll
    for (int j = 0; j < C::kStages - 1; ++j) issue(j, pgs[j]);
    auto scale_of = [&](const uint8_t* s, int pg) { return pg >= 0 ? int(__ldg(s + (size_t)pg * H + h)) : 0; };
    int ks_n = scale_of(a.c.k_scales, pgs[0]), vs_n = scale_of(a.c.v_scales, pgs[0]);

    for (int i = 0; i < n_my; ++i) {
      issue(i + C::kStages - 1, pgs[C::kStages - 1]);
      const int pg = pgs[0], ks = ks_n, vs = vs_n;
#pragma unroll
      for (int j = 0; j + 1 < C::kStages; ++j) pgs[j] = pgs[j + 1];
      pgs[C::kStages - 1] = page_of(i + C::kStages);
      ks_n = scale_of(a.c.k_scales, pgs[0]);
      vs_n = scale_of(a.c.v_scales, pgs[0]);
      cp_async_wait<C::kStages - 1>();
      const int t0 = gpos(i);
      if (pg < 0) {
        if (a.status && lane == 0) atomicOr(a.status, MOE_DEV_INDEX_OOB);
      }
      const uint4* st = reinterpret_cast<const uint4*>(ring + (i % C::kStages) * C::kStageBytes) + lane;

      // scores
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][j] = 0.0f;
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const uint4 ka = st[(2 * j) * 32], kb = st[(2 * j + 1) * 32];
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a0 = e4m3x2_f16x2(wa[k]), a2 = e4m3x2_f16x2_hi(wa[k]);
          const uint32_t a1 = e4m3x2_f16x2(wb[k]), a3 = e4m3x2_f16x2_hi(wb[k]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(s[n], a0, a1, a2, a3, qf[4 * j + k][n][0], qf[4 * j + k][n][1]);
        }
      }
      const bool full = pg >= 0 && t0 + 16 <= L - T + 1;   // every row sees every position
      const float kf = exp2i(ks - 127);
      bool raise = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[n][j] *= qs[n][j & 1] * kf;
          if (!full && (pg < 0 || t0 + g + (j >> 1) * 8 >= vis[n][j & 1])) s[n][j] = -INFINITY;
          raise |= s[n][j] > m[n][j & 1] + kRaise;
        }
      if (WT) {
        const int64_t pair = (int64_t)b * H + h;
        float* sc = p.scores + (pair * p.cap + t0) * C::kRows + rt * NT * 8 + 2 * c;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (t0 + g < L) *reinterpret_cast<float2*>(sc + (size_t)g * C::kRows + n * 8) = make_float2(s[n][0], s[n][1]);
          if (t0 + g + 8 < L)
            *reinterpret_cast<float2*>(sc + (size_t)(g + 8) * C::kRows + n * 8) = make_float2(s[n][2], s[n][3]);
        }
      }
      if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(s[n][j], s[n][j + 2]);
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
            x = fmaxf(x, m[n][j]);
            const float f = x == m[n][j] ? 1.0f : ex2(m[n][j] - x);   // equal also where both are -inf
            m[n][j] = x;
            l[n][j] *= f;
#pragma unroll
            for (int t = 0; t < MT; ++t) o[t][n][j] *= f, o[t][n][j + 2] *= f;
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          e[j] = s[n][j] == -INFINITY ? 0.0f : ex2(s[n][j] - m[n][j & 1]);
          l[n][j & 1] += e[j];
        }
        pb[n][0] = movm(f16x2_bits(e[0], e[1]));
        pb[n][1] = movm(f16x2_bits(e[2], e[3]));
      }
      if (pg < 0) continue;

      // output
      uint32_t vw[4][KC * 2];   // codes of the positions 2c, 2c+1, 2c+8, 2c+9
      if (D == 128) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 v = st[(2 * KC + j) * 32];
          vw[j][0] = v.x;
          vw[j][1] = v.y;
          vw[j][KC * 2 - 2] = v.z;
          vw[j][KC * 2 - 1] = v.w;
        }
      } else {
        // lanes g and g ^ 1 hold the two positions of a pair for the same 16
        // channels: each keeps its half (8 channels) of both
        const uint4 u = st[(2 * KC) * 32], v = st[(2 * KC + 1) * 32];
        const bool odd = g & 1;
        const uint32_t su0 = odd ? u.x : u.z, su1 = odd ? u.y : u.w, sv0 = odd ? v.x : v.z, sv1 = odd ? v.y : v.w;
        const uint32_t ru0 = __shfl_xor_sync(0xFFFFFFFFu, su0, 4), ru1 = __shfl_xor_sync(0xFFFFFFFFu, su1, 4);
        const uint32_t rv0 = __shfl_xor_sync(0xFFFFFFFFu, sv0, 4), rv1 = __shfl_xor_sync(0xFFFFFFFFu, sv1, 4);
        vw[0][0] = odd ? ru0 : u.x;
        vw[0][1] = odd ? ru1 : u.y;
        vw[1][0] = odd ? u.z : ru0;
        vw[1][1] = odd ? u.w : ru1;
        vw[2][0] = odd ? rv0 : v.x;
        vw[2][1] = odd ? rv1 : v.y;
        vw[3][0] = odd ? v.z : rv0;
        vw[3][1] = odd ? v.w : rv1;
      }
      bool poison = false;
      if (!full) {
        // positions past the end hold anything: zero codes
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool out = t0 + 2 * c + (j & 1) + (j >> 1) * 8 >= L;
#pragma unroll
          for (int w = 0; w < KC * 2; ++w) {
            if (out) vw[j][w] = 0;
            poison |= any_nan4(vw[j][w]);
          }
        }
        poison = __any_sync(0xFFFFFFFFu, poison) && T > 1;
      }
      if (vs > unit) {
        const float f = exp2i(unit - vs);
        unit = vs;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[t][n][j] *= f;
      }
      // one pass; or, where a NaN is visible to some tokens only (0 * NaN is
      // NaN), a pass for each token over what it sees
      for (int pass = 0; pass < (poison ? T : 1); ++pass) {
        const float f = exp2i(vs - unit);
        const bool direct = vs == unit && !poison;
        const int seen = poison ? L - T + pass + 1 : 0x7FFFFFFF;
#pragma unroll
        for (int w = 0; w < KC * 2; ++w) {
          uint32_t x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = t0 + 2 * c + (j & 1) + (j >> 1) * 8 >= seen ? 0u : vw[j][w];
          const uint32_t p0 = __byte_perm(x[0], x[1], 0x5140), p1 = __byte_perm(x[0], x[1], 0x7362);
          const uint32_t p2 = __byte_perm(x[2], x[3], 0x5140), p3 = __byte_perm(x[2], x[3], 0x7362);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t lo2 = k ? p1 : p0, hi2 = k ? p3 : p2;
            const uint32_t a0 = e4m3x2_f16x2(lo2), a1 = e4m3x2_f16x2_hi(lo2);
            const uint32_t a2 = e4m3x2_f16x2(hi2), a3 = e4m3x2_f16x2_hi(hi2);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (direct) {
                mma_f16(o[2 * w + k][n], a0, a1, a2, a3, pb[n][0], pb[n][1]);
              } else {
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_f16(d, a0, a1, a2, a3, pb[n][0], pb[n][1]);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (!poison || vis[n][j & 1] == seen) o[2 * w + k][n][j] = fmaf(d[j], f, o[2 * w + k][n][j]);
              }
            }
          }
        }
      }
    }
    cp_async_wait<0>();

    // lanes' sums; the warp's partials to shared memory
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[n][j] += __shfl_xor_sync(0xFFFFFFFFu, l[n][j], 4);
        l[n][j] += __shfl_xor_sync(0xFFFFFFFFu, l[n][j], 8);
        l[n][j] += __shfl_xor_sync(0xFFFFFFFFu, l[n][j], 16);
      }
    __syncthreads();   // every warp has left the ring
    float* mo = reinterpret_cast<float*>(smem);                    // [warp][8 NT][D]
    float* mm = mo + kDecWarps * 8 * NT * D;                       // [warp][8 NT]
    float* ml = mm + kDecWarps * 8 * NT;
    {
      const float f = exp2i(unit - 127);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = n * 8 + 2 * c + j;
          float* row = mo + ((size_t)warp * 8 * NT + r) * D + g * (D / 8);
#pragma unroll
          for (int t = 0; t < MT; ++t)
            *reinterpret_cast<float2*>(row + 2 * t) = make_float2(o[t][n][j] * f, o[t][n][j + 2] * f);
          if (g == 0) {
            mm[warp * 8 * NT + r] = m[n][j];
            ml[warp * 8 * NT + r] = l[n][j];
          }
        }
    }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == nu;
    const int64_t pair = (int64_t)b * H + h;
    const int slot = u0 > 0 ? 0 : 1;   // continues an earlier CTA's part, or begins the pair
    float* part = p.parts + ((size_t)blockIdx.x * 2 + slot) * C::kRows * (D + 2);
    // 4 channels per thread
    auto finish = [&](int r, int d4, float4 acc, float M, float Ls) {
      const int tok = r / p.G, hq = h * p.G + r % p.G;
      const float inv = Ls > 0.0f ? 1.0f / Ls : (Ls == 0.0f ? 0.0f : Ls);   // NaN stays NaN
      const int64_t row = ((int64_t)b * T + tok) * a.n_heads + hq;
      const __nv_bfloat162 y0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
      const __nv_bfloat162 y1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      uint2 y;
      y.x = *reinterpret_cast<const uint32_t*>(&y0);
      y.y = *reinterpret_cast<const uint32_t*>(&y1);
      *reinterpret_cast<uint2*>(a.out + row * D + d4) = y;
      if (d4 == 0) {
        const float lse2 = Ls == 0.0f ? -INFINITY : M + log2f(Ls);
        if (a.lse) a.lse[row] = lse2 * kLn2;
        if (WT) p.lse2[pair * C::kRows + r] = lse2;
      }
    };
    for (int i = tid; i < C::kRows * (D / 4); i += kDecThreads) {
      const int r = i / (D / 4), d4 = (i % (D / 4)) * 4;
      if (r >= p.rows) continue;
      const int w0 = r / (8 * NT), rr = r % (8 * NT);   // row tile; row inside it
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < C::kGroups; ++k) M = fmaxf(M, mm[(k * RT + w0) * 8 * NT + rr]);
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float Ls = 0.0f;
#pragma unroll
      for (int k = 0; k < C::kGroups; ++k) {
        const int wr = (k * RT + w0) * 8 * NT + rr;
        const float mw = mm[wr];
        if (mw == -INFINITY && ml[wr] == 0.0f) continue;
        const float f = mw == M ? 1.0f : ex2(mw - M);
        const float4 v = *reinterpret_cast<const float4*>(mo + (size_t)wr * D + d4);
        acc.x = fmaf(v.x, f, acc.x);
        acc.y = fmaf(v.y, f, acc.y);
        acc.z = fmaf(v.z, f, acc.z);
        acc.w = fmaf(v.w, f, acc.w);
        Ls = fmaf(ml[wr], f, Ls);
      }
      if (whole) {
        finish(r, d4, acc, M, Ls);
      } else {
        *reinterpret_cast<float4*>(part + (size_t)r * D + d4) = acc;
        if (d4 == 0) {
          part[C::kRows * D + r] = M;
          part[C::kRows * (D + 1) + r] = Ls;
        }
      }
    }
    if (!whole) {
      // CTAs of this pair: those whose ranges meet units [s0, s1)
      const int64_t s0 = pair0 + (int64_t)h * nu, s1 = s0 + nu;
      const int c0 = int(((s0 + 1) * N - 1) / W), c1 = int((s1 * N - 1) / W);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const unsigned seen = atomicAdd(p.counter + pair, 1u);
        s_last = seen == unsigned(c1 - c0);
        if (s_last) p.counter[pair] = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int i = tid; i < C::kRows * (D / 4); i += kDecThreads) {
          const int r = i / (D / 4), d4 = (i % (D / 4)) * 4;
          if (r >= p.rows) continue;
          float M = -INFINITY;
          float Ls = 0.0f;
          float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int k = c0; k <= c1; ++k) {
            const float* q = p.parts + ((size_t)k * 2 + (k == c0 ? 1 : 0)) * C::kRows * (D + 2);
            const float mw = __ldcg(q + C::kRows * D + r), lw = __ldcg(q + C::kRows * (D + 1) + r);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(q + (size_t)r * D + d4));
            if (mw == -INFINITY && lw == 0.0f) continue;
            const float Mn = fmaxf(M, mw);
            const float f0 = M == Mn ? 1.0f : ex2(M - Mn), f1 = mw == Mn ? 1.0f : ex2(mw - Mn);
            M = Mn;
            acc.x = acc.x * f0 + v.x * f1;
            acc.y = acc.y * f0 + v.y * f1;
            acc.z = acc.z * f0 + v.z * f1;
            acc.w = acc.w * f0 + v.w * f1;
            Ls = Ls * f0 + lw * f1;
          }
          finish(r, d4, acc, M, Ls);
        }
      }
    }
    __syncthreads();   // shared memory is used again
    pos += u1 - u0;
  }
}

// weights[pair][j] += sum over the query rows of exp(score - log-sum-exp).
template <int ROWS>
__global__ void __launch_bounds__(256) decode_weights_kernel(const DecParams p) {
  const DecodeArgs& a = p.a;
  const int b = blockIdx.z, h = blockIdx.y;
  const int64_t pair = (int64_t)b * a.c.n_kv_heads + h;
  bool ignore = false;
  const int L = dec_length(a, b, &ignore);
  __shared__ float s_lse[ROWS];
  for (int r = threadIdx.x; r < ROWS; r += blockDim.x) s_lse[r] = r < p.rows ? p.lse2[pair * ROWS + r] : 0.0f;
  __syncthreads();
  for (int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; j < L; j += (int64_t)gridDim.x * blockDim.x) {
    const float4* s = reinterpret_cast<const float4*>(p.scores + (pair * p.cap + j) * ROWS);
    float w = 0.0f;
#pragma unroll
    for (int r4 = 0; r4 < ROWS / 4; ++r4) {
      const float4 v = __ldcs(s + r4);
      const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * r4 + i;
        if (r < p.rows && x[i] != -INFINITY) w += ex2(x[i] - s_lse[r]);
      }
    }
    a.weights[pair * a.w_stride + j] += w;
  }
}

size_t ws_layout(const moe_kv_cache& c, int n_seq, int n_new, int n_heads, int width, bool weights, int n_cta, DecWs* w) {
  const int rows = n_new * (n_heads / c.n_kv_heads);
  const DecPlan pl = dec_plan(rows);
  w->rows = 8 * pl.nt * pl.rt;
  w->n_cta = n_cta;
  const size_t pairs = (size_t)n_seq * c.n_kv_heads;
  w->parts = round_up(pairs * 4, 256);
  w->lse2 = w->parts + round_up((size_t)n_cta * 2 * w->rows * (c.head_dim + 2) * 4, 256);
  w->scores = w->lse2 + (weights ? round_up(pairs * w->rows * 4, 256) : 0);
  w->total = w->scores + (weights ? pairs * ((size_t)width * c.page_size) * w->rows * 4 : 0);
  if (w->total == 0) w->total = 256;
  return w->total;
}

template <int D, int NT, int RT, bool WT>
int launch_one(const DecParams& p, int n_cta, cudaStream_t s) {
  using C = DecCfg<D, NT, RT, WT>;
  MOE_CUDA_TRY(cudaFuncSetAttribute(decode_attn_kernel<D, NT, RT, WT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(C::kSmem)));
  decode_attn_kernel<D, NT, RT, WT><<<n_cta, kDecThreads, C::kSmem, s>>>(p);
  int st = launch_status();
  if (st != MOE_OK || !WT) return st;
  if (p.cap == 0) return MOE_OK;
  const int64_t blocks = (p.cap + 255) / 256;
  const dim3 grid(unsigned(blocks < 64 ? blocks : 64), p.a.c.n_kv_heads, p.a.n_seq);
  decode_weights_kernel<C::kRows><<<grid, 256, 0, s>>>(p);
  return launch_status();
}
template <int D, bool WT>
int launch_plan(const DecParams& p, const DecPlan& pl, int n_cta, cudaStream_t s) {
  if (pl.nt == 1) return launch_one<D, 1, 1, WT>(p, n_cta, s);
  if (pl.rt == 1) return launch_one<D, 2, 1, WT>(p, n_cta, s);
  if (pl.rt == 2) return launch_one<D, 2, 2, WT>(p, n_cta, s);
  return launch_one<D, 2, 4, WT>(p, n_cta, s);
}

}  // namespace

size_t attn_decode_ws_bytes(const moe_kv_cache& c, int n_seq, int n_new, int n_heads, int width, bool weights,
                            const DeviceInfo& di) {
  DecWs w;
  return ws_layout(c, n_seq, n_new, n_heads, width, weights, di.sm_count, &w);
}

int launch_attn_decode(const DecodeArgs& a, const DeviceInfo& di, cudaStream_t s) {
  DecWs w;
  const bool wt = a.weights != nullptr;
  ws_layout(a.c, a.n_seq, a.n_new, a.n_heads, a.width, wt, di.sm_count, &w);
  DecParams p{};
  p.a = a;
  p.G = a.n_heads / a.c.n_kv_heads;
  p.rows = a.n_new * p.G;
  char* base = static_cast<char*>(a.ws);
  p.counter = reinterpret_cast<unsigned*>(base);
  p.parts = reinterpret_cast<float*>(base + w.parts);
  p.lse2 = reinterpret_cast<float*>(base + w.lse2);
  p.scores = reinterpret_cast<float*>(base + w.scores);
  p.cap = (int64_t)a.width * a.c.page_size;
  const DecPlan pl = dec_plan(p.rows);
  if (a.c.head_dim == 128) return wt ? launch_plan<128, true>(p, pl, w.n_cta, s) : launch_plan<128, false>(p, pl, w.n_cta, s);
  return wt ? launch_plan<64, true>(p, pl, w.n_cta, s) : launch_plan<64, false>(p, pl, w.n_cta, s);
}

}  // namespace moe
