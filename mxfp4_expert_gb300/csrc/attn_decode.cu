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
// Inside a CTA the warps take chunks of 32 positions. A warp's next chunks are on
// their way into its own part of shared memory by cp.async: no CTA barrier. Both
// products run on the e4m3 warp MMA (m16n8k32, exact products, fp32 sums), which
// takes the cache's codes as they are: no conversion, 4096 multiplies a cycle and
// SM (measured: one MMA per 1.07 cycles; f16's m16n8k16 takes 2.03, and its
// conversions from E4M3 another 1.5 per 512 bytes).
//   scores   S^T[pos][row] = K q^T. A bf16 query value is two e4m3 terms, t0 its
//            first 4 significant bits, t1 the other 4 times 16, after a power
//            of two per row that puts the row's largest in [2^7, 2^8): exact
//            down to 2^-13 of that, then within 2^-22 of it. Lane (g, c) takes
//            16-byte pieces of the positions 2g and 2g + 1 as consecutive
//            words of its A fragment; q is laid out in the same order.
//   output   O^T[d][row] = V^T P^T. ldmatrix transposes bytes on the way from
//            shared memory, so lane (g, c) holds 4 consecutive positions of
//            channel g. The probabilities of a chunk, relative to the chunk's
//            largest times 2^8, are three e4m3 terms (12 significant bits, and
//            2^-18 of the largest); since S's rows were dealt 2g, 2g + 1, a
//            movmatrix on byte pairs turns them into the B operand.
//   joining  a chunk's product goes into O with an fp32 factor per row that
//            holds its reference and its page's value scale. A page of 16
//            positions shares its chunk with another: the probabilities then
//            carry the difference of the scales, and their reference is the
//            largest product of both, so no page is rounded for another's sake.
// The references of O and of the sum follow the maximum only when it passes them
// by 2^30: fp32 has the range, and O is hardly ever rescaled.
#include "attn.h"
#include "fp8kv.cuh"

namespace moe {
namespace {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kMaxSeqs = 4096;
constexpr float kRaise = 30.0f;    // log2 by which a score may pass the reference
constexpr int kChunk = 32;         // positions per warp step
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Workspace: counters [n_seq * n_kv], then partials, then (with weights) the
// rows' log2-sum-exp and the scores.
struct DecWs {
  size_t parts, lse2, scores, total;
  int n_cta, rows;    // CTAs; query rows padded to the row tiles
};

struct DecPlan {
  int nt, rt;         // blocks of 8 query rows per warp; row tiles
};
// Up to 24 rows stay with one warp (its output takes 32 registers a block at
// head_dim 128); more are cut into tiles whose warps read the same positions.
inline DecPlan dec_plan(int rows) {
  if (rows <= 8) return {1, 1};
  if (rows <= 16) return {2, 1};
  if (rows <= 24) return {3, 1};
  if (rows <= 32) return {2, 2};
  if (rows <= 48) return {3, 2};
  return {2, 4};
}

struct DecParams {
  DecodeArgs a;
  int G, rows;              // query heads per kv head; query rows n_new * G
  unsigned* counter;        // [n_seq * n_kv]
  float* parts;             // [n_cta][2][rows padded][D + 4]: output, then the references and the sum
  float* lse2;              // [n_seq * n_kv][rows padded] (weights)
  float* scores;            // [n_seq * n_kv][cap][rows padded] (weights)
  int64_t cap;
  int log2_page;
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
__device__ __forceinline__ void mma_fp8(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// Two 16 x 16 byte matrices, rows of 16 bytes at the lanes' addresses (lanes 0
// .. 15 the first's), transposed: lane (g, c) gets bytes 4c .. 4c + 3 of the
// columns g and g + 8 of the first, then of the second.
__device__ __forceinline__ void ldm_trans8(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// e4m3 pairs (a, b) and (c, d) -> one word, a in the lowest byte
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return uint32_t(f32x2_to_e4m3x2(a, b)) | uint32_t(f32x2_to_e4m3x2(c, d)) << 16;
}
__device__ __forceinline__ float top4(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFF00000u); }
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
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kGroups = kDecWarps / RT;         // chunks in work per CTA step
  static constexpr int kUnit = kChunk * kGroups;         // positions per unit
  static constexpr int kRows = 8 * NT * RT;              // padded query rows
  static constexpr uint32_t kKBytes = kChunk * D;
  static constexpr uint32_t kVCol = kChunk * 16 + 64;    // 16 channels of a chunk; 64 bytes on, for the banks
  static constexpr uint32_t kStageBytes = kKBytes + D / 16 * kVCol;
  static constexpr uint32_t kRing = kDecWarps * kStages * kStageBytes;
  static constexpr int kLd = D + 4;                      // row stride of the merge, floats
  static constexpr uint32_t kMerge = kDecWarps * 8 * NT * (kLd + 3) * 4;   // reuses the ring
  static constexpr uint32_t kPrefix = kRing > kMerge ? kRing : kMerge;
  static constexpr uint32_t kSmem = kPrefix + (kMaxSeqs + 1) * 4;
  static constexpr int kPart = kRows * (D + 4);          // floats of a partial result
};

template <int D, int NT, int RT, bool WT>
__global__ void __launch_bounds__(kDecThreads) decode_attn_kernel(const DecParams p) {
  using C = DecCfg<D, NT, RT, WT>;
  constexpr int KS = D / 32;      // MMA steps over the channels
  constexpr int MT = D / 16;      // 16-channel blocks of the output
  constexpr int KC = D / 64;      // 16-byte pieces per lane and position
  extern __shared__ __align__(128) uint8_t smem[];
  int* prefix = reinterpret_cast<int*>(smem + C::kPrefix);
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
  const uint32_t ring_s = smem_addr(ring);

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
    const int n_my = last > first + tg * kChunk ? (last - first - tg * kChunk + C::kUnit - 1) / C::kUnit : 0;
    const int32_t* table = a.table + (size_t)b * a.width;
    const size_t head_bytes = (size_t)P * D, page_bytes = head_bytes * H;
    const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k_codes) + h * head_bytes;
    const uint8_t* vbase = static_cast<const uint8_t*>(a.c.v_codes) + h * head_bytes;

    auto gpos = [&](int i) { return first + (i * C::kGroups + tg) * kChunk; };
    // Pages and scales of 32 chunks at a time, lane l those of the l-th: halves
    // (16 positions) A and B, -1 outside the table or the cache. Scales of the
    // chunks in work and of those being fetched.
    int pg_a = -1, pg_b = -1;
    uint32_t sc_next = 0, sc = 0;                                   // scale bytes kA kB vA vB
    uint32_t bad_na = 0, bad_nb = 0, bad_a = 0, bad_b = 0;          // chunks whose half has no page
    auto lookup = [&](int i0) {
      const int i = i0 + lane;
      const int t = gpos(i);
      pg_a = pg_b = -1;
      uint32_t w = 0;
      bool oob_a = false, oob_b = false;
      if (i < n_my) {
        pg_a = __ldg(table + (t >> p.log2_page));
        oob_a = pg_a < 0 || pg_a >= a.c.n_pages;
        if (oob_a) pg_a = -1;
        if (t + 16 < last) {
          pg_b = P == 16 ? __ldg(table + (t >> 4) + 1) : pg_a;
          oob_b = pg_b < 0 || pg_b >= a.c.n_pages;
          if (oob_b) pg_b = -1;
        }
        if (pg_a >= 0) {
          const size_t o = (size_t)pg_a * H + h;
          w = __ldg(a.c.k_scales + o) | uint32_t(__ldg(a.c.v_scales + o)) << 16;
        }
        if (pg_b >= 0) {
          const size_t o = (size_t)pg_b * H + h;
          w |= uint32_t(__ldg(a.c.k_scales + o)) << 8 | uint32_t(__ldg(a.c.v_scales + o)) << 24;
        } else {
          w |= (w & 0x00FF00FFu) << 8;
        }
      }
      sc_next = w;
      bad_na = __ballot_sync(0xFFFFFFFFu, oob_a);
      bad_nb = __ballot_sync(0xFFFFFFFFu, oob_b);
      if ((bad_na | bad_nb) && lane == 0 && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    };
    auto issue = [&](int i) {
      if ((i & 31) == 0) lookup(i);
      const int pa = __shfl_sync(0xFFFFFFFFu, pg_a, i & 31), pb = __shfl_sync(0xFFFFFFFFu, pg_b, i & 31);
      if (i < n_my) {
        const int slot = gpos(i) & (P - 1);
        const size_t ra = (size_t)max(pa, 0) * page_bytes + slot * D;
        const size_t rb = P == 16 ? (size_t)max(pb, 0) * page_bytes : ra + 16 * D;
        const uint32_t st = ring_s + (i % C::kStages) * C::kStageBytes;
        // keys: lane (g, c) what it will use, at its own 16 bytes of each row of 512
        const uint32_t ko = (2 * g) * D + c * 16;
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          if ((mt ? pb : pa) < 0) continue;
          const uint8_t* k0 = kbase + (mt ? rb : ra) + ko;
#pragma unroll
          for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int j = 0; j < KC; ++j)
              cp_async16(st + ((mt * 2 + o) * KC + j) * 512 + lane * 16, k0 + o * D + 64 * j);
        }
        // values: rows of D bytes, a lane 16 of them, to [16-channel block][position]
        constexpr int LPR = D / 16, RPI = 32 / LPR;   // lanes per row, rows per instruction
        const uint32_t vd = st + C::kKBytes + (lane % LPR) * C::kVCol + (lane / LPR) * 16;
        const uint32_t vo = (lane / LPR) * D + (lane % LPR) * 16;
#pragma unroll
        for (int n = 0; n < kChunk / RPI; ++n) {
          const bool second = n >= 16 / RPI;
          if ((second ? pb : pa) < 0) continue;
          cp_async16(vd + n * RPI * 16, vbase + (second ? rb + (n * RPI - 16) * D : ra + n * RPI * D) + vo);
        }
      }
      cp_async_commit();
    };

    // query rows -> B fragments (two e4m3 terms) and the factors that undo their scale
    uint32_t qf[2][KS][NT][2];
    float qs[NT][2];         // of rows 2c, 2c+1 of each block: 2^e scale log2(e)
    int vis[NT][2];          // positions that those rows see
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = (rt * NT + n) * 8 + g;
      float x[KC * 16];
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
        for (int i = 0; i < KC * 16; ++i) top = fmaxf(top, fabsf(x[i]));
      } else {
#pragma unroll
        for (int i = 0; i < KC * 16; ++i) x[i] = 0.0f;
      }
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      int e = 0;
      if (top > 0.0f && top < INFINITY) {
        frexpf(top, &e);
        e -= 8;              // the row's largest value in [2^7, 2^8)
      }
#pragma unroll
      for (int i = 0; i < KC * 16; i += 4) {
        float t0[4], t1[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // inf has no e4m3 code: the row is NaN, as softmax of infinite scores is
          const float y = fabsf(x[i + k]) == INFINITY ? __int_as_float(0x7FC00000) : scale2(x[i + k], -e);
          const uint32_t code = f32x2_to_e4m3x2(top4(y), 0.0f) & 0xFFu;
          t0[k] = e4m3_is_nan(code) ? y : e4m3_to_f32(code);
          t1[k] = (y - t0[k]) * 16.0f;
        }
        // 8 channels per MMA step: the first word is b0, the second b1
        qf[0][i / 8][n][(i / 4) & 1] = e4m3x4(t0[0], t0[1], t0[2], t0[3]);
        qf[1][i / 8][n][(i / 4) & 1] = e4m3x4(t1[0], t1[1], t1[2], t1[3]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int er = __shfl_sync(0xFFFFFFFFu, e, (2 * c + j) * 4);
        const int rr = (rt * NT + n) * 8 + 2 * c + j;
        qs[n][j] = scale2(a.scale * kLog2e, er);
        vis[n][j] = rr < p.rows ? L - T + rr / p.G + 1 : 0;
      }
    }

    // O (in units of 2^ro), the sum (of 2^m)
    float o[MT][NT][4], m[NT][2], ro[NT][2], l[NT][2];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[t][n][j] = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) m[n][j] = ro[n][j] = -INFINITY, l[n][j] = 0.0f;

#pragma unroll 1
    for (int j = 0; j < C::kStages - 1; ++j) {
      issue(j);
      if (j == 0) sc = sc_next, bad_a = bad_na, bad_b = bad_nb;
    }

#pragma unroll 1
    for (int i = 0; i < n_my; ++i) {
      issue(i + C::kStages - 1);
      if ((i & 31) == 0) sc = sc_next, bad_a = bad_na, bad_b = bad_nb;   // fetches are ahead by less than 32
      cp_async_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t w = __shfl_sync(0xFFFFFFFFu, sc, i & 31);
      const int t0 = gpos(i);
      const int va = int(w >> 16 & 0xFFu), vb = int(w >> 24);
      const bool no_a = bad_a >> (i & 31) & 1u, no_b = bad_b >> (i & 31) & 1u;
      const uint32_t st = (i % C::kStages) * C::kStageBytes;
      const uint4* kst = reinterpret_cast<const uint4*>(ring + st) + lane;
      const bool full = !no_a && !no_b && t0 + kChunk <= L - T + 1;   // every row sees every position

      uint32_t pf[3][NT][2];      // probabilities: terms, row blocks, halves
      float beta[NT][2];
      {
        uint4 kw[2][2][KC];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int j = 0; j < KC; ++j) kw[mt][x][j] = kst[((mt * 2 + x) * KC + j) * 32];
        const float kfa = exp2i(int(w & 0xFFu) - 127), kfb = exp2i(int(w >> 8 & 0xFFu) - 127);
        const float vfa = float(va - 127), vfb = float(vb - 127);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float s[2][4];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            float s1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j) s[mt][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < KC; ++j) {
              const uint4 x = kw[mt][0][j], y = kw[mt][1][j];
              const uint32_t a0[4] = {x.x, y.x, x.y, y.y}, a1[4] = {x.z, y.z, x.w, y.w};
              mma_fp8(s[mt], a0, qf[0][2 * j][n][0], qf[0][2 * j][n][1]);
              mma_fp8(s1, a0, qf[1][2 * j][n][0], qf[1][2 * j][n][1]);
              mma_fp8(s[mt], a1, qf[0][2 * j + 1][n][0], qf[0][2 * j + 1][n][1]);
              mma_fp8(s1, a1, qf[1][2 * j + 1][n][0], qf[1][2 * j + 1][n][1]);
            }
            // s[mt][x]: position t0 + 16 mt + 2g + x / 2, row 2c + x % 2
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              s[mt][x] = fmaf(s1[x], 0.0625f, s[mt][x]) * (qs[n][x & 1] * (mt ? kfb : kfa));
              if (!full && ((mt ? no_b : no_a) || t0 + 16 * mt + 2 * g + (x >> 1) >= vis[n][x & 1])) s[mt][x] = -INFINITY;
            }
          }
          if (WT) {
            float* sp = p.scores + (((int64_t)b * H + h) * p.cap + t0 + 2 * g) * C::kRows + (rt * NT + n) * 8 + 2 * c;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int x = 0; x < 2; ++x)
                if (t0 + 16 * mt + 2 * g + x < L)
                  *reinterpret_cast<float2*>(sp + (16 * mt + x) * C::kRows) = make_float2(s[mt][2 * x], s[mt][2 * x + 1]);
          }
          // the chunk's largest score, and largest score times value scale
          float us[2], ms[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float xa = fmaxf(s[0][j], s[0][j + 2]), xb = fmaxf(s[1][j], s[1][j + 2]);
            us[j] = fmaxf(xa + vfa, xb + vfb);
            us[j] = fmaxf(us[j], __shfl_xor_sync(0xFFFFFFFFu, us[j], 4));
            us[j] = fmaxf(us[j], __shfl_xor_sync(0xFFFFFFFFu, us[j], 8));
            us[j] = fmaxf(us[j], __shfl_xor_sync(0xFFFFFFFFu, us[j], 16));
            ms[j] = fmaxf(xa, xb);
          }
          if (va == vb) {
            ms[0] = us[0] - vfa;
            ms[1] = us[1] - vfa;
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              ms[j] = fmaxf(ms[j], __shfl_xor_sync(0xFFFFFFFFu, ms[j], 4));
              ms[j] = fmaxf(ms[j], __shfl_xor_sync(0xFFFFFFFFu, ms[j], 8));
              ms[j] = fmaxf(ms[j], __shfl_xor_sync(0xFFFFFFFFu, ms[j], 16));
            }
          }
          const bool raise = ms[0] > m[n][0] + kRaise || ms[1] > m[n][1] + kRaise || us[0] > ro[n][0] + kRaise ||
                             us[1] > ro[n][1] + kRaise;
          if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (ms[j] > m[n][j] + kRaise) {
                l[n][j] *= ex2(m[n][j] - ms[j]);
                m[n][j] = ms[j];
              }
              if (us[j] > ro[n][j] + kRaise) {
                const float f = ex2(ro[n][j] - us[j]);
                ro[n][j] = us[j];
#pragma unroll
                for (int t = 0; t < MT; ++t) o[t][n][j] *= f, o[t][n][j + 2] *= f;
              }
            }
          }
          // probabilities times 2^8 over the chunk's largest, in three terms
          float pr[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const bool none = us[j] == -INFINITY;
            const float ref = none ? 0.0f : 8.0f - us[j];
            beta[n][j] = none ? 0.0f : ex2(us[j] - 8.0f - ro[n][j]);
#pragma unroll
            for (int x = j; x < 4; x += 2) {
              pr[0][x] = ex2(s[0][x] + (vfa + ref));
              pr[1][x] = ex2(s[1][x] + (vfb + ref));
            }
            if (va == vb) {
              const float sum = (pr[0][j] + pr[0][j + 2]) + (pr[1][j] + pr[1][j + 2]);
              // a row of NaN scores has no largest one, but must not pass for empty
              l[n][j] += none ? sum : sum * ex2(us[j] - 8.0f - vfa - m[n][j]);
            } else {
              const float mr = m[n][j] == -INFINITY ? 0.0f : m[n][j];
              l[n][j] += (ex2(s[0][j] - mr) + ex2(s[0][j + 2] - mr)) + (ex2(s[1][j] - mr) + ex2(s[1][j + 2] - mr));
            }
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            float t0v[4], t1v[4], t2v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              t0v[x] = top4(pr[mt][x]);
              const float r = pr[mt][x] - t0v[x];
              t1v[x] = top4(r);
              t2v[x] = r - t1v[x];
            }
            // row 2c's pair (positions 2g, 2g + 1), row 2c + 1's pair
            pf[0][n][mt] = movm(e4m3x4(t0v[0], t0v[2], t0v[1], t0v[3]));
            pf[1][n][mt] = movm(e4m3x4(t1v[0], t1v[2], t1v[1], t1v[3]));
            pf[2][n][mt] = movm(e4m3x4(t2v[0], t2v[2], t2v[1], t2v[3]));
          }
        }
      }

      // output
      const uint32_t va_s = ring_s + st + C::kKBytes + lane * 16;
      if (full) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          uint32_t x[4];
          ldm_trans8(x, va_s + t * C::kVCol);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_fp8(d, x, pf[2][n][0], pf[2][n][1]);
            mma_fp8(d, x, pf[1][n][0], pf[1][n][1]);
            mma_fp8(d, x, pf[0][n][0], pf[0][n][1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[t][n][j] = fmaf(d[j], beta[n][j & 1], o[t][n][j]);
          }
        }
      } else {
        // Positions past the end hold anything: their codes are zeroed. A half
        // without a page too. Where a NaN is visible to some tokens only (0 * NaN is NaN) every token takes
        // a pass over what it sees.
        auto keep4 = [&](int first_pos, int seen) {   // bytes of 4 consecutive positions
          const int k = seen - first_pos;
          return k >= 4 ? 0xFFFFFFFFu : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
        };
        bool poison = false;
        if (T > 1) {
          const uint32_t ka = no_a ? 0u : keep4(t0 + 4 * c, L), kb = no_b ? 0u : keep4(t0 + 16 + 4 * c, L);
#pragma unroll 1
          for (int t = 0; t < MT; ++t) {
            uint32_t x[4];
            ldm_trans8(x, va_s + t * C::kVCol);
            poison |= any_nan4(x[0] & ka) || any_nan4(x[1] & ka) || any_nan4(x[2] & kb) || any_nan4(x[3] & kb);
          }
          poison = __any_sync(0xFFFFFFFFu, poison);
        }
        const int n_pass = poison ? T : 1;
#pragma unroll 1
        for (int pass = 0; pass < n_pass; ++pass) {
          const int seen = poison ? L - T + pass + 1 : L;
          const uint32_t ka = no_a ? 0u : keep4(t0 + 4 * c, seen), kb = no_b ? 0u : keep4(t0 + 16 + 4 * c, seen);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            uint32_t x[4];
            ldm_trans8(x, va_s + t * C::kVCol);
            x[0] &= ka;
            x[1] &= ka;
            x[2] &= kb;
            x[3] &= kb;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma_fp8(d, x, pf[2][n][0], pf[2][n][1]);
              mma_fp8(d, x, pf[1][n][0], pf[1][n][1]);
              mma_fp8(d, x, pf[0][n][0], pf[0][n][1]);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (!poison || vis[n][j & 1] == seen) o[t][n][j] = fmaf(d[j], beta[n][j & 1], o[t][n][j]);
            }
          }
        }
      }
      __syncwarp();   // every lane has read the stage before it is filled again
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
    constexpr int LD = C::kLd;
    float* mo = reinterpret_cast<float*>(smem);                    // [warp][8 NT][LD]
    float* mr = mo + kDecWarps * 8 * NT * LD;                      // [warp][8 NT]: reference of O
    float* mm = mr + kDecWarps * 8 * NT;                           //   of the sum
    float* ml = mm + kDecWarps * 8 * NT;                           //   the sum
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = warp * 8 * NT + n * 8 + 2 * c + j;
        float* row = mo + (size_t)r * LD + g;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          row[16 * t] = o[t][n][j];
          row[16 * t + 8] = o[t][n][j + 2];
        }
        if (g == 0) {
          mr[r] = ro[n][j];
          mm[r] = m[n][j];
          ml[r] = l[n][j];
        }
      }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == nu;
    const int64_t pair = (int64_t)b * H + h;
    const int slot = u0 > 0 ? 0 : 1;   // continues an earlier CTA's part, or begins the pair
    float* part = p.parts + ((size_t)blockIdx.x * 2 + slot) * C::kPart;
    // running (O, its reference, sum, its reference) + another's
    struct Acc {
      float4 o;
      float r, m, l;
    };
    auto join = [](Acc& x, float4 v, float r, float mw, float lw) {
      if (mw == -INFINITY && lw == 0.0f) return;   // saw nothing
      if (r > -INFINITY) {
        const float R = fmaxf(x.r, r);
        const float f0 = x.r == R ? 1.0f : ex2(x.r - R), f1 = r == R ? 1.0f : ex2(r - R);
        x.r = R;
        x.o.x = x.o.x * f0 + v.x * f1;
        x.o.y = x.o.y * f0 + v.y * f1;
        x.o.z = x.o.z * f0 + v.z * f1;
        x.o.w = x.o.w * f0 + v.w * f1;
      }
      const float M = fmaxf(x.m, mw);
      const float g0 = x.m == M ? 1.0f : ex2(x.m - M), g1 = mw == M ? 1.0f : ex2(mw - M);
      x.m = M;
      x.l = x.l * g0 + lw * g1;
    };
    // 4 channels per thread
    auto finish = [&](int r, int d4, const Acc& x) {
      const int tok = r / p.G, hq = h * p.G + r % p.G;
      const int64_t row = ((int64_t)b * T + tok) * a.n_heads + hq;
      float f = 0.0f;                               // nothing seen: zeros
      if (x.l != 0.0f) f = x.r == -INFINITY ? x.l : ex2(x.r - x.m) / x.l;   // a row of NaN scores: NaN
      const __nv_bfloat162 y0 = __floats2bfloat162_rn(x.o.x * f, x.o.y * f);
      const __nv_bfloat162 y1 = __floats2bfloat162_rn(x.o.z * f, x.o.w * f);
      uint2 y;
      y.x = *reinterpret_cast<const uint32_t*>(&y0);
      y.y = *reinterpret_cast<const uint32_t*>(&y1);
      *reinterpret_cast<uint2*>(a.out + row * D + d4) = y;
      if (d4 == 0) {
        const float lse2 = x.l == 0.0f ? -INFINITY : (x.m == -INFINITY ? x.l : x.m + log2f(x.l));
        if (a.lse) a.lse[row] = lse2 * kLn2;
        if (WT) p.lse2[pair * C::kRows + r] = lse2;
      }
    };
    for (int i = tid; i < C::kRows * (D / 4); i += kDecThreads) {
      const int r = i / (D / 4), d4 = (i % (D / 4)) * 4;
      if (r >= p.rows) continue;
      const int w0 = r / (8 * NT), rr = r % (8 * NT);   // row tile; row inside it
      Acc x{make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY, -INFINITY, 0.0f};
#pragma unroll
      for (int k = 0; k < C::kGroups; ++k) {
        const int wr = (k * RT + w0) * 8 * NT + rr;
        join(x, *reinterpret_cast<const float4*>(mo + (size_t)wr * LD + d4), mr[wr], mm[wr], ml[wr]);
      }
      if (whole) {
        finish(r, d4, x);
      } else {
        *reinterpret_cast<float4*>(part + (size_t)r * D + d4) = x.o;
        if (d4 == 0) *reinterpret_cast<float4*>(part + C::kRows * D + r * 4) = make_float4(x.r, x.m, x.l, 0.0f);
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
          Acc x{make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY, -INFINITY, 0.0f};
          for (int k = c0; k <= c1; ++k) {
            const float* q = p.parts + ((size_t)k * 2 + (k == c0 ? 1 : 0)) * C::kPart;
            const float4 v = __ldcg(reinterpret_cast<const float4*>(q + (size_t)r * D + d4));
            const float4 t = __ldcg(reinterpret_cast<const float4*>(q + C::kRows * D + r * 4));
            join(x, v, t.x, t.y, t.z);
          }
          finish(r, d4, x);
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
  w->lse2 = w->parts + round_up((size_t)n_cta * 2 * w->rows * (c.head_dim + 4) * 4, 256);
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
  if (pl.rt == 1) return pl.nt == 2 ? launch_one<D, 2, 1, WT>(p, n_cta, s) : launch_one<D, 3, 1, WT>(p, n_cta, s);
  if (pl.rt == 2) return pl.nt == 2 ? launch_one<D, 2, 2, WT>(p, n_cta, s) : launch_one<D, 3, 2, WT>(p, n_cta, s);
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
  p.log2_page = a.c.page_size == 16 ? 4 : a.c.page_size == 32 ? 5 : a.c.page_size == 64 ? 6 : 7;
  const DecPlan pl = dec_plan(p.rows);
  if (a.c.head_dim == 128) return wt ? launch_plan<128, true>(p, pl, w.n_cta, s) : launch_plan<128, false>(p, pl, w.n_cta, s);
  return wt ? launch_plan<64, true>(p, pl, w.n_cta, s) : launch_plan<64, false>(p, pl, w.n_cta, s);
}

}  // namespace moe
