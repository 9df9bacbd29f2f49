// Attention of a few new tokens per sequence over the 8-bit paged cache.
//
// Bound by reading the cache once: 2 head_dim bytes per position and
// key/value head. What this asks of a kernel is many bytes in flight, few
// instructions per byte, and work cut evenly whatever the lengths are.
//
// Work. All (sequence, key/value head) pairs are laid end to end in chunks of 32
// positions; CTA c of N takes chunks [c W / N, (c + 1) W / N) of the W, its warps
// equal parts of that, so work is even whatever the lengths are and a warp meets
// no barrier on its way: one warp's change from pair to pair hides behind the
// other warps' reads. A warp writes the output of a pair that lies in its part
// whole; the (at most two) others' unnormalised output, references and sum go to
// the workspace. When its warps are done the CTA joins theirs, and what still
// reaches past the CTA is joined by the last CTA of the pair to finish (a
// counter): always in order of position, so results do not depend on who is last.
// At most one pair begins in a CTA and reaches past it, so a pair's counter is
// that of the CTA it begins in, and the counters' place does not depend on the
// sizes of a call: one workspace serves calls of all sizes in turn.
//
// A warp's next chunks are on their way into its own part of shared memory by
// cp.async. Both products run on the f16 warp MMA (m16n8k16) with positions or
// channels as its 16 rows and the query rows as its 8 columns, so up to 8 query
// rows cost one column block. E4M3 converts to f16 exactly, two codes an
// instruction (three instructions for four codes, with the move of the upper
// pair). The e4m3 warp MMA was built too and is slower: on this architecture it
// is expanded into the same conversions and f16 MMAs, and wants two terms of q
// and three of the probabilities (520 instructions a chunk at head_dim 64).
//   scores   S^T[pos][row] = K q^T: lane (g, c) takes 4 consecutive codes of a
//            16-byte piece as its k = 2c, 2c+1, 2c+8, 2c+9 of one MMA; q is
//            laid out in the same order, as f16 scaled by a power of two per
//            row that puts the row's largest in [2^11, 2^12): exact down to
//            2^-18 of that, then within 2^-37 of it.
//   output   O^T[d][row] = V^T P^T: ldmatrix transposes bytes on the way from
//            shared memory, so lane (g, c) holds 4 consecutive positions of
//            channel g, and converts them to two k pairs. S's rows are dealt so
//            that movmatrix turns its probabilities, as f16 pairs, into the B
//            operand in the same order. They are relative to the chunk's
//            largest times 2^12: 11 significant bits down to 2^-26 of it.
//   joining  a chunk's product goes into O with an fp32 factor per row that
//            holds its reference and its page's value scale. A page of 16
//            positions shares its chunk with another: the probabilities then
//            carry the difference of the scales, and their reference is the
//            largest product of both, so no page is rounded for another's sake.
// The references of O and of the sum follow the maximum only when it passes them
// by 2^30: fp32 has the range, and O is hardly ever rescaled. Scores may be of any
// size (kFar); partial results carry O's reference relative to the sum's.
//
// Measured: 32 sequences of up to 65,536, 8 heads of 64: 265 us, 6.3 TB/s. 16 of
// up to 20,011, 4 heads of 128, 20 query rows, page 16: 92 us, 2.6 TB/s: three
// tiles share each position, and the conversions, products and exponentials of
// three warps a scheduler are too few to hide one another (half of the issue
// slots are used). One sequence of 1,000: 14.6 us, of which the reads are 0.2:
// launch, one chunk a warp, join.
#include "attn.h"
#include "f32x2.cuh"
#include "fp8kv.cuh"

namespace moe {
namespace {

constexpr int kMaxSeqs = 4096;
constexpr float kRaise = 30.0f;    // log2 by which a score may pass the reference
// Beyond this a score and a value scale's exponent, or 12, do not add up exactly in
// fp32. Where a row's largest score is, the warp takes its rows' scores relative to
// a base of their own, a score that the row has, and starts the chunk anew.
constexpr float kFar = 4194304.0f;
constexpr int kChunk = 32;         // positions per warp step
constexpr int kInRing = 1 << 30;   // flag of a partial result's pair: it lies in the ring
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Workspace: counters, always this many bytes, one for each CTA; then partials,
// then (with weights) the rows' references and sums, and the scores.
constexpr size_t kCounterBytes = MOE_ATTN_DECODE_COUNTER_BYTES;
constexpr int kMaxCtas = int(kCounterBytes / 4);
struct DecWs {
  size_t parts, norm, scores, total;
  int n_cta, rows;    // CTAs; query rows padded to the row tiles
};

struct DecPlan {
  int nt, rt;         // blocks of 8 query rows per warp; row tiles
};
// A block of 8 query rows takes a warp 32 registers for the output and 16 for q at
// head_dim 128; one-block warps fit twelve to a CTA, others eight. So row tiles of
// one block, whose warps read the same positions, while they divide the twelve; at
// head_dim 64 from 33 rows on, and from 49 always, two or three blocks a warp. us
// for 16 sequences of 20,011 and of 1,000, page 16, 4 key/value heads (tiles x
// blocks):
//         head_dim 128                        head_dim 64
//   rows  chosen          other               chosen          other
//   12    2x1  65   20.7  1x2  70   26.8      2x1  50   18.5  1x2  53   20.5
//   16    2x1  68   24.7  1x2  70   26.8      2x1  49   18.6  1x2  53   20.6
//   20    3x1  91   26.8  1x3  109  39.1      3x1  66   18.6  1x3  70   26.7
//   32    4x1  117  30.9  2x2  120  37.0      4x1  85   22.7  2x2  87   24.8
//   48    6x1  165  37.2  2x3  187  53.4      2x3  111  32.9  6x1  119  26.4
//   64    4x2  213  53.4  2x4  337  73.4      4x2  154  34.8  2x4  165  43.3
inline DecPlan dec_plan(int rows, int d) {
  if (rows <= 8) return {1, 1};
  if (rows <= 16) return {1, 2};
  if (rows <= 24) return {1, 3};
  if (rows <= 32) return {1, 4};
  if (rows <= 48) return d == 128 ? DecPlan{1, 6} : DecPlan{3, 2};
  return {2, 4};
}

struct DecParams {
  DecodeArgs a;
  int G, rows;              // query heads per kv head; query rows n_new * G
  unsigned* counter;        // [CTAs]: of the pair that begins in the CTA and reaches past it
  float* parts;             // per CTA: 2 partial results, then 2 per warp: [rows][D] outputs, [rows][4] references and sum
  float2* norm;             // [n_seq * n_kv][rows padded]: reference and 1 / sum (weights)
  float* scores;            // [n_seq * n_kv][cap][rows padded] (weights)
  int64_t cap;
  int log2_page;
  uint32_t g_magic;         // r / G = r g_magic >> 16 for r < 64
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
// ... from 0
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
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
// 2^(s - 127) for a scale byte
__device__ __forceinline__ float scale_value(uint32_t s) { return __uint_as_float(s ? s << 23 : 0x00400000u); }
// Length of sequence b, cut to what table, weights and workspace hold.
__device__ __forceinline__ int dec_length(const DecodeArgs& a, int b, bool* bad) {
  const int x = __ldg(a.lengths + b);
  int64_t cap = (int64_t)a.width * a.c.page_size;
  if (a.weights && a.w_stride < cap) cap = a.w_stride;
  const int l = x < 0 ? 0 : (x > cap ? int(cap) : x);
  if (l != x) *bad = true;
  return l;
}

// A pair that this CTA joins, and the CTAs that have parts of it.
struct Edge {
  int b, h, c0, c1;
};

// D: head_dim. NT: blocks of 8 query rows per warp. RT: row tiles (warps w, w
// + 1, .. RT work on the same positions). WT: scores are kept for the weights.
template <int D, int NT, int RT, bool WT>
struct DecCfg {
  // One block of rows takes 168 registers a thread, so 12 warps; more blocks
  // take up to 255. The stages of all warps fill shared memory.
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = 24 / kWarps * (D == 128 ? 1 : 2);
  static constexpr int kGroups = kWarps / RT;            // warps with a part of their own
  static constexpr int kRows = 8 * NT * RT;              // padded query rows
  static constexpr uint32_t kKBytes = kChunk * D;
  static constexpr uint32_t kStageBytes = 2 * kKBytes;   // values as they come, 16-byte pieces exchanged within 128 bytes
  static constexpr uint32_t kRing = kWarps * kStages * kStageBytes;
  static_assert(8 * NT * (D + 4) * 4 <= kStages * kStageBytes, "a warp's results fit its part of the ring");
  static constexpr uint32_t kSmem = kRing + (2 * kMaxSeqs + 1) * 4;   // ring, prefix sums, lengths
  static_assert(kSmem + 1024 <= 232448, "shared memory");
  static constexpr int kPartW = 8 * NT * (D + 4);        // floats of a warp's partial result
  static constexpr int kPart = kRows * (D + 4);          // and of a CTA's
  static constexpr int kPartsCta = 2 * kPart + 2 * kWarps * kPartW;
};

template <int D, int NT, int RT, bool WT>
__global__ void __launch_bounds__(DecCfg<D, NT, RT, WT>::kThreads, 1) decode_attn_kernel(const DecParams p) {
  using C = DecCfg<D, NT, RT, WT>;
  constexpr int KS = D / 16;      // MMA steps over the channels
  constexpr int MT = D / 16;      // 16-channel blocks of the output
  constexpr int KC = D / 64;      // 16-byte pieces per lane and position
  extern __shared__ __align__(1024) uint8_t smem[];
  int* prefix = reinterpret_cast<int*>(smem + C::kRing);
  int* lens = prefix + kMaxSeqs + 1;
  constexpr int kDecWarps = C::kWarps, kDecThreads = C::kThreads;
  __shared__ int s_scan[kDecWarps];
  __shared__ Edge s_edge[2];
  __shared__ float s_base[kDecWarps][8 * NT];   // see kFar
  __shared__ int s_pair[2 * C::kGroups];   // pairs of the warps' partial results, -1: none
  const DecodeArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int H = a.c.n_kv_heads, P = a.c.page_size, B = a.n_seq, T = a.n_new;

  // chunks of the sequences before each one (per kv head)
  {
    bool bad = false;
    int before = 0;
    for (int b0 = 0; b0 < B; b0 += kDecThreads) {
      const int b = b0 + tid;
      int n = 0;
      if (b < B) {
        const int L = dec_length(a, b, &bad);
        lens[b] = L;
        n = L > 0 ? (L + kChunk - 1) / kChunk : 1;
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
  const int64_t W = (int64_t)prefix[B] * H;
  const int64_t N = min((int64_t)gridDim.x, (W + C::kGroups - 1) / C::kGroups);   // no warp idles while others have two
  if (blockIdx.x >= N) return;
  const int64_t cta0 = blockIdx.x * W / N, cta1 = (blockIdx.x + 1) * W / N;
  float* cta_parts = p.parts + (size_t)blockIdx.x * C::kPartsCta;

  const int rt = warp % RT, tg = warp / RT;
  int64_t pos = cta0 + tg * (cta1 - cta0) / C::kGroups;
  const int64_t end = cta0 + (tg + 1) * (cta1 - cta0) / C::kGroups;
  uint8_t* ring = smem + (size_t)warp * C::kStages * C::kStageBytes;
  const uint32_t ring_s = smem_addr(ring);
  if (rt == 0 && lane < 2) s_pair[2 * tg + lane] = -1;
  __syncwarp();

  // sequence of a chunk: the last b with prefix[b] H <= x
  auto seq_of = [&](int64_t x) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)prefix[mid] * H <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  // (O, its reference relative to m, m, sum) of 4 channels of a row, + another's
  struct Acc {
    float4 o;
    float r, m, l;
  };
  auto join = [](Acc& x, float4 v, float r, float mw, float lw) {
    if (mw == -INFINITY && lw == 0.0f) return;   // saw nothing
    const float M = fmaxf(x.m, mw);
    const float dx = x.m == M ? 0.0f : x.m - M, dw = mw == M ? 0.0f : mw - M;
    x.m = M;
    x.l = x.l * ex2(dx) + lw * ex2(dw);
    x.r += dx;
    r += dw;
    if (r > -INFINITY) {
      const float R = fmaxf(x.r, r);
      const float f0 = x.r == R ? 1.0f : ex2(x.r - R), f1 = r == R ? 1.0f : ex2(r - R);
      x.r = R;
      x.o.x = x.o.x * f0 + v.x * f1;
      x.o.y = x.o.y * f0 + v.y * f1;
      x.o.z = x.o.z * f0 + v.z * f1;
      x.o.w = x.o.w * f0 + v.w * f1;
    }
  };
  auto tok_of = [&](int r) { return int(uint32_t(r) * p.g_magic >> 16); };   // new token of a query row
  // What O is multiplied with for the output, 2^r / l, as two factors, x first: r
  // holds a value scale of 2^-127 to 2^127 and may lie 30 from the maximum as m
  // may, so 2^r can leave fp32's range where the output does not.
  auto out_factor = [](float r, float l) {
    if (l == 0.0f) return make_float2(0.0f, 0.0f);             // nothing seen: zeros
    if (r == -INFINITY) return make_float2(l, 1.0f);           // a row of NaN scores: NaN
    const float f = ex2(0.5f * r);
    return make_float2(f / l, f);
  };
  auto write_lse = [&](int b, int h, int r, int64_t row, float m, float l) {
    const float m0 = m == -INFINITY ? 0.0f : m;   // nothing seen, or NaN scores
    if (a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (m0 + log2f(l)) * kLn2;
    if (WT) p.norm[((int64_t)b * H + h) * C::kRows + r] = make_float2(m0, l == 0.0f ? 0.0f : 1.0f / l);
  };
  auto finish = [&](int b, int h, int r, int d4, const Acc& x) {
    const int tok = tok_of(r);
    const int64_t row = ((int64_t)b * T + tok) * a.n_heads + h * p.G + r - tok * p.G;
    const float2 f = out_factor(x.r, x.l);
    const __nv_bfloat162 y0 = __floats2bfloat162_rn(x.o.x * f.x * f.y, x.o.y * f.x * f.y);
    const __nv_bfloat162 y1 = __floats2bfloat162_rn(x.o.z * f.x * f.y, x.o.w * f.x * f.y);
    uint2 y;
    y.x = *reinterpret_cast<const uint32_t*>(&y0);
    y.y = *reinterpret_cast<const uint32_t*>(&y1);
    *reinterpret_cast<uint2*>(a.out + row * D + d4) = y;
    if (d4 == 0) write_lse(b, h, r, row, x.m, x.l);
  };

  // ---- this warp's chunks: fetched as one sequence, whatever pairs they belong to
  const int n_my = int(end - pos);
  // A chunk's halves A and B (16 positions each) are 16-row groups of the code
  // arrays: group * 16 D bytes in; kNone past the sequence's end or where there
  // is no page. Lane l looks up the l-th chunk of a block of 32, half a block
  // ahead and in steps, so that no load is waited for.
  constexpr uint32_t kNone = 0xFFFFFFFFu;
  uint32_t grp_a = kNone, grp_b = kNone;                    // of the block being fetched
  uint32_t sc = 0, no_a = 0, no_b = 0;                      // of the block in work: bytes kA kB vA vB; halves that are none
  int nx_a = -1, nx_b = -1;                                 // next block: pages, then groups
  uint32_t nx_h = 0, nx_slot = 0, nx_sc[4] = {0, 0, 0, 0};
  const uint32_t gpp = P / 16;                              // groups per page and head
  auto look_pages = [&](int i0) {
    nx_a = nx_b = -2;                                       // nothing there, and nothing wrong
    if (i0 + lane < n_my) {
      const int64_t x = pos + i0 + lane;
      const int b = seq_of(x), nu = prefix[b + 1] - prefix[b];
      const int64_t rel = x - (int64_t)prefix[b] * H;
      const int h = rel <= 0x7FFFFFFF ? int(rel) / nu : int(rel / nu);
      const int t = int(rel - (int64_t)h * nu) * kChunk;
      const int L = lens[b];
      const int32_t* tab = a.table + (size_t)b * a.width + (t >> p.log2_page);
      if (t < L) nx_a = max(__ldg(tab), -1);
      if (t + 16 < L) nx_b = P == 16 ? max(__ldg(tab + 1), -1) : nx_a;
      nx_h = h;
      nx_slot = uint32_t(t & (P - 1)) >> 4;
    }
  };
  auto look_scales = [&]() {
    const bool bad = nx_a == -1 || nx_b == -1 || nx_a >= a.c.n_pages || nx_b >= a.c.n_pages;
    if (bad && a.status) atomicOr(a.status, MOE_DEV_INDEX_OOB);
    const uint32_t ra = uint32_t(nx_a) * H + nx_h, rb = uint32_t(nx_b) * H + nx_h;
    const bool in_a = nx_a >= 0 && nx_a < a.c.n_pages, in_b = nx_b >= 0 && nx_b < a.c.n_pages;
    if (in_a) {
      nx_sc[0] = __ldg(a.c.k_scales + ra);
      nx_sc[2] = __ldg(a.c.v_scales + ra);
    }
    if (in_b) {
      nx_sc[1] = __ldg(a.c.k_scales + rb);
      nx_sc[3] = __ldg(a.c.v_scales + rb);
    }
    nx_a = in_a ? int(ra * gpp + nx_slot) : -1;
    nx_b = in_b ? int(rb * gpp + (P == 16 ? 0 : nx_slot + 1)) : -1;
  };
  auto issue = [&](int i) {
    switch (i & 31) {
      case 0:
        grp_a = uint32_t(nx_a);
        grp_b = uint32_t(nx_b);
        break;
      case 8: look_pages((i & ~31) + 32); break;
      case 20: look_scales(); break;
    }
    const uint32_t ga = __shfl_sync(0xFFFFFFFFu, grp_a, i & 31), gb = __shfl_sync(0xFFFFFFFFu, grp_b, i & 31);
    if (i < n_my) {
      // Keys: lane (g, c) what it will use, at its own 16 bytes of each row of
      // 512. Values: 512 consecutive bytes at a time, the 16-byte pieces of each
      // 128 permuted so that 8 positions' pieces of the same channels lie in
      // different banks (a permutation over more than 128 bytes would cut the
      // L2 requests into 16-byte ones: measured, 1.5 times the traffic into the
      // SM and 0.75 of the rate).
      const uint32_t st = ring_s + (i % C::kStages) * C::kStageBytes;
      const uint32_t kd = st + lane * 16;
      const uint32_t vd = st + C::kKBytes + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
      const uint8_t* kl = static_cast<const uint8_t*>(a.c.k_codes) + (4 * (g >> 1) + (g & 1)) * D + c * 16;
      const uint8_t* vl = static_cast<const uint8_t*>(a.c.v_codes) + lane * 16;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t gr = half ? gb : ga;
        if (gr == kNone) continue;
        const uint8_t* ks = kl + (size_t)gr * (16 * D);
        const uint8_t* vs = vl + (size_t)gr * (16 * D);
#pragma unroll
        for (int o = 0; o < 2; ++o)
#pragma unroll
          for (int j = 0; j < KC; ++j) cp_async16(kd + ((2 * half + o) * KC + j) * 512, ks + 2 * o * D + 64 * j);
#pragma unroll
        for (int n = 0; n < D / 32; ++n) {
          const int k = half * (D / 32) + n;   // the odd ones: positions 4 .. 7 of 8
          cp_async16((k & 1 ? vd ^ 64 : vd) + k * 512, vs + n * 512);
        }
      }
    }
    cp_async_commit();
  };
  // The block in work follows the one being fetched by less than 32 chunks.
  auto enter_block = [&]() {
    no_a = __ballot_sync(0xFFFFFFFFu, grp_a == kNone);
    no_b = __ballot_sync(0xFFFFFFFFu, grp_b == kNone);
    const bool b_too = grp_b != kNone;   // else A's, so that the halves' scales are equal
    sc = nx_sc[0] | nx_sc[b_too ? 1 : 0] << 8 | nx_sc[2] << 16 | nx_sc[b_too ? 3 : 2] << 24;
  };

  // a pair's query rows: lane (g, c) the channels 64 j + 16 c + [0, 16) of row g of each block
  uint4 qw[NT][2 * KC];
  auto load_q = [&](int x) {
    const int b = seq_of(pos + x), nu = prefix[b + 1] - prefix[b];
    const int64_t rel = pos + x - (int64_t)prefix[b] * H;
    const int h = rel <= 0x7FFFFFFF ? int(rel) / nu : int(rel / nu);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = (rt * NT + n) * 8 + g;
      const int tok = tok_of(r);
      const __nv_bfloat16* q = a.q + ((int64_t)b * T + tok) * a.q_ts + (int64_t)(h * p.G + r - tok * p.G) * a.q_hs;
#pragma unroll
      for (int j = 0; j < 2 * KC; ++j)
        qw[n][j] = r < p.rows ? *reinterpret_cast<const uint4*>(q + 64 * (j >> 1) + 16 * c + 8 * (j & 1))
                              : make_uint4(0, 0, 0, 0);
    }
  };

  if (n_my > 0) {
    look_pages(0);
    load_q(0);
    look_scales();
  }
#pragma unroll 1
  for (int j = 0; j < C::kStages - 1; ++j) issue(j);

  int i = 0;
  while (i < n_my) {
    // ---- a pair, or the part of it that is this warp's
    const int b = seq_of(pos + i), nu = prefix[b + 1] - prefix[b];
    const int64_t rel = pos + i - (int64_t)prefix[b] * H;
    const int h = rel <= 0x7FFFFFFF ? int(rel) / nu : int(rel / nu);
    const int u0 = int(rel - (int64_t)h * nu), u1 = min(nu, u0 + (n_my - i));
    const int i1 = i + (u1 - u0);
    const int tbase = (u0 - i) * kChunk;     // chunk i's first position - 32 i
    const int L = lens[b];

    // query rows -> B fragments and the factors that undo their scale
    uint32_t qf[KS][NT][2];
    float qs[NT][2];         // of rows 2c, 2c+1 of each block: 2^e scale log2(e)
    int vis[NT][2];          // positions that those rows see
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[KC * 16];
      uint32_t top = 0;      // the row's largest magnitude, as bf16 bits
#pragma unroll
      for (int j = 0; j < 2 * KC; ++j) {
        const uint32_t w[4] = {qw[n][j].x, qw[n][j].y, qw[n][j].z, qw[n][j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          top = max(top, max(w[i] & 0x7FFFu, w[i] >> 16 & 0x7FFFu));
          x[8 * j + 2 * i] = bf16_lo(w[i]);
          x[8 * j + 2 * i + 1] = bf16_hi(w[i]);
        }
      }
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
      // 2^-e puts the largest in [2^11, 2^12); in two factors, since it may leave fp32's range. A row with inf or NaN
      // keeps them.
      const int e = top >= 0x7F80u ? 0 : max(int(top >> 7), 1) - 138, eh = e / 2;
      const float f0 = pow2(-eh), f1 = pow2(eh - e);
#pragma unroll
      for (int i = 0; i < KC * 16; i += 2)
        qf[i / 4][n][(i / 2) & 1] = f16x2_bits(x[i] * f0 * f1, x[i + 1] * f0 * f1);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int er = __shfl_sync(0xFFFFFFFFu, e, (2 * c + j) * 4);
        const int rr = (rt * NT + n) * 8 + 2 * c + j;
        qs[n][j] = a.scale * kLog2e * pow2(er / 2) * pow2(er - er / 2);
        vis[n][j] = rr < p.rows ? L - T + tok_of(rr) + 1 : 0;
      }
    }

    // O (in units of 2^ro), the sum (of 2^m). `far`: relative to the row's s_base
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
    bool far = false;

#pragma unroll 1
    for (; i < i1; ++i) {
      issue(i + C::kStages - 1);
      if ((i & 31) == 0) enter_block();
      cp_async_wait<C::kStages - 1>();
      __syncwarp();
      const uint32_t w = __shfl_sync(0xFFFFFFFFu, sc, i & 31);
      const int t0 = tbase + i * kChunk;
      const int va = int(w >> 16 & 0xFFu), vb = int(w >> 24);
      const bool none_a = no_a >> (i & 31) & 1u, none_b = no_b >> (i & 31) & 1u;
      const uint32_t st = (i % C::kStages) * C::kStageBytes;
      const uint4* kst = reinterpret_cast<const uint4*>(ring + st) + lane;
      const bool full = !none_a && !none_b && t0 + kChunk <= L - T + 1;   // every row sees every position

      // scores: s[mt][n][x] is position t0 + 16 mt + 4 (g / 2) + g % 2 + 2 (x / 2), row 2c + x % 2
      float s[2][NT][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          const uint4 x = kst[(mt * 2 * KC + j) * 32], y = kst[((mt * 2 + 1) * KC + j) * 32];
          const uint32_t wx[4] = {x.x, x.y, x.z, x.w}, wy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a0 = e4m3x2_f16x2(wx[k]), a1 = e4m3x2_f16x2(wy[k]);
            const uint32_t a2 = e4m3x2_f16x2_hi(wx[k]), a3 = e4m3x2_f16x2_hi(wy[k]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t b0 = qf[4 * j + k][n][0], b1 = qf[4 * j + k][n][1];
              if (j == 0 && k == 0)
                mma_f16_zero(s[mt][n], a0, a1, a2, a3, b0, b1);
              else
                mma_f16(s[mt][n], a0, a1, a2, a3, b0, b1);
            }
          }
        }

      uint32_t pf[NT][4];         // probabilities: B fragments of the two halves
      float beta[NT][2];
      const float kfa = scale_value(w & 0xFFu), kfb = scale_value(w >> 8 & 0xFFu);
      const float vfa = float(va - 127), vfb = float(vb - 127);
      const int p0 = t0 + 4 * (g >> 1) + (g & 1);
      // the chunk's largest score, and largest score times value scale
      auto largest = [&](int n, float (&us)[2], float (&ms)[2]) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float xa = fmaxf(s[0][n][j], s[0][n][j + 2]), xb = fmaxf(s[1][n][j], s[1][n][j + 2]);
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
      };
      // `far`: a row's scores relative to its base, which follows the largest
      auto rebase = [&](int n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = fmaxf(fmaxf(s[0][n][j], s[0][n][j + 2]), fmaxf(s[1][n][j], s[1][n][j + 2]));
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, k));
          float base = s_base[warp][n * 8 + 2 * c + j];
          __syncwarp();
          if (x > base + kRaise || (m[n][j] == -INFINITY && x > -INFINITY)) {
            m[n][j] += base - x;
            ro[n][j] += base - x;
            s_base[warp][n * 8 + 2 * c + j] = base = x;
          }
#pragma unroll
          for (int k = j; k < 4; k += 2) s[0][n][k] -= base, s[1][n][k] -= base;
        }
        __syncwarp();
      };
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const uint64_t f2 = mul2(pack2(qs[n][0], qs[n][1]), pack2(mt ? kfb : kfa, mt ? kfb : kfa));
#pragma unroll
            for (int x = 0; x < 4; x += 2)
              unpack2(mul2(pack2(s[mt][n][x], s[mt][n][x + 1]), f2), s[mt][n][x], s[mt][n][x + 1]);
          }
          if (!full) {
            asm volatile("" ::: "memory");   // a branch, not selects in every chunk
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if ((mt ? none_b : none_a) || p0 + 16 * mt + 2 * (x >> 1) >= vis[n][x & 1]) s[mt][n][x] = -INFINITY;
          }
          if (WT) {
            float* sp = p.scores + (((int64_t)b * H + h) * p.cap + p0) * C::kRows + (rt * NT + n) * 8 + 2 * c;
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int x = 0; x < 2; ++x)
                if (p0 + 16 * mt + 2 * x < L)
                  *reinterpret_cast<float2*>(sp + (16 * mt + 2 * x) * C::kRows) =
                      make_float2(s[mt][n][2 * x], s[mt][n][2 * x + 1]);
          }
          if (far) rebase(n);
          float us[2], ms[2];
          largest(n, us, ms);
          const bool raise = ms[0] > m[n][0] + kRaise || ms[1] > m[n][1] + kRaise || us[0] > ro[n][0] + kRaise ||
                             us[1] > ro[n][1] + kRaise;
          if (__any_sync(0xFFFFFFFFu, raise)) {
            const bool out_there = (fabsf(ms[0]) > kFar && ms[0] > -INFINITY) || (fabsf(ms[1]) > kFar && ms[1] > -INFINITY);
            if (!far && __any_sync(0xFFFFFFFFu, out_there)) {
              far = true;
#pragma unroll
              for (int k = 0; k < NT; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float base = m[k][j] == -INFINITY ? 0.0f : m[k][j];
                  s_base[warp][k * 8 + 2 * c + j] = base;
                  m[k][j] -= base;
                  ro[k][j] -= base;
                }
              __syncwarp();
              rebase(n);   // the blocks after this one come to it in their turn
              largest(n, us, ms);
            }
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
          // probabilities times 2^12 over the chunk's largest
          float pr[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // nothing seen, NaN scores only, or all so far below the reference (which is above
            // -kFar) that they count for nothing and would not add up with the 12
            const bool none = !(us[j] > -2.0f * kFar);
            const float ref = none ? -INFINITY : 12.0f - us[j];
            beta[n][j] = none ? 0.0f : ex2(us[j] - 12.0f - ro[n][j]);
#pragma unroll
            for (int x = j; x < 4; x += 2) {
              pr[0][x] = ex2(s[0][n][x] + (vfa + ref));
              pr[1][x] = ex2(s[1][n][x] + (vfb + ref));
            }
            if (va == vb) {
              const float sum = (pr[0][j] + pr[0][j + 2]) + (pr[1][j] + pr[1][j + 2]);
              // a row of NaN scores has no largest one, but must not pass for empty
              l[n][j] += none ? sum : sum * ex2(us[j] - 12.0f - vfa - m[n][j]);
            } else {
              const float mr = m[n][j] == -INFINITY ? 0.0f : m[n][j];
              l[n][j] += (ex2(s[0][n][j] - mr) + ex2(s[0][n][j + 2] - mr)) + (ex2(s[1][n][j] - mr) + ex2(s[1][n][j + 2] - mr));
            }
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            pf[n][2 * mt] = movm(f16x2_bits(pr[mt][0], pr[mt][1]));
            pf[n][2 * mt + 1] = movm(f16x2_bits(pr[mt][2], pr[mt][3]));
          }
        }
      }

      // output
      // piece 0 of position `lane`; piece t is at this address ^ 16 t
      const int line = D == 128 ? lane : lane >> 1;
      const uint32_t va_s = ring_s + st + C::kKBytes + line * 128 +
                            (((D == 128 ? 0 : (lane & 1) << 2) ^ (line & 7)) << 4);
      if (full) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          uint32_t x[4];
          ldm_trans8(x, va_s ^ (t << 4));
          // tokens 4c, 4c+1 and 4c+2, 4c+3 of each half: an MMA's two k pairs
          const uint32_t a0 = e4m3x2_f16x2(x[0]), a1 = e4m3x2_f16x2(x[1]), a2 = e4m3x2_f16x2_hi(x[0]),
                         a3 = e4m3x2_f16x2_hi(x[1]);
          const uint32_t e0 = e4m3x2_f16x2(x[2]), e1 = e4m3x2_f16x2(x[3]), e2 = e4m3x2_f16x2_hi(x[2]),
                         e3 = e4m3x2_f16x2_hi(x[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float d[4];
            mma_f16_zero(d, a0, a1, a2, a3, pf[n][0], pf[n][1]);
            mma_f16(d, e0, e1, e2, e3, pf[n][2], pf[n][3]);
            const uint64_t b2 = pack2(beta[n][0], beta[n][1]);
#pragma unroll
            for (int j = 0; j < 4; j += 2)
              unpack2(fma2(pack2(d[j], d[j + 1]), b2, pack2(o[t][n][j], o[t][n][j + 1])), o[t][n][j], o[t][n][j + 1]);
          }
        }
      } else {
        // Positions past the end, and halves without a page, hold anything:
        // their codes are zeroed. Where a NaN is visible to some tokens only (0
        // * NaN is NaN) every token takes a pass over what it sees.
        auto keep4 = [&](int first_pos, int seen) {   // bytes of 4 consecutive positions
          const int k = seen - first_pos;
          return k >= 4 ? 0xFFFFFFFFu : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
        };
        bool poison = false;
        if (T > 1) {
          const uint32_t ka = none_a ? 0u : keep4(t0 + 4 * c, L), kb = none_b ? 0u : keep4(t0 + 16 + 4 * c, L);
#pragma unroll 1
          for (int t = 0; t < MT; ++t) {
            uint32_t x[4];
            ldm_trans8(x, va_s ^ (t << 4));
            poison |= any_nan4(x[0] & ka) || any_nan4(x[1] & ka) || any_nan4(x[2] & kb) || any_nan4(x[3] & kb);
          }
          poison = __any_sync(0xFFFFFFFFu, poison);
        }
        const int n_pass = poison ? T : 1;
#pragma unroll 1
        for (int pass = 0; pass < n_pass; ++pass) {
          const int seen = poison ? L - T + pass + 1 : L;
          const uint32_t ka = none_a ? 0u : keep4(t0 + 4 * c, seen), kb = none_b ? 0u : keep4(t0 + 16 + 4 * c, seen);
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            uint32_t x[4];
            ldm_trans8(x, va_s ^ (t << 4));
            x[0] &= ka;
            x[1] &= ka;
            x[2] &= kb;
            x[3] &= kb;
            const uint32_t a0 = e4m3x2_f16x2(x[0]), a1 = e4m3x2_f16x2(x[1]), a2 = e4m3x2_f16x2_hi(x[0]),
                           a3 = e4m3x2_f16x2_hi(x[1]);
            const uint32_t e0 = e4m3x2_f16x2(x[2]), e1 = e4m3x2_f16x2(x[3]), e2 = e4m3x2_f16x2_hi(x[2]),
                           e3 = e4m3x2_f16x2_hi(x[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float d[4];
              mma_f16_zero(d, a0, a1, a2, a3, pf[n][0], pf[n][1]);
              mma_f16(d, e0, e1, e2, e3, pf[n][2], pf[n][3]);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (!poison || vis[n][j & 1] == seen) o[t][n][j] = fmaf(d[j], beta[n][j & 1], o[t][n][j]);
            }
          }
        }
      }
      __syncwarp();   // every lane has read the stage before it is filled again
    }
    if (i1 < n_my) load_q(i1);

    // ---- results
    const bool whole = u0 == 0 && u1 == nu;
    const int slot = u0 > 0 ? 0 : 1;   // continues an earlier warp's part, or begins the pair
    // the warp's last ones through its part of the ring, which is done with
    const bool last_one = i1 == n_my;
    float* part = last_one ? reinterpret_cast<float*>(ring) : cta_parts + 2 * C::kPart + (2 * warp + slot) * C::kPartW;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float sum = l[n][j];
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
        const int lr = n * 8 + 2 * c + j, r = rt * 8 * NT + lr;
        // the sum's reference as a number of its own, O's relative to that
        float mm = m[n][j], rr = ro[n][j];
        if (mm > -INFINITY) {
          if (far) {
            sum *= ex2(mm);
            mm = s_base[warp][lr];
          } else {
            rr -= mm;
          }
        }
        if (!whole) {
          // 8 lanes write 8 consecutive channels
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            part[lr * D + 16 * t + g] = o[t][n][j];
            part[lr * D + 16 * t + g + 8] = o[t][n][j + 2];
          }
          if (g == 0)
            *reinterpret_cast<float4*>(part + 8 * NT * D + lr * 4) = make_float4(rr, mm, sum, 0.0f);
        } else {
          const bool have = r < p.rows;
          const int tok = tok_of(r);
          const int64_t row = ((int64_t)b * T + tok) * a.n_heads + h * p.G + r - tok * p.G;
          const float2 f = out_factor(rr, sum);
          // lanes g and g ^ 1 swap, so that each holds two neighbouring channels
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const float give = g & 1 ? o[t][n][j] : o[t][n][j + 2];
            const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 4);
            const float keep = g & 1 ? o[t][n][j + 2] : o[t][n][j];
            const float y0 = (g & 1 ? got : keep) * f.x * f.y, y1 = (g & 1 ? keep : got) * f.x * f.y;
            const __nv_bfloat162 y = __floats2bfloat162_rn(y0, y1);
            if (have) *reinterpret_cast<__nv_bfloat162*>(a.out + row * D + 16 * t + (g & 1 ? g + 7 : g)) = y;
          }
          if (have && g == 0) write_lse(b, h, r, row, mm, sum);
        }
      }
    if (!whole && rt == 0 && lane == 0) s_pair[2 * tg + slot] = (b * H + h) | (last_one ? kInRing : 0);
  }
  cp_async_wait<0>();
  __syncthreads();

  // the warps' partial results, in order of position
  const unsigned have = __ballot_sync(0xFFFFFFFFu, lane < 2 * C::kGroups && s_pair[lane < 2 * C::kGroups ? lane : 0] >= 0);
  for (int i = tid; i < C::kRows * (D / 4) && have; i += kDecThreads) {
    const int r = i / (D / 4), d4 = (i % (D / 4)) * 4;
    if (r >= p.rows) continue;
    const int w0 = r / (8 * NT), rr = r % (8 * NT);   // row tile; row inside it
    int cur = -1;
    Acc x;
    auto flush = [&]() {
      if (cur < 0) return;
      const int b = cur / H, h = cur % H, nu = prefix[b + 1] - prefix[b];
      const int64_t s0 = (int64_t)prefix[b] * H + (int64_t)h * nu;
      if (s0 >= cta0 && s0 + nu <= cta1) {
        finish(b, h, r, d4, x);
      } else {
        float* q = cta_parts + (s0 < cta0 ? 0 : C::kPart);
        *reinterpret_cast<float4*>(q + r * D + d4) = x.o;
        if (d4 == 0) *reinterpret_cast<float4*>(q + C::kRows * D + r * 4) = make_float4(x.r, x.m, x.l, 0.0f);
      }
    };
#pragma unroll 1
    for (unsigned left = have; left; left &= left - 1) {
      const int slot = __ffs(left) - 1, pair = s_pair[slot] & ~kInRing, from = (slot >> 1) * RT + w0;
      const float* q = s_pair[slot] & kInRing
                           ? reinterpret_cast<const float*>(smem + (size_t)from * C::kStages * C::kStageBytes)
                           : cta_parts + 2 * C::kPart + (2 * from + (slot & 1)) * C::kPartW;
      const float4 v = *reinterpret_cast<const float4*>(q + rr * D + d4);
      const float4 t = *reinterpret_cast<const float4*>(q + 8 * NT * D + rr * 4);
      if (pair != cur) {
        flush();
        cur = pair;
        x = Acc{make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY, -INFINITY, 0.0f};
      }
      join(x, v, t.x, t.y, t.z);
    }
    flush();
  }

  // Pairs that reach past this CTA: the one of its first chunk, and that of its
  // last where it is another. CTAs c0 .. c1 have chunks of the pair.
  __threadfence();
  __syncthreads();
  if (tid < 2) {
    const int64_t at = tid ? cta1 - 1 : cta0;
    const int b = seq_of(at), nu = prefix[b + 1] - prefix[b];
    const int64_t pair0 = (int64_t)prefix[b] * H;
    const int h = int((at - pair0) / nu);
    const int64_t s0 = pair0 + (int64_t)h * nu, s1 = s0 + nu;
    Edge e{-1, 0, 0, 0};
    if ((s0 < cta0 || s1 > cta1) && !(tid && s0 <= cta0)) {
      const int c0 = int(((s0 + 1) * N - 1) / W), c1 = int((s1 * N - 1) / W);
      if (atomicAdd(p.counter + c0, 1u) == unsigned(c1 - c0)) {   // the last of them
        p.counter[c0] = 0;
        e = Edge{b, h, c0, c1};
      }
    }
    s_edge[tid] = e;
  }
  __syncthreads();
#pragma unroll 1
  for (int k2 = 0; k2 < 2; ++k2) {
    const Edge e = s_edge[k2];
    if (e.b < 0) continue;
    __threadfence();
    for (int i = tid; i < C::kRows * (D / 4); i += kDecThreads) {
      const int r = i / (D / 4), d4 = (i % (D / 4)) * 4;
      if (r >= p.rows) continue;
      Acc x{make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY, -INFINITY, 0.0f};
      constexpr int KB = 4;   // loads in flight
#pragma unroll 1
      for (int k0 = e.c0; k0 <= e.c1; k0 += KB) {
        float4 v[KB], t[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          const int kc = min(k0 + k, e.c1);
          const float* q = p.parts + (size_t)kc * C::kPartsCta + (kc == e.c0 ? C::kPart : 0);
          v[k] = __ldcg(reinterpret_cast<const float4*>(q + r * D + d4));
          t[k] = __ldcg(reinterpret_cast<const float4*>(q + C::kRows * D + r * 4));
        }
#pragma unroll
        for (int k = 0; k < KB; ++k)
          if (k0 + k <= e.c1) join(x, v[k], t[k].x, t[k].y, t[k].z);
      }
      finish(e.b, e.h, r, d4, x);
    }
  }
}

// weights[pair][j] += sum over the query rows of 2^(score - reference) / sum (not
// of 2^(score - log-sum-exp): in a large one the sum's logarithm is rounded away).
// Bound by reading the scores back, mostly from L2.
template <int ROWS>
__global__ void __launch_bounds__(256) decode_weights_kernel(const DecParams p) {
  const DecodeArgs& a = p.a;
  const int b = blockIdx.z, h = blockIdx.y;
  const int64_t pair = (int64_t)b * a.c.n_kv_heads + h;
  bool ignore = false;
  const int L = dec_length(a, b, &ignore);
  __shared__ float2 s_norm[ROWS];
  for (int r = threadIdx.x; r < ROWS; r += blockDim.x)
    s_norm[r] = r < p.rows ? p.norm[pair * ROWS + r] : make_float2(0.0f, 0.0f);
  __syncthreads();
  // 4 positions per thread and turn, each 4 rows at a time: the loads of all at once
  constexpr int PT = 4;
  for (int64_t j0 = (int64_t)blockIdx.x * 256 * PT; j0 < L; j0 += (int64_t)gridDim.x * 256 * PT) {
    float w[PT], old[PT];
    float* out = a.weights + pair * a.w_stride + j0 + threadIdx.x;
#pragma unroll
    for (int k = 0; k < PT; ++k) {
      w[k] = 0.0f;
      old[k] = j0 + threadIdx.x + 256 * k < L ? out[256 * k] : 0.0f;
    }
#pragma unroll
    for (int r4 = 0; r4 < ROWS / 4; ++r4) {
      float4 v[PT];
#pragma unroll
      for (int k = 0; k < PT; ++k) {
        const int64_t j = j0 + threadIdx.x + 256 * k;
        v[k] = j < L ? __ldcs(reinterpret_cast<const float4*>(p.scores + (pair * p.cap + j) * ROWS) + r4)
                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int k = 0; k < PT; ++k) {
        const float x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // rows that are padding have a factor of 0; rows that see nothing have scores of -inf
          const float2 f = s_norm[4 * r4 + i];
          if (x[i] != -INFINITY) w[k] = fmaf(ex2(x[i] - f.x), f.y, w[k]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < PT; ++k)
      if (j0 + threadIdx.x + 256 * k < L) out[256 * k] = old[k] + w[k];
  }
}

// CTAs that can have work, and the workspace's parts. Mirrors DecCfg.
size_t ws_layout(const moe_kv_cache& c, int n_seq, int n_new, int n_heads, int width, bool weights, int sm_count, DecWs* w) {
  const int rows = n_new * (n_heads / c.n_kv_heads);
  const DecPlan pl = dec_plan(rows, c.head_dim);
  const int warps = pl.nt == 1 ? 12 : 8, groups = warps / pl.rt;
  w->rows = 8 * pl.nt * pl.rt;
  const size_t pairs = (size_t)n_seq * c.n_kv_heads;
  const size_t cap = (size_t)width * c.page_size;
  const size_t chunks = pairs * (cap > 0 ? (cap + kChunk - 1) / kChunk : 1);
  const size_t ctas = (chunks + groups - 1) / groups;
  const size_t most = sm_count < kMaxCtas ? sm_count : kMaxCtas;
  w->n_cta = int(ctas < most ? (ctas ? ctas : 1) : most);
  const size_t part = (size_t)(c.head_dim + 4) * 4 * (2 * w->rows + 2 * warps * 8 * pl.nt);
  w->parts = kCounterBytes;
  w->norm = w->parts + round_up(w->n_cta * part, 256);
  w->scores = w->norm + (weights ? round_up(pairs * w->rows * 8, 256) : 0);
  w->total = w->scores + (weights ? pairs * cap * w->rows * 4 : 0);
  return w->total;
}

template <int D, int NT, int RT, bool WT>
int launch_one(const DecParams& p, int n_cta, cudaStream_t s) {
  using C = DecCfg<D, NT, RT, WT>;
  MOE_CUDA_TRY(cudaFuncSetAttribute(decode_attn_kernel<D, NT, RT, WT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(C::kSmem)));
  decode_attn_kernel<D, NT, RT, WT><<<n_cta, C::kThreads, C::kSmem, s>>>(p);
  int st = launch_status();
  if (st != MOE_OK || !WT) return st;
  if (p.cap == 0) return MOE_OK;
  const int64_t blocks = (p.cap + 1023) / 1024;
  const dim3 grid(unsigned(blocks < 64 ? blocks : 64), p.a.c.n_kv_heads, p.a.n_seq);
  decode_weights_kernel<C::kRows><<<grid, 256, 0, s>>>(p);
  return launch_status();
}
template <int D, bool WT>
int launch_plan(const DecParams& p, const DecPlan& pl, int n_cta, cudaStream_t s) {
  if (pl.nt == 1 && pl.rt == 3) return launch_one<D, 1, 3, WT>(p, n_cta, s);
  if (pl.nt == 1 && pl.rt == 4) return launch_one<D, 1, 4, WT>(p, n_cta, s);
  if (pl.nt == 1 && pl.rt == 2) return launch_one<D, 1, 2, WT>(p, n_cta, s);
  if (pl.nt == 1 && pl.rt == 1) return launch_one<D, 1, 1, WT>(p, n_cta, s);
  if (pl.rt != 4) return launch_one<D, D == 128 ? 1 : 3, D == 128 ? 6 : 2, WT>(p, n_cta, s);   // 33 to 48 rows
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
  p.g_magic = (65536u + p.G - 1) / p.G;
  char* base = static_cast<char*>(a.ws);
  p.counter = reinterpret_cast<unsigned*>(base);
  p.parts = reinterpret_cast<float*>(base + w.parts);
  p.norm = reinterpret_cast<float2*>(base + w.norm);
  p.scores = reinterpret_cast<float*>(base + w.scores);
  p.cap = (int64_t)a.width * a.c.page_size;
  p.log2_page = a.c.page_size == 16 ? 4 : a.c.page_size == 32 ? 5 : a.c.page_size == 64 ? 6 : 7;
  const DecPlan pl = dec_plan(p.rows, a.c.head_dim);
  if (a.c.head_dim == 128) return wt ? launch_plan<128, true>(p, pl, w.n_cta, s) : launch_plan<128, false>(p, pl, w.n_cta, s);
  return wt ? launch_plan<64, true>(p, pl, w.n_cta, s) : launch_plan<64, false>(p, pl, w.n_cta, s);
}

}  // namespace moe
