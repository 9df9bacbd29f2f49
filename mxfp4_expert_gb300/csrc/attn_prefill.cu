// Attention over whole prompts (packed sequences, grouped heads) on the
// 5th-generation tensor cores.
//
// out_i = sum_j softmax_j(scale q_i . k_j) v_j over the keys j that query i
// sees. Work is 4 D flops per visible (query, key) pair and head; both
// products run on tcgen05 (bf16 in, fp32 accumulators in tensor memory), the
// exponentials between them on the special-function units.
//
// Work items. 128 consecutive queries of one head are a query tile. The tiles
// of a sequence and key/value head, ordered by position and then by head of the
// group, are taken two at a time: the pair shares every key and value tile that
// is loaded, and (heads of one group) mostly the same causal range too. Items
// differ in cost by their number of key tiles; a persistent CTA per SM takes
// items c, 2N - 1 - c, 2N + c, ... of the list ordered by falling cost, which
// is nowhere written down: a scheduler warp finds item r by bisection over the
// cost (how many items cost at least x is a sum over sequences, in closed form).
//
// Tensor memory (512 columns): scores S0, S1 (128 fp32 columns each), outputs
// O0, O1 (D each). A key tile's scores come as two halves of 64 keys, each with
// 64 of the 128 columns. Its probabilities, bf16, go over the first half's
// scores, as the A operand of the second product; the next key tile's first
// scores go where the second half's were, and so on by turns.
//
// Warp roles, meeting only at mbarriers:
//   producer (one warp)    the next item; this one's Q tiles, then K0 V0 K1 V1
//                          ... by TMA into a ring
//   MMA 0, 1 (a warp each) of its query tile: S = Q K^T and O += P V. A warp is
//                          held while it issues (the tensor cores take few MMAs
//                          ahead), so one for both tiles would see late that the
//                          other tile is ready
//   scan (one warp)        masked key tiles only, see below
//   softmax 0, 1 (4 warps each, one thread per query): S to registers,
//                          probabilities (fp32 sum, bf16 store), and at the end
//                          O / sum; releases what the products have read
//
// What bounds it: the chain of a query tile. 128 x 128 scores take the
// special-function units 512 cycles (32 a cycle, measured) and the tensor cores
// 557 + 514 for the two products, but a softmax thread is at them for 1900,
// and each hand-over between warps costs 200 to 400. Therefore
//   - scores in halves: as soon as the second half's are in registers the next
//     tile's first half is computed, so that the softmax warps find it ready.
//     Products with 64 keys take 860 cycles a tile instead of 557 (they read as
//     much of Q), which is less than waiting;
//   - a half's probabilities are taken against the reference that was there,
//     which is raised, and O rescaled, only where a half passes it by 2^16 (with
//     scores of 128 keys that rise by 6, 12, 24 and 100 in log2 from tile to tile:
//     211, 242, 260 and 329 us for 8,192 tokens, 189 where they do not);
//   - the first 64 keys' product runs while the other 64 are worked on;
//   - little code: the two halves are one loop and waits call one function. With
//     the halves unrolled the warps waited twice as long for instructions.
// 16,384 tokens, 16 heads over 2 of 128, causal: 690 us, 1,590 TFLOP/s (call
// after call the card's power limit makes it 730); whole tiles of scores, halves
// unrolled, were 749.
//
// Masked places must not count, whatever they hold, but 0 * inf is NaN in the
// second product. For a tile that some query of the item does not see whole the
// scan warp zeroes the value rows past the sequence's end, and non-finite
// values in the others. Where it found one (a broken model) the queries that
// see it get it back at the end: the thread of the query reads the tile's
// values from global memory and adds the non-finite ones to its output.
#include <cuda.h>

#include "attn.h"
#include "f32x2.cuh"
#include "fp8kv.cuh"
#include "tma.cuh"
#include "umma.cuh"

namespace moe {
namespace {

constexpr int kQT = 128, kKT = 128;            // queries per tile, keys per tile
constexpr int kWProd = 0, kWMma0 = 1, kWMma1 = 2, kWSoft = 4;   // and 3: scan
constexpr int kPfWarps = 12;   // 168 registers a thread
constexpr int kPfThreads = kPfWarps * 32;
constexpr float kPfMost = 16.0f;   // log2 of what the reference may be passed by
// Probabilities are taken 2^38 below their reference, so at most 2^-22 each: O, a
// sum of products with values of any size, then stays finite for up to 2^22 keys
// wherever the output is. In return what is below 2^-88 of the reference is 0,
// and outputs lose bits below 2^-80 (bf16 and fp32 end at 2^-126). An exponent of
// -38 has 2^-19 as its rounding: 2^-20 of a probability.
constexpr float kPfBias = 38.0f;
// A score times c is rounded for the reference and not for the probabilities. Up to
// 2^31 they differ by 2^64 at most, which the bias leaves room for. Beyond, scores
// that are not equal differ by 128 at least: only the largest counts, and with the
// power of two below c in its place both products are exact.
constexpr float kPfFar = 2147483648.0f;
constexpr uint32_t kBoxBytes = 128 * 128;      // 128 rows of 64 channels
constexpr int kScanRing = 4;
constexpr float kLn2f = 0.6931471805599453f, kLog2ef = 1.4426950408889634f;

template <int D>
struct PfPlan {
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kTile = kBoxes * kBoxBytes;
  static constexpr int kStages = D == 128 ? 5 : 8;
  // two items' Q where there is room: the next item's is loaded before this one's
  // last scores are done (24 packed prompts of 6,001 tokens, heads of 64: 31.6 us
  // with two, 32.9 with one)
  static constexpr int kQBufs = D == 128 ? 1 : 2;
  static constexpr uint32_t kQ = 0, kRing = kQBufs * 2 * kTile, kBars = kRing + kStages * kTile;
  static constexpr int kNBars = 2 * kQBufs + 2 * kStages + 18 + kScanRing + 4;
  static constexpr uint32_t kItems = kBars + kNBars * 8;
  static constexpr uint32_t kTotal = kItems + 2 * 80 + kScanRing * 4 + 16 + 1024;   // + alignment slack
};
static_assert(PfPlan<128>::kTotal <= 232448 && PfPlan<64>::kTotal <= 232448, "shared memory");

struct PfItem {
  int n;               // key tiles, -1: no more items
  int q0[2], head[2], rows[2], t0[2], nkt[2];   // per query tile: global row, head, rows (0: none), position, key tiles
  int kv0, nk, off, vmin, hk;                   // keys: global row, count; nk - nq; fewest keys a query sees
};
static_assert(sizeof(PfItem) <= 80, "item");

struct PfParams {
  CUtensorMap map[3];    // q, k, v: 64-channel x 128-row boxes
  int swapped[3];        // dimensions are (channel, token, head) instead of (channel, head, token)
  int one_head[3];       // heads share their memory: head coordinate 0
  PrefillArgs a;
  float c;               // |scale| log2(e)
  float c_pow2;          // the power of two not above c
  int negate;            // scale < 0
};

// ---- tensor-memory helpers -------------------------------------------------------
// The MMA warp runs as a whole and lets one lane issue: its operands then are
// uniform for the compiler and live in uniform registers, which the instructions
// want; from within a branch of one lane each of them is moved there first.
// Four products in a row: 64 of the contracted elements; the first adds to what
// is there only if `accumulate`. A in shared memory (steps of 32 bytes), and B
// too (steps of `db` * 16 bytes).
__device__ __forceinline__ void umma_ss_4(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b64 a, b;\n elect.sync _|q, 0xFFFFFFFF;\n setp.ne.b32 p, %4, 0;\n"
      " setp.eq.b32 t, 0, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      " add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n}\n" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void umma_ts_4(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, q, t;\n .reg .b32 a;\n .reg .b64 b;\n elect.sync _|q, 0xFFFFFFFF;\n setp.ne.b32 p, %4, 0;\n"
      " setp.eq.b32 t, 0, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      " add.s32 a, %1, 8;\n add.s64 b, %2, 128;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 16;\n add.s64 b, %2, 256;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 24;\n add.s64 b, %2, 384;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void umma_commit_1(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_1(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n @q mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar)
      : "memory");
}
// Descriptor of an operand whose rows (keys) are K and whose 64-channel boxes
// are M or N ("MN-major"), 128-byte swizzle: lbo = bytes between boxes, 1024
// bytes between groups of 8 keys.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t saddr, uint32_t lbo) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
#define MOE_RW8(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), \
                      "+r"(v[i + 6]), "+r"(v[i + 7])
#define MOE_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), \
                     "=r"(v[i + 6]), "=r"(v[i + 7])
// 32 columns of the warp's lanes; no wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : MOE_R8(v, 0), MOE_R8(v, 8), MOE_R8(v, 16), MOE_R8(v, 24)
      : "r"(taddr));
}
// ... and the values of a load come after it, for the compiler too.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : MOE_RW8(v, 0), MOE_RW8(v, 8), MOE_RW8(v, 16), MOE_RW8(v, 24)::"memory");
}
__device__ __forceinline__ void tie32(uint32_t (&v)[32]) {
  asm volatile("" : MOE_RW8(v, 0), MOE_RW8(v, 8), MOE_RW8(v, 16), MOE_RW8(v, 24));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#define MOE_I8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), \
                     "r"(v[i + 6]), "r"(v[i + 7])
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      MOE_I8(v, 0), MOE_I8(v, 8)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ float pf_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---- the list of items ---------------------------------------------------------------
struct PfSeq {
  int q0, nq, k0, nk, pairs;
};
__device__ __forceinline__ PfSeq pf_seq(const PrefillArgs& a, int G, int b, bool* bad) {
  PfSeq s;
  int q1, k1;
  packed_range(a.cu_q, b, a.total_q, &s.q0, &q1, bad);
  packed_range(a.cu_k, b, a.total_k, &s.k0, &k1, bad);
  s.nq = q1 - s.q0;
  s.nk = k1 - s.k0;
  s.pairs = ((s.nq + kQT - 1) / kQT * G + 1) / 2;
  return s;
}
// Bounded wait of a lane. The long way is one function for all: the warps' loops
// together are near what the instruction cache holds.
__device__ __noinline__ bool pf_wait_long(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return uwait(bar, parity, abort, status);
}
__device__ __forceinline__ bool pf_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return mbar_try_wait(bar, parity) || pf_wait_long(bar, parity, abort, status);
}
// ... of a whole warp: every lane gets the same answer, also where one gives up,
// so the warp stays together for what its lanes do jointly afterwards. The softmax
// warps take the lane's form and one vote a key tile (a vote at each of their
// waits: 768 instead of 735 us for 16,384 tokens).
__device__ __forceinline__ bool pf_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)) ||
         __all_sync(0xFFFFFFFFu, pf_wait_long(bar, parity, abort, status));
}
// Keys that the tile which ends before query `end` sees.
__device__ __forceinline__ int pf_kv_end(const PfSeq& s, int end, int causal) {
  return causal ? min(max(end - s.nq + s.nk, 0), s.nk) : s.nk;   // end <= nq: no step leaves an int
}
// Pairs with at least c key tiles (at least one counts as one): the last ones.
__device__ __forceinline__ int pf_count_ge(const PfSeq& s, int G, int causal, int c) {
  if (c <= 1) return s.pairs;
  const int x = (c - 1) * kKT + 1;          // keys that such a pair sees at least
  if (s.nk < x || s.pairs == 0) return 0;
  if (!causal) return s.pairs;
  const int y = x - (s.nk - s.nq);          // its last query's position + 1, at least
  if (s.nq < y) return 0;
  const int i0 = y <= 0 ? 0 : (y + kQT - 1) / kQT - 1;   // first tile position that reaches it
  return s.pairs - int((int64_t)i0 * G / 2);
}
__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xFFFFFFFFu, v); }

// Whole warp: item number idx (< total), into *out by one lane. `own` is sequence
// number `lane`, kept in registers: each count looks at every sequence. `most`:
// no item has more key tiles.
__device__ void pf_find_item(const PfParams& P, int G, const PfSeq& own, int most, int idx, bool sorted, PfItem* out) {
  const PrefillArgs& a = P.a;
  const int lane = threadIdx.x & 31;
  const int r = idx / a.n_kv, hk = idx % a.n_kv;
  bool ignore = false;
  auto seq = [&](int b) { return b == lane ? own : pf_seq(a, G, b, &ignore); };
  auto count = [&](int c) {
    int n = 0;
    for (int b = lane; b < a.n_seq; b += 32) n += pf_count_ge(seq(b), G, a.causal, c);
    return warp_sum(n);
  };
  int c = 1, skip = 0;      // the item costs c; so many cost more
  if (sorted) {
    int lo = 1, hi = most;
    while (lo < hi) {       // largest c with count(c) > r
      const int mid = (lo + hi + 1) >> 1;
      if (count(mid) > r) lo = mid; else hi = mid - 1;
    }
    c = lo;
    skip = count(c + 1);
  }
  int before = skip;
  for (int b0 = 0; b0 < a.n_seq; b0 += 32) {
    const int b = b0 + lane;
    PfSeq s{0, 0, 0, 0, 0};
    int n = 0, first = 0;
    if (b < a.n_seq) {
      s = seq(b);
      const int ge = pf_count_ge(s, G, a.causal, c);
      n = sorted ? ge - pf_count_ge(s, G, a.causal, c + 1) : s.pairs;
      first = s.pairs - ge;
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    const int lo = before + incl - n;
    const bool mine = r >= lo && r < lo + n;
    if (mine) {
      const int p = first + (r - lo);
      const int tiles = (s.nq + kQT - 1) / kQT * G;
      PfItem it;
      it.kv0 = s.k0;
      it.nk = s.nk;
      it.off = s.nk - s.nq;
      it.hk = hk;
      it.vmin = s.nk;
      it.n = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = 2 * p + j, pos = t / G * kQT;
        const bool have = t < tiles;
        it.head[j] = hk * G + t % G;
        it.t0[j] = pos;
        it.q0[j] = s.q0 + pos;
        it.rows[j] = have ? min(kQT, s.nq - pos) : 0;
        const int end = have ? pf_kv_end(s, min(pos + kQT, s.nq), a.causal) : 0;
        it.nkt[j] = (end + kKT - 1) / kKT;
        it.n = max(it.n, it.nkt[j]);
        if (have && a.causal) it.vmin = min(it.vmin, min(max(pos + 1 + it.off, 0), s.nk));
      }
      *out = it;
    }
    if (__any_sync(0xFFFFFFFFu, mine)) return;
    before += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) prefill_kernel(const __grid_constant__ PfParams P) {
  using Plan = PfPlan<D>;
  constexpr int NS = Plan::kStages;
  constexpr int NB = Plan::kBoxes, NQ = Plan::kQBufs;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + Plan::kBars);
  uint64_t* q_empty = q_full + NQ;     // [NQ] each
  uint64_t* full = q_empty + NQ;
  uint64_t* empty = full + NS;
  uint64_t* s_full = empty + NS;       // [2][2]: query tile, half of the keys
  uint64_t* p_first = s_full + 4;      // [2]: the first half's probabilities are there, the second half's scores taken
  uint64_t* p_second = p_first + 2;    // [2]: the second half's probabilities
  uint64_t* h_done = p_second + 2;       // [2]: the first half's product
  uint64_t* o_full = h_done + 2;       // [2]
  uint64_t* o_free = o_full + 2;       // [2]
  uint64_t* scanned = o_free + 2;      // [kScanRing]
  uint64_t* fin = scanned + kScanRing;       // [2]: a warp's MMAs at the end
  uint64_t* turn = fin + 2;                  // [2]: the other MMA warp has issued
  uint64_t* it_full = turn + 2;              // [2]
  uint64_t* it_empty = it_full + 2;          // [2]
  PfItem* items = reinterpret_cast<PfItem*>(smem + Plan::kItems);
  volatile int* poison = reinterpret_cast<volatile int*>(smem + Plan::kItems + 2 * 80);   // [kScanRing]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + Plan::kItems + 2 * 80 + kScanRing * 4);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);

  const PrefillArgs& a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.n_heads / a.n_kv;
  int* status = a.status;

  if (tid == 0) {
    for (int i = 0; i < NQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 2);   // both MMA warps
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 3);     // both MMA warps, scan
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[2 * i], 1);
      mbar_init(&s_full[2 * i + 1], 1);
      mbar_init(&p_first[i], 4);
      mbar_init(&p_second[i], 4);
      mbar_init(&h_done[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&it_full[i], 1);
      mbar_init(&fin[i], 1);
      mbar_init(&turn[i], 1);
      mbar_init(&it_empty[i], 11);   // 2 MMA, scan, 8 softmax warps
    }
    for (int i = 0; i < kScanRing; ++i) mbar_init(&scanned[i], 1);
    *abort = 0;
    mbar_fence_init();
  }
  if (warp == kWMma0) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t base = smem_addr(smem);
  const uint32_t q_s = base + Plan::kQ, ring_s = base + Plan::kRing;

  // The t-th item of this CTA, copied out of its slot (whole warp; one lane
  // arrives when all have it).
  auto next_item = [&](int t, bool arrives, PfItem* it) {
    if (!pf_wait_warp(&it_full[t & 1], uint32_t(t >> 1) & 1u, abort, status)) return false;
    *it = items[t & 1];
    __syncwarp();
    if (arrives) mbar_arrive(&it_empty[t & 1]);
    return it->n >= 0;
  };

  if (warp < kWSoft) {
    if (warp == kWProd) {
      // ---- producer: items, and their loads -------------------------------------------------
      bool bad = false, ok = true;
      PfSeq own{0, 0, 0, 0, 0};
      int total = 0, most = 1;
      for (int b = lane; b < a.n_seq; b += 32) {
        const PfSeq x = pf_seq(a, G, b, &bad);
        if (b == lane) own = x;
        total += x.pairs;
        most = max(most, (x.nk + kKT - 1) / kKT);
      }
      total = warp_sum(total) * a.n_kv;
      most = __reduce_max_sync(0xFFFFFFFFu, most);
      bad = __any_sync(0xFFFFFFFFu, bad);
      if (bad && blockIdx.x == 0 && lane == 0 && status) atomicOr(status, MOE_DEV_INDEX_OOB);
      const int N = gridDim.x, c = blockIdx.x;
      // item t of this CTA into its slot; false if there is none (nor any later)
      auto publish = [&](int t) {
        if (t >= 2 && !pf_wait_warp(&it_empty[t & 1], uint32_t((t >> 1) - 1) & 1u, abort, status)) {
          ok = false;
          return false;
        }
        const int64_t idx = (int64_t)t * N + (t & 1 ? N - 1 - c : c);
        if (idx < total)
          pf_find_item(P, G, own, most, int(idx), total > N, &items[t & 1]);
        else if (lane == 0)
          items[t & 1].n = -1;
        __threadfence_block();
        __syncwarp();
        if (lane == 0) mbar_arrive(&it_full[t & 1]);
        return idx < total;
      };
      int s = 0, issued_q = 0, loads = 0;   // ring stage
      uint32_t par = 1;                     // phase of its release: the first lap waits for none
      bool more = publish(0);
      for (int t = 0; ok && more; ++t) {
        more = publish(t + 1);
        const PfItem& it = items[t & 1];
        if (lane == 0 && it.n > 0) {
          // Q: after the last products with what was there
          const int qb = issued_q % NQ;
          if (issued_q >= NQ && !pf_wait(&q_empty[qb], uint32_t(issued_q / NQ - 1) & 1u, abort, status)) ok = false;
          if (ok) {
            const int have1 = it.rows[1] > 0;
            mbar_arrive_expect_tx(&q_full[qb], (1 + have1) * Plan::kTile);
            for (int j = 0; j <= have1; ++j)
              for (int x = 0; x < NB; ++x) {
                const int h = P.one_head[0] ? 0 : it.head[j], r = it.q0[j];
                tma_load_3d(q_s + (2 * qb + j) * Plan::kTile + x * kBoxBytes, &P.map[0], x * 64, P.swapped[0] ? r : h,
                            P.swapped[0] ? h : r, &q_full[qb]);
              }
            ++issued_q;
          }
          for (int i = 0; ok && i < 2 * it.n; ++i) {
            const int w = 1 + (i & 1);
            if (loads >= NS && !pf_wait(&empty[s], par, abort, status)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&full[s], Plan::kTile);
            const int h = P.one_head[w] ? 0 : it.hk, r = it.kv0 + (i >> 1) * kKT;
            for (int x = 0; x < NB; ++x)
              tma_load_3d(ring_s + s * Plan::kTile + x * kBoxBytes, &P.map[w], x * 64, P.swapped[w] ? r : h,
                          P.swapped[w] ? h : r, &full[s]);
            ++loads;
            if (++s == NS) s = 0, par ^= 1;
          }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
      }
      if (lane == 0 && *abort) {   // copies in flight land before the CTA's shared memory goes away
        for (int i = loads > NS ? loads - NS : 0; i < loads; ++i) mbar_wait(&full[i % NS], uint32_t(i / NS) & 1u, status);
        for (int i = issued_q > NQ ? issued_q - NQ : 0; i < issued_q; ++i)
          mbar_wait(&q_full[i % NQ], uint32_t(i / NQ) & 1u, status);
      }
    } else if (warp == kWMma0 || warp == kWMma1) {
      // ---- MMA --------------------------------------------------------------------------
      // The whole warp; what is needed per key tile is kept up to date by
      // additions (no division by the ring's length, no descriptor built anew).
      constexpr uint32_t kTile16 = Plan::kTile >> 4, kBox16 = kBoxBytes >> 4;
      const int j = warp == kWMma1;
      const uint32_t id_s = umma_idesc_bf16(kQT, kKT / 2) | (P.negate ? 1u << 13 : 0u);   // bit 13: negate A
      const uint32_t id_o = umma_idesc_bf16(kQT, D) | (1u << 16);                     // bit 16: B is MN-major
      const uint64_t dq0 = umma_desc_sw128(q_s + j * Plan::kTile);
      const uint64_t dk = umma_desc_sw128(ring_s), dv = umma_desc_mn_sw128(ring_s, kBoxBytes);
      const uint32_t ts = tmem + j * kKT, to = tmem + 256 + j * D;
      const uint32_t empty_s = smem_addr(empty), q_empty_s = smem_addr(q_empty);
      uint64_t dq = dq0;
      uint32_t st = 0, par = 0;                      // ring stage and phase
      uint32_t q_buf = NQ - 1, q_par = 1, p_par = 0, o_par = 1;      // phases of Q, of the probabilities, of O's release
      uint32_t turn_par = 1 - j;                     // tile 0 begins
      uint32_t g = 0;                                // columns of a key tile's first scores: g * 64
      bool ok = true, o_used = false;
      auto wait = [&](uint64_t* bar, uint32_t ph) { return pf_wait_warp(bar, ph, abort, status); };
      auto scores = [&](uint32_t stage, int half, uint32_t col) {
        const uint64_t b0 = dk + stage * kTile16 + half * (kBox16 / 2);
#pragma unroll
        for (int x = 0; x < NB; ++x) umma_ss_4(ts + col, dq + x * kBox16, b0 + x * kBox16, id_s, x > 0);
        umma_commit_1(smem_addr(&s_full[2 * j + half]));
      };
      // On to the next stage. The softmax warps see from the scores that follow
      // when a stage has been read; one of a tile that is not theirs is given
      // up here.
      auto next_stage = [&](bool unused) {
        if (unused) mbar_arrive_1(empty_s + 8 * st);
        if (++st == NS) st = 0, par ^= 1;
      };
      PfItem it;
      for (int t = 0; ok && next_item(t, lane == 0, &it); ++t) {
        const int n = __shfl_sync(0xFFFFFFFFu, it.n, 0);
        const int nkt = __shfl_sync(0xFFFFFFFFu, j ? it.nkt[1] : it.nkt[0], 0);
        if (n == 0) continue;
        if (++q_buf == NQ) q_buf = 0, q_par ^= 1;
        dq = dq0 + q_buf * (2 * kTile16);
        if (!(ok = wait(&q_full[q_buf], q_par)) || !(ok = wait(&full[st], par))) break;
        tc_fence_after();
        if (nkt > 0) {
          scores(st, 0, 64 * g);
          scores(st, 1, 64 - 64 * g);
        }
        next_stage(nkt == 0);
        if (n == 1) umma_commit_1(q_empty_s + 8 * q_buf);
        for (int i = 0; i < n; ++i) {
          if (!(ok = wait(&full[st], par))) break;
          const uint64_t b0 = dv + st * kTile16;
          if (i < nkt) {
            if (i == 0) {              // the last item's output has been read
              if (o_used && !(ok = wait(&o_free[j], o_par))) break;
              o_used = true;
              o_par ^= 1;
            }
            if (i + 1 < nkt) {         // the next tile's first scores, where this one's second ones were
              const uint32_t st1 = st + 1 == NS ? 0 : st + 1;
              if (!(ok = wait(&full[st1], st1 ? par : par ^ 1)) || !(ok = wait(&p_first[j], p_par))) break;
              tc_fence_after();
              scores(st1, 0, 64 - 64 * g);
            } else {
              if (!(ok = wait(&p_first[j], p_par))) break;
              tc_fence_after();
            }
            umma_ts_4(to, ts + 64 * g, b0, id_o, i > 0);
            umma_commit_1(smem_addr(&h_done[j]));
            if (!(ok = wait(&p_second[j], p_par))) break;
            p_par ^= 1;
          }
          if (i < nkt) {
            tc_fence_after();
            umma_ts_4(to, ts + 64 * g + 32, b0 + 4 * 128, id_o, true);
            if (i + 1 == nkt) umma_commit_1(smem_addr(&o_full[j]));
          }
          // the two tiles' second products and next scores strictly in turn
          if (!(ok = wait(&turn[j], turn_par))) break;
          turn_par ^= 1;
          next_stage(i >= nkt);
          if (i + 1 < n) {
            if (i + 1 < nkt)
              scores(st, 1, 64 * g);
            else if (!(ok = wait(&full[st], par)))
              break;
            mbar_arrive_1(smem_addr(&turn[1 - j]));
            next_stage(i + 1 >= nkt);
            if (i + 2 == n) umma_commit_1(q_empty_s + 8 * q_buf);
          } else {
            mbar_arrive_1(smem_addr(&turn[1 - j]));
          }
          if (i < nkt) g ^= 1;
        }
      }
      // every MMA has finished before tensor memory is freed
      umma_commit_1(smem_addr(&fin[j]));
      mbar_wait(&fin[j], 0, status);
    } else {
      // ---- scan -------------------------------------------------------------------------
      int s = 0, ns = 0;             // ring stage; masked tiles
      uint32_t par = 0;
      PfItem it;
      bool ok = true;
      for (int t = 0; ok && next_item(t, lane == 0, &it); ++t) {
        for (int e = 0; e < 2 * it.n; ++e) {
          const int i = e >> 1;
          if (!pf_wait_warp(&full[s], par, abort, status)) {
            ok = false;
            break;
          }
          if ((e & 1) && (i + 1) * kKT > it.vmin) {
            uint8_t* v = smem + Plan::kRing + s * Plan::kTile;
            const int rows = min(kKT, it.nk - i * kKT);
            uint32_t found = 0;
            for (int x = 0; x < NB; ++x) {
              uint4* box = reinterpret_cast<uint4*>(v + x * kBoxBytes);
              for (int e = lane; e < rows * 8; e += 32) {
                const uint4 w = box[e];
                // a half has exponent 255 iff adding one to its exponent field carries into its sign
                found |= ((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u) |
                         ((w.z & 0x7F807F80u) + 0x00800080u) | ((w.w & 0x7F807F80u) + 0x00800080u);
              }
              for (int e = rows * 8 + lane; e < kKT * 8; e += 32) box[e] = make_uint4(0, 0, 0, 0);
            }
            const bool any = __any_sync(0xFFFFFFFFu, (found & 0x80008000u) != 0);
            if (any) {
              for (int e = lane; e < rows * 64 * NB / 2; e += 32) {   // two values at a time
                uint32_t* p2 = reinterpret_cast<uint32_t*>(v + (e / (rows * 32)) * kBoxBytes) + e % (rows * 32);
                const uint32_t w = *p2;
                *p2 = ((w & 0x7F80u) == 0x7F80u ? 0u : w & 0xFFFFu) | ((w & 0x7F800000u) == 0x7F800000u ? 0u : w & 0xFFFF0000u);
              }
            }
            fence_async_smem();   // the zeros, before the tensor cores read them
            __syncwarp();
            if (lane == 0) {
              poison[ns & (kScanRing - 1)] = any ? 1 : 0;
              __threadfence_block();
              mbar_arrive(&scanned[ns & (kScanRing - 1)]);
            }
            ++ns;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[s]);
          if (++s == NS) s = 0, par ^= 1;
        }
      }
    }
  } else {
    // ---- softmax ------------------------------------------------------------------------
    const int j = (warp - kWSoft) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + j * kKT, to = tmem + lanes + 256 + j * D;
    int st = 0;                     // ring stage of the next key tile's keys
    int nsf = 0, nof = 0, ns = 0;   // scores and outputs awaited; masked tiles
    bool ok = true;
    PfItem it;
    const float c = P.c;
    for (int t = 0; ok && next_item(t, lane == 0, &it); ++t) {
      const int nkt = it.nkt[j];
      const int vis = a.causal ? min(max(it.t0[j] + row + it.off + 1, 0), it.nk) : it.nk;
      const int vis_w = __shfl_sync(0xFFFFFFFFu, vis, 0);   // the warp's fewest
      float m = -INFINITY, l = 0.0f;   // reference, sum in units of 2^m
      float cc = c, ref = 0.0f;        // exponent of a probability: score * cc - ref
      unsigned bad = 0;                // masked tiles with non-finite values (a pair's queries span at most 4)
      for (int i = 0; i < nkt; ++i) {
        const int k0 = i * kKT;
        const bool masked = k0 + kKT > it.vmin;
        const uint32_t ph = uint32_t(nsf) & 1u, ta = ts + 64 * ph, tb = ts + 64 - 64 * ph;
        ++nsf;
        const int n_vis = vis - k0;
        const bool cut = k0 + kKT > vis_w;   // some lane of the warp does not see the whole tile
        uint32_t s[2][32];
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (!pf_wait(&s_full[2 * j + half], ph, abort, status)) ok = false;
          if (half == 1) {   // the products before these scores are done, too: their values are released with the keys
            if (warp == kWSoft + 4 * j && lane == 0) {
              if (i > 0) mbar_arrive(&empty[st == 0 ? NS - 1 : st - 1]);
              mbar_arrive(&empty[st]);
            }
            st = st + 2 >= NS ? st + 2 - NS : st + 2;
          }
          tc_fence_after();
          tmem_ld32(half ? tb : ta, s[0]);
          tmem_ld32((half ? tb : ta) + 32, s[1]);
          tmem_wait_ld32(s[0]);
          tie32(s[1]);
          if (half == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_first[j]);
          }
          float mx[4];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint32_t(&x)[32] = s[b];
            if (cut) {
#pragma unroll
              for (int y = 0; y < 32; ++y)
                if (64 * half + 32 * b + y >= n_vis) x[y] = 0xFF800000u;
            }
            float a0 = __uint_as_float(x[0]), a1 = __uint_as_float(x[1]);
#pragma unroll
            for (int y = 2; y + 4 <= 30; y += 4) {
              a0 = max3(a0, __uint_as_float(x[y]), __uint_as_float(x[y + 1]));
              a1 = max3(a1, __uint_as_float(x[y + 2]), __uint_as_float(x[y + 3]));
            }
            mx[2 * b] = max3(a0, __uint_as_float(x[30]), __uint_as_float(x[31]));
            mx[2 * b + 1] = a1;
          }
          const float raw = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]), mine = raw * c;
          const float r = (i == 0 && half == 0) || mine > m + kPfMost ? mine : -INFINITY;
          if (__any_sync(0xFFFFFFFFu, r > m)) {
            const float f = r > m ? pf_ex2(m - r) : 1.0f;
            if (r > m) {
              m = r;
              const bool far = fabsf(m) > kPfFar;
              cc = far ? P.c_pow2 : c;
              ref = far ? raw * P.c_pow2 : m + kPfBias;
            }
            l *= f;
            // what is in O: the earlier tiles' products, which have finished
            // when this tile's second scores have, since these were issued after
            // them; in the second half this tile's first product too, after
            // which the next tile's first scores are issued
            if (half == 1 || i > 0) {
              if (!pf_wait(half ? &h_done[j] : &s_full[2 * j + 1], ph, abort, status)) ok = false;
              tc_fence_after();
            }
            if (i > 0 || half == 1) {
#pragma unroll 1
              for (int z = 0; z < D; z += 16) {
                uint32_t o[16];
                tmem_ld16(to + z, o);
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                tmem_st16(to + z, o);
              }
            }
          }
          const uint64_t c2 = pack2(cc, cc), r2 = pack2(-ref, -ref);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint32_t(&x)[32] = s[b];
            float e[32];
#pragma unroll
            for (int y = 0; y < 32; y += 2)
              unpack2(fma2(pack2(__uint_as_float(x[y]), __uint_as_float(x[y + 1])), c2, r2), e[y], e[y + 1]);
#pragma unroll
            for (int y = 0; y < 32; ++y) e[y] = pf_ex2(e[y]);
            uint32_t pb[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) pb[y] = bf16x2_bits(e[2 * y], e[2 * y + 1]);
            tmem_st16(ta + 32 * half + 16 * b, pb);
            uint64_t sum[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) sum[y] = add2(pack2(e[2 * y], e[2 * y + 1]), pack2(e[2 * y + 8], e[2 * y + 9]));
#pragma unroll
            for (int y = 16; y < 32; y += 8)
#pragma unroll
              for (int z = 0; z < 4; ++z) sum[z] = add2(sum[z], pack2(e[y + 2 * z], e[y + 2 * z + 1]));
            float a0, a1;
            unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a0, a1);
            l += a0 + a1;
          }
          if (half == 0) {
            if (masked) {
              const int slot = ns & (kScanRing - 1);
              if (!pf_wait(&scanned[slot], uint32_t(ns / kScanRing) & 1u, abort, status)) ok = false;
              ++ns;
              if (poison[slot]) bad |= 1u << (i - it.vmin / kKT);
            }
            tmem_wait_st();
          }
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_second[j]);
      }
      if (!ok) break;
      const int st_end = (st + 2 * (it.n - nkt)) % NS;
      // masked tiles of the item that this query tile does not take part in
      {
        const int from = max(it.vmin / kKT, nkt);
        if (it.n > from) ns += it.n - from;
      }
      if (it.rows[j] == 0) {
        st = st_end;
        continue;
      }
      const bool mine = row < it.rows[j];
      const int64_t orow = (int64_t)(it.q0[j] + row) * a.n_heads + it.head[j];
      __nv_bfloat16* out = a.out + orow * D;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      if (nkt > 0) {
        if (!pf_wait_warp(&o_full[j], uint32_t(nof++) & 1u, abort, status)) break;
        if (warp == kWSoft + 4 * j && lane == 0) mbar_arrive(&empty[st == 0 ? NS - 1 : st - 1]);
        tc_fence_after();
      }
#pragma unroll
      for (int x = 0; x < D; x += 32) {
        uint32_t o[32];
        if (nkt > 0) {
          tmem_ld32(to + x, o);
          tmem_wait_ld32(o);
          if (x + 32 == D) {   // all of O is in registers: the next item may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[j]);
          }
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = 0;
        }
        for (unsigned left = bad; left; left &= left - 1) {
          const int k0 = (it.vmin / kKT + __ffs(left) - 1) * kKT;
          const __nv_bfloat16* v = a.v + (int64_t)(it.kv0 + k0) * a.v_ts + it.hk * a.v_hs + x;
          const int keys = min(kKT, vis - k0);
          for (int k = 0; k < keys; ++k) {
            const uint4* w4 = reinterpret_cast<const uint4*>(v + k * a.v_ts);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint4 w = w4[y];
              const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                uint32_t &o0 = o[8 * y + 2 * z], &o1 = o[8 * y + 2 * z + 1];
                if ((ww[z] & 0x7F80u) == 0x7F80u) o0 = __float_as_uint(__uint_as_float(o0) + bf16_lo(ww[z]));
                if ((ww[z] & 0x7F800000u) == 0x7F800000u) o1 = __float_as_uint(__uint_as_float(o1) + bf16_hi(ww[z]));
              }
            }
          }
        }
        uint32_t b[16];
#pragma unroll
        for (int y = 0; y < 16; ++y)
          b[y] = l == 0.0f ? 0u : bf16x2_bits(__uint_as_float(o[2 * y]) * inv, __uint_as_float(o[2 * y + 1]) * inv);
        if (mine) {
#pragma unroll
          for (int y = 0; y < 4; ++y)
            *reinterpret_cast<uint4*>(out + x + y * 8) = make_uint4(b[4 * y], b[4 * y + 1], b[4 * y + 2], b[4 * y + 3]);
        }
      }
      st = st_end;
      if (mine && a.lse) a.lse[orow] = l == 0.0f ? -INFINITY : (m + log2f(l * pow2(int(kPfBias)))) * kLn2f;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWMma0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Tensor map of bf16 rows [tokens][heads][D] with these strides (elements):
// boxes of 64 channels of one head by 128 tokens, 128-byte swizzle. The outer
// dimension is the one with the larger stride.
int encode_rows(PfParams* p, int w, const __nv_bfloat16* base, int tokens, int heads, int D, int64_t ts, int64_t hs) {
  if (heads > 1 && hs == 0) {
    p->one_head[w] = 1;
    heads = 1;
  }
  if (heads == 1) hs = D;
  if (tokens == 1) ts = D;
  const bool sw = hs > ts;
  p->swapped[w] = sw;
  const uint64_t dims[3] = {uint64_t(D), uint64_t(sw ? tokens : heads), uint64_t(sw ? heads : tokens)};
  const uint64_t strides[2] = {uint64_t(sw ? ts : hs) * 2, uint64_t(sw ? hs : ts) * 2};
  const uint32_t box[3] = {64, sw ? 128u : 1u, sw ? 1u : 128u};
  return tma_encode(&p->map[w], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D>
int launch_pf(const PfParams& P, const DeviceInfo& di, cudaStream_t s) {
  constexpr uint32_t smem = PfPlan<D>::kTotal;
  if (smem > di.smem_optin) return MOE_ERR_UNSUPPORTED_SHAPE;
  MOE_CUDA_TRY(cudaFuncSetAttribute(prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
  const int64_t G = P.a.n_heads / P.a.n_kv;
  const int64_t most = P.a.n_kv * (((int64_t)P.a.total_q / kQT + P.a.n_seq) * G / 2 + P.a.n_seq);
  const int grid = int(most < di.sm_count ? most : di.sm_count);
  prefill_kernel<D><<<grid, kPfThreads, smem, s>>>(P);
  return launch_status();
}

}  // namespace

int launch_attn_prefill(const PrefillArgs& a, const DeviceInfo& di, cudaStream_t s) {
  PfParams P{};
  int st;
  if ((st = encode_rows(&P, 0, a.q, a.total_q, a.n_heads, a.D, a.q_ts, a.q_hs))) return st;
  if (a.total_k > 0) {
    if ((st = encode_rows(&P, 1, a.k, a.total_k, a.n_kv, a.D, a.k_ts, a.k_hs))) return st;
    if ((st = encode_rows(&P, 2, a.v, a.total_k, a.n_kv, a.D, a.v_ts, a.v_hs))) return st;
  }
  P.a = a;
  // a scale of 0 must still turn a masked score (-inf) into a probability of 0
  const float c = fabsf(a.scale) * kLog2ef;
  P.c = c > 1e-30f ? c : 1e-30f;
  P.c_pow2 = exp2f(floorf(log2f(P.c)));
  P.negate = a.scale < 0.0f;
  return a.D == 128 ? launch_pf<128>(P, di, s) : launch_pf<64>(P, di, s);
}

}  // namespace moe
