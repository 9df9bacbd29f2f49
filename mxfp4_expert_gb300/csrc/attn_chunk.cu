// Attention of chunks of new tokens over the 8-bit paged cache, on the
// 5th-generation tensor cores.
//
// out_i = sum_j softmax_j(scale q_i . k_j) v_j over the positions j that token i
// sees, 4 head_dim flops a visible pair and head. Keys and values come as E4M3 codes
// with a power of two per page and head; both products run on tcgen05 in f16, of
// which every code is a number. The scales stay outside: a key page's is a factor
// of its scores, a value page's of its probabilities.
//
// Work items. The rows of a sequence and key/value head are its new tokens times
// the heads of the group (row r: token r / G, head r % G); 256 of them, two query
// tiles of 128, are an item and share every key and value tile that is converted.
// Costs, in closed form, lay all items end to end; CTA c of N takes the stretch from
// c / N to (c + 1) / N of the whole, cut at key tiles: work is even whatever the
// lengths are, and few rows over many positions are shared out. An item that is cut
// leaves partial results in the workspace, which a second kernel joins.
//
// Tensor memory and the order of the products are the prompt kernel's: scores S0,
// S1 (128 fp32 columns each, two halves of 64 keys), outputs O0, O1; probabilities go
// over scores as the A operand of the second product.
//
// Warp roles:
//   producer (one warp)    items; page-table entries, scale bytes; raw pages by
//                          1-D bulk copies into a ring
//   MMA 0, 1 (a warp each) of its query tile: S = Q K^T and O += P V
//   converters (4 warps)   codes to f16, two an instruction, into the operand
//                          ring; values that nobody sees to zero
//   softmax 0, 1 (4 warps each, one thread per row): Q to f16 (a power of two per
//                          row puts its largest in [2^14, 2^15)), then scores to
//                          probabilities, and O / sum at the end
//
// Numerics. A row has two references: its scores' (a score it has had, raised when
// passed by 2^16), which the sum is relative to, and its products' p 2^(value scale)
// (an integer power of two above the scores', raised when passed by 2^7), which O is
// relative to: probabilities are f16, 2^8 above that reference, so at most 2^15, of
// 11 bits down to 2^-22 and none below 2^-33 of it. Differences of scores beyond
// 2^17 are taken before they are scaled. Sums and outputs are fp32.
//
// Masked places must not count, whatever they hold, but 0 * NaN is NaN in the
// second product: in a tile that some row of the item does not see whole the
// converters put 0 for NaN; the rows that see it get it back at the end.
//
// Measured: the last 4,096 tokens of 32,768, 32 heads over 4 of 128, in 1,640 us (1,257
// TFLOP/s, 0.66 of the GEMM rate); chunks of four sequences, 1,024 tokens in all (68 to
// 555 each) behind 40,413 to 65,536, in 854 (1,145 TFLOP/s). What bounds it for heads of
// 128 is shared memory: a key tile costs 256 rows 2,066 wavefronts of
// tensor operands (Q is read once for each half), about 1,120 of the converters and
// 256 of the copies, of 3,950 cycles. Heads of 64 in short pages are bound by the
// softmax threads (24 follow-ups of 63 tokens on average: 130 us, 4,600 cycles a tile),
// items of few rows by the converters (2,200 cycles a tile), a single short call by its
// chain (37 tokens behind 5,000: 32 us).
// - Instructions have to be few as well: with long waits in line, the converters' loop
//   unrolled and every mask in its own pass, the same took 1,122 instead of 888 us.
// - Scores of 128 keys in one product read Q once, but a tile's chain of products then
//   stands between two softmax passes: 1,098 instead of 868 us for the four sequences.
// - Moving registers between the roles (setmaxnreg) 905 instead of 870, the next half's
//   scores fetched early 954 to 983 instead of 888, no turns between the MMA warps 880.
#include <math.h>

#include "attn.h"
#include "attn_tc.cuh"
#include "f32x2.cuh"
#include "fp8kv.cuh"
#include "umma.cuh"

namespace moe {
namespace {

constexpr int kQT = 128, kKT = 128;        // rows per query tile, keys per tile
constexpr int kThreads = 512;
constexpr int kWProd = 0, kWMma0 = 1, kWMma1 = 2, kWConv = 4, kWSoft = 8;
constexpr uint32_t kBoxBytes = 128 * 128;  // 128 rows of 64 f16 channels
constexpr int kSlots = 16;                 // key tiles whose scale bytes are kept
constexpr float kRaiseSum = 16.0f, kRaiseOut = 7.0f, kPBias = 8.0f;   // log2; see above
constexpr float kFar = 131072.0f;
constexpr float kLn2f = 0.6931471805599453f;
// Work of an item beside its keys, in keys, and the least work of a CTA, in keys of
// a whole group: cuts of one item are then more than a tile apart (an item of n >= 2
// tiles costs at most G (128 n + 256 + 1) + 256, so a tile at most 257 G + 128).
constexpr int kItemKeys = 256, kCtaKeys = 512;

template <int D>
struct Plan {
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kTile = kBoxes * kBoxBytes;      // f16 operand tile
  static constexpr uint32_t kRaw = 128 * D;                  // codes of a tile
  static constexpr int kStages = D == 128 ? 4 : 8, kRaws = D == 128 ? 2 : 6;
  static constexpr uint32_t kQ = 0, kRing = 2 * kTile, kRawRing = kRing + kStages * kTile;
  static constexpr uint32_t kInfo = kRawRing + kRaws * kRaw;
  static constexpr uint32_t kBars = kInfo + kSlots * 64;
  static constexpr int kNBars = 2 * kRaws + 2 * kStages + 2 + 4 + 2 * 6 + 2 + 4 + 2 * kSlots;
  static constexpr uint32_t kItems = kBars + kNBars * 8;
  static constexpr uint32_t kTotal = kItems + 2 * 96 + 16 + 1024;   // + alignment slack
};
static_assert(Plan<128>::kTotal <= 232448 && Plan<64>::kTotal <= 232448, "shared memory");

struct Item {
  int n;                 // key tiles of this part, -1: no more items
  int t0;                // its first key tile
  int nkt[2];            // of them, those that each query tile sees
  int rows[2];           // rows of each query tile, 0: none
  int r0;                // first row
  int b, hk, q0;         // sequence, key/value head, sequence's first token
  int off, nk, vmin;     // nk - nq, positions, fewest positions a row sees
  int slot;              // partial result's place, -1: the item is whole
};
static_assert(sizeof(Item) <= 96, "item");

// A key tile's eight groups of 16 positions: scale bytes of the keys, exponents of the
// values' scales, groups without a page; NaN that each converter warp found in the
// values.
struct __align__(64) Info {
  uint32_t k[2], bad;
  uint8_t poison[4];
  float v[8];
};

// What a CTA leaves for the join.
struct __align__(32) Desc {
  int last;              // 1: the CTA's last item is cut, its part is in slot 2 c + 1
  int first;             // bit 0: the first item continues an earlier CTA's (slot 2 c), bit 1: and a later CTA's it
  int q0, r0, rows, hk;  // of the last item
};

struct Params {
  ChunkArgs a;
  int G, log2_page;
  float cm;              // |scale| log2(e) = cm 2^ce, cm in [1, 2)
  int ce, negate;        // negate: scale < 0
  Desc* desc;            // [CTAs]
  float4* parts;         // per slot: [D / 4][256] outputs, then [256] references and sums
};

// ---- the list of items -----------------------------------------------------------
struct Seq {
  int q0, nq, nk, items;
  int64_t off, work;     // G (nk - nq); work of one key/value head's items
};
// work of the items before number p: G times kItemKeys and, about, the positions each one's last row sees
__device__ __forceinline__ int64_t work_before(int64_t off, int G, int64_t p) {
  const int64_t p0 = off >= 0 ? 0 : min(-off >> 8, p);
  return 128 * (p * (p + 1) - p0 * (p0 + 1)) + (p - p0) * off + p * (G * kItemKeys);
}
__device__ __forceinline__ Seq load_seq(const Params& P, int b, bool* bad) {
  const ChunkArgs& a = P.a;
  Seq s;
  int q1;
  const int x = __ldg(a.lengths + b);
  packed_range(a.cu_q, b, a.total_q, &s.q0, &q1, bad);
  s.nq = q1 - s.q0;
  s.nk = min(max(x, 0), a.width << P.log2_page);
  if (s.nk != x) *bad = true;
  s.items = int(((int64_t)s.nq * P.G + 255) >> 8);
  s.off = (int64_t)P.G * (s.nk - s.nq);
  s.work = work_before(s.off, P.G, s.items);
  return s;
}
// key tiles that rows [0, end) of the sequence see
__device__ __forceinline__ int tiles_to(const Seq& s, int G, int64_t end) {
  const int64_t rows = (int64_t)s.nq * G;
  const int t = int(uint32_t((end < rows ? end : rows) - 1) / uint32_t(G));       // rows fit an int
  return (min(max(s.nk - s.nq + (t + 1), 0), s.nk) + kKT - 1) / kKT;   // no step leaves an int
}
// A place in the list: item (sequence, head, number) and a key tile inside it,
// which is 0 or cuts the item.
struct Pos {
  int b, hk, p, t;
};
__device__ __forceinline__ bool same_item(const Pos& x, const Pos& y) { return x.b == y.b && x.hk == y.hk && x.p == y.p; }

// Whole warp: first sequence from b on that has items, n_seq if none.
__device__ __forceinline__ int seq_from(const Params& P, int b) {
  const int lane = threadIdx.x & 31;
  bool bad;
  for (; b < P.a.n_seq; b += 32) {
    int q0 = 0, q1 = 0;
    if (b + lane < P.a.n_seq) packed_range(P.a.cu_q, b + lane, P.a.total_q, &q0, &q1, &bad);
    const unsigned any = __ballot_sync(0xFFFFFFFFu, q1 > q0);
    if (any) return b + __ffs(any) - 1;
  }
  return P.a.n_seq;
}
__device__ __forceinline__ Pos next_item(const Params& P, const Seq& s, Pos x) {
  x.t = 0;
  if (++x.p == s.items) {
    x.p = 0;
    if (++x.hk == P.a.c.n_kv_heads) {
      x.hk = 0;
      x.b = seq_from(P, x.b + 1);
    }
  }
  return x;
}
// Whole warp: the places at at[0], at[1] of the whole work (n_seq where there is
// none), and the whole work into *total. Two rounds over the sequences: the places
// depend on the total.
__device__ void find_places(const Params& P, int c, int* n_cta, Pos (&x)[2], bool* bad) {
  const int lane = threadIdx.x & 31, H = P.a.c.n_kv_heads, n_seq = P.a.n_seq;
  Seq own{};
  if (lane < n_seq) own = load_seq(P, lane, bad);
  int64_t total = own.work * H;
  for (int b = lane + 32; b < n_seq; b += 32) total += load_seq(P, b, bad).work * H;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  const int64_t least = (int64_t)P.G * kCtaKeys;
  const int N = total >= least * gridDim.x ? int(gridDim.x) : max(int(total / least), 1);
  *n_cta = N;
  int64_t at[2], before[2];
  int b[2], hk[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = c + k;
    at[k] = total / N * i + total % N * i / N;
    b[k] = -1;
    if (c >= N || i >= N || total == 0) b[k] = n_seq;
  }
  int64_t sum = 0;
  bool ignore;
  for (int b0 = 0; b0 < n_seq && (b[0] < 0 || b[1] < 0); b0 += 32) {
    const int64_t w = b0 == 0 ? own.work * H : b0 + lane < n_seq ? load_seq(P, b0 + lane, &ignore).work * H : 0;
    int64_t incl = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    incl += sum;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, w > 0 && at[k] < incl);
      if (b[k] < 0 && hit) {
        b[k] = b0 + __ffs(hit) - 1;
        before[k] = __shfl_sync(0xFFFFFFFFu, incl - w, __ffs(hit) - 1);
      }
    }
    sum = __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    x[k] = Pos{n_seq, 0, 0, 0};
    if (b[k] < 0 || b[k] >= n_seq) continue;
    const Seq s = load_seq(P, b[k], &ignore);
    int64_t rem = at[k] - before[k];
    int h = 0;
    while (h + 1 < H && rem >= s.work) rem -= s.work, ++h;
    hk[k] = h;
    // the last item that begins at or before rem: 32 candidates a round
    int lo = 0, hi = s.items;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, p = lo + lane * step;
      const unsigned ok = __ballot_sync(0xFFFFFFFFu, p < hi && work_before(s.off, P.G, p) <= rem);
      const int i = 31 - __clz(ok);              // lane 0's begins before rem
      hi = min(hi, lo + (i + 1) * step);
      lo += i * step;
    }
    const int64_t w0 = work_before(s.off, P.G, lo), w1 = work_before(s.off, P.G, lo + 1);
    const int n = tiles_to(s, P.G, 256 * ((int64_t)lo + 1));
    // the two CTAs on both sides of a cut come here with the same numbers
    x[k] = Pos{b[k], hk[k], lo, n > 0 ? int(float(rem - w0) / float(w1 - w0) * n + 0.5f) : 0};
    if (x[k].t >= n && n > 0) x[k] = next_item(P, s, x[k]);
  }
}

__device__ __forceinline__ uint32_t f16x2_of(uint32_t w) {      // codes in the low half of a word
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of_hi(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float pow2c(int e) { return pow2(min(max(e, -126), 127)); }
// How far, in log2, the score s of a page with scale byte k and factor c lies above
// the score sr of one with kr and cr: taken in units of the larger scale.
__device__ __forceinline__ float above(float s, int k, float c, float sr, int kr, float cr) {
  const int d = kr - k;
  return fmaf(-sr, pow2c(min(d, 0)), s * pow2c(min(-d, 0))) * (d > 0 ? cr : c);
}
// Codes that are NaN, to zero.
__device__ __forceinline__ uint32_t drop_nan4(uint32_t w) {
  const uint32_t m = __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  return w & ~m;
}
// Bounded wait of a lane, the long way of which is one function for all (little code:
// inlined, the warps waited for instructions; 256 us instead of 197 for 1,024 tokens
// behind 7,168) ...
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return uwait(bar, parity, abort, status);
}
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort, status);
}
// ... and of a whole warp, whose lanes all get the same answer.
__device__ __forceinline__ bool bar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)) || __all_sync(0xFFFFFFFFu, wait_long(bar, parity, abort, status));
}
// f16 operands, fp32 accumulator, both K-major.
constexpr uint32_t idesc_f16(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

// NG: groups of keys with a scale of their own in half a tile, 4, 2 or 1 for pages of
// 16, 32 or more.
template <int D, int NG>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(const __grid_constant__ Params P) {
  using Pl = Plan<D>;
  constexpr int NS = Pl::kStages, NR = Pl::kRaws, NB = Pl::kBoxes;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Info* info = reinterpret_cast<Info*>(smem + Pl::kInfo);
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + Pl::kBars);
  uint64_t* raw_empty = raw_full + NR;
  uint64_t* full = raw_empty + NR;
  uint64_t* empty = full + NS;
  uint64_t* q_full = empty + NS;       // [2]
  uint64_t* s_full = q_full + 2;       // [2][2]: query tile, half of the keys
  uint64_t* p_first = s_full + 4;      // [2]: the first half's probabilities are there, the second half's scores taken
  uint64_t* p_second = p_first + 2;    // [2]: the second half's probabilities
  uint64_t* h_done = p_second + 2;     // [2]: the first half's product
  uint64_t* o_full = h_done + 2;       // [2]
  uint64_t* o_free = o_full + 2;       // [2]
  uint64_t* fin = o_free + 2;          // [2]: a warp's MMAs at the end
  uint64_t* turn = fin + 2;            // [2]: the other MMA warp has issued
  uint64_t* it_full = turn + 2;        // [2]
  uint64_t* it_empty = it_full + 2;    // [2]
  uint64_t* info_full = it_empty + 2;  // [kSlots]
  uint64_t* v_done = info_full + kSlots;   // [kSlots]: the tile's values are converted
  Item* items = reinterpret_cast<Item*>(smem + Pl::kItems);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + Pl::kItems + 2 * 96);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);

  const ChunkArgs& a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = P.G, page = 1 << P.log2_page, H = a.c.n_kv_heads;
  int* status = a.status;

  if (tid == 0) {
    for (int i = 0; i < NR; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&empty[i], 2);     // both query tiles
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[2 * i], 1);
      mbar_init(&s_full[2 * i + 1], 1);
      mbar_init(&p_first[i], 4);
      mbar_init(&p_second[i], 4);
      mbar_init(&h_done[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&o_free[i], 4);
      mbar_init(&fin[i], 1);
      mbar_init(&turn[i], 1);
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 14);   // 2 MMA, 4 converter, 8 softmax warps
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&info_full[i], 1);
      mbar_init(&v_done[i], 4);
    }
    *abort = 0;
    mbar_fence_init();
  }
  if (warp == kWMma0) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t base = smem_addr(smem);
  const uint32_t q_s = base + Pl::kQ, ring_s = base + Pl::kRing, raw_s = base + Pl::kRawRing;

  // The t-th item of this CTA, copied out of its slot (whole warp; one lane
  // arrives when all have it).
  auto take_item = [&](int t, Item* it) {
    if (!bar_wait_warp(&it_full[t & 1], uint32_t(t >> 1) & 1u, abort, status)) return false;
    *it = items[t & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&it_empty[t & 1]);
    return it->n >= 0;
  };

  if (warp < 4) {
    if (warp == kWProd) {
      // ---- producer: items, and their pages -------------------------------------------------
      bool bad = false, ok = true;
      const int c = blockIdx.x;
      int n_cta;
      Pos place[2];
      find_places(P, c, &n_cta, place, &bad);
      Pos at = place[0];
      const Pos end = place[1];
      if (__any_sync(0xFFFFFFFFu, bad) && c == 0 && lane == 0 && status) atomicOr(status, MOE_DEV_INDEX_OOB);
      bool ignore;
      if (lane == 0) {
        Desc d{};
        if (at.t > 0) d.first = 1 | (same_item(at, end) ? 2 : 0);
        if (end.t > 0 && !(at.t > 0 && same_item(at, end))) {
          const Seq s = load_seq(P, end.b, &ignore);
          d.last = 1;
          d.q0 = s.q0;
          d.r0 = 256 * end.p;
          d.rows = int(min((int64_t)256, (int64_t)s.nq * G - d.r0));
          d.hk = end.hk;
        }
        P.desc[c] = d;
      }
      // item t of this CTA into its slot; false if there is none (nor any later)
      auto publish = [&](int t) {
        if (t >= 2 && !bar_wait_warp(&it_empty[t & 1], uint32_t((t >> 1) - 1) & 1u, abort, status)) {
          ok = false;
          return false;
        }
        const bool last = same_item(at, end);
        const bool have = at.b < a.n_seq && !(last && end.t <= at.t);
        if (have) {
          const Seq s = load_seq(P, at.b, &ignore);
          Item it;
          const int64_t rows = (int64_t)s.nq * G, r0 = 256 * (int64_t)at.p;
          const int n = tiles_to(s, G, r0 + 256), t1 = last ? end.t : n;
          it.n = t1 - at.t;
          it.t0 = at.t;
          it.r0 = int(r0);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int64_t f = r0 + j * kQT;
            it.rows[j] = int(min(max(rows - f, (int64_t)0), (int64_t)kQT));
            it.nkt[j] = it.rows[j] ? min(max(tiles_to(s, G, f + kQT) - at.t, 0), it.n) : 0;
          }
          it.b = at.b;
          it.hk = at.hk;
          it.q0 = s.q0;
          it.off = s.nk - s.nq;
          it.nk = s.nk;
          it.vmin = min(max(int(r0 / G) + 1 + it.off, 0), s.nk);
          it.slot = at.t > 0 ? 2 * c : t1 < n ? 2 * c + 1 : -1;
          if (lane == 0) items[t & 1] = it;
          at = last ? end : next_item(P, s, at);
          if (last) at.b = a.n_seq;
        } else if (lane == 0) {
          items[t & 1].n = -1;
        }
        __threadfence_block();
        __syncwarp();
        if (lane == 0) mbar_arrive(&it_full[t & 1]);
        return have;
      };
      const int per = page / 16;            // groups of a page
      const uint32_t bytes = uint32_t(page) * D;
      int r = 0, loads = 0, tiles = 0;      // raw slot, loads and key tiles so far
      bool more = publish(0);
      bool outside = false;
      for (int t = 0; ok && more; ++t) {
        const Item it = items[t & 1];
        more = it.n == 0 && publish(t + 1);    // else once its first tile is on its way
        // lane g < 8: group g's page (-1: none); scale bytes of a page
        auto load_page = [&](int i) {
          const int pos = (it.t0 + i) * kKT + 16 * lane;
          if (lane >= 8 || i >= it.n || pos >= it.nk) return -2;
          const int x = __ldg(a.table + (size_t)it.b * a.width + (pos >> P.log2_page));
          return x >= 0 && x < a.c.n_pages ? x : -1;
        };
        auto load_scales = [&](int pg) {
          if (pg < 0) return 0u;
          const size_t x = (size_t)pg * H + it.hk;
          return uint32_t(__ldg(a.c.k_scales + x)) | uint32_t(__ldg(a.c.v_scales + x)) << 8;
        };
        int pg = load_page(0), pg1 = load_page(1);
        uint32_t sc = load_scales(pg);
        for (int i = 0; i < it.n; ++i) {
          const int pg2 = load_page(i + 2);
          const uint32_t sc1 = load_scales(pg1);
          outside |= pg == -1;
          const int slot = tiles % kSlots;
          const unsigned none = __ballot_sync(0xFFFFFFFFu, pg == -1) & 0xFFu;
          if (lane == 0) info[slot].bad = none;     // the converters read it after the copies' barrier
          __threadfence_block();
          __syncwarp();
          const bool leads = lane < 8 && lane % per == 0 && pg >= 0;
          const uint32_t sum = bytes * __popc(__ballot_sync(0xFFFFFFFFu, leads));
          const size_t from = leads ? ((size_t)pg * H + it.hk) * bytes : 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (loads >= NR && !bar_wait_warp(&raw_empty[r], uint32_t(loads / NR - 1) & 1u, abort, status)) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&raw_full[r], sum);
            __syncwarp();
            if (leads)
              bulk_g2s(smem + Pl::kRawRing + r * Pl::kRaw + lane * (16 * D),
                       static_cast<const uint8_t*>(e ? a.c.v_codes : a.c.k_codes) + from, bytes, &raw_full[r]);
            ++loads;
            if (++r == NR) r = 0;
          }
          if (!ok) break;
          if (lane < 8) {
            reinterpret_cast<uint8_t*>(info[slot].k)[lane] = uint8_t(sc);
            info[slot].v[lane] = float(int(sc >> 8) - 127);
          }
          __threadfence_block();
          __syncwarp();
          if (lane == 0) mbar_arrive(&info_full[slot]);
          ++tiles;
          pg = pg1, pg1 = pg2, sc = sc1;
          if (i == 0) more = publish(t + 1);
          if (!ok) break;
        }
      }
      if (__any_sync(0xFFFFFFFFu, outside) && lane == 0 && status) atomicOr(status, MOE_DEV_INDEX_OOB);
      if (*abort) {   // copies in flight land before the CTA's shared memory goes away
        for (int i = loads > NR ? loads - NR : 0; i < loads; ++i) mbar_wait(&raw_full[i % NR], uint32_t(i / NR) & 1u, status);
      }
    } else if (warp == kWMma0 || warp == kWMma1) {
      // ---- MMA --------------------------------------------------------------------------
      constexpr uint32_t kTile16 = Pl::kTile >> 4, kBox16 = kBoxBytes >> 4;
      const int j = warp == kWMma1;
      const uint32_t id_s = idesc_f16(kQT, kKT / 2), id_o = idesc_f16(kQT, D) | (1u << 16);   // bit 16: B is MN-major
      const uint64_t dq = umma_desc_sw128(q_s + j * Pl::kTile);
      const uint64_t dk = umma_desc_sw128(ring_s), dv = umma_desc_mn_sw128(ring_s, kBoxBytes);
      const uint32_t ts = tmem + j * kKT, to = tmem + 256 + j * D;
      const uint32_t empty_s = smem_addr(empty);
      uint32_t st = 0, par = 0;                      // ring stage and phase
      uint32_t q_par = 0, p_par = 0, o_par = 1;      // phases of Q, of the probabilities, of O's release
      uint32_t turn_par = 1 - j;                     // tile 0 begins
      uint32_t g = 0;                                // columns of a key tile's first scores: g * 64
      bool ok = true, o_used = false;
      auto wait = [&](uint64_t* bar, uint32_t ph) { return bar_wait_warp(bar, ph, abort, status); };
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
      Item it;
      for (int t = 0; ok && take_item(t, &it); ++t) {
        const int n = __shfl_sync(0xFFFFFFFFu, it.n, 0);
        const int nkt = __shfl_sync(0xFFFFFFFFu, j ? it.nkt[1] : it.nkt[0], 0);
        if (n == 0) continue;
        if (!(ok = wait(&full[st], par))) break;
        if (nkt > 0) {
          if (!(ok = wait(&q_full[j], q_par))) break;
          q_par ^= 1;
          tc_fence_after();
          scores(st, 0, 64 * g);
          scores(st, 1, 64 - 64 * g);
        }
        next_stage(nkt == 0);
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
          } else {
            mbar_arrive_1(smem_addr(&turn[1 - j]));
          }
          if (i < nkt) g ^= 1;
        }
      }
      // every MMA has finished before tensor memory is freed
      umma_commit_1(smem_addr(&fin[j]));
      mbar_wait(&fin[j], 0, status);
    }
  } else if (warp < kWSoft) {
    // ---- converters -----------------------------------------------------------------------
    // A thread's vectors of 16 codes: a row's 64-channel box has four, 8 lanes take those of two rows, for heads of 128
    // of one box of the first and the other of the second, so that neither their loads nor their stores meet in a bank.
    constexpr int RPI = 32;             // rows between a thread's
    const int ct = tid - kWConv * 32, c4 = ct & 3, pair = (ct >> 2) & 1, row0 = ct >> 2;
    const uint32_t out0 = row0 * 128 + (((2 * c4) ^ (row0 & 7)) << 4), out1 = row0 * 128 + (((2 * c4 + 1) ^ (row0 & 7)) << 4);
    const uint32_t in0 = row0 * D + c4 * 16;
    int s = 0, r = 0, loads = 0, tiles = 0;
    bool ok = true;
    Item it;
    for (int t = 0; ok && take_item(t, &it); ++t) {
      for (int e = 0; e < 2 * it.n; ++e) {
        const int i = e >> 1;
        if (!bar_wait_warp(&raw_full[r], uint32_t(loads / NR) & 1u, abort, status) ||
            (loads >= NS && !bar_wait_warp(&empty[s], uint32_t(loads / NS - 1) & 1u, abort, status))) {
          ok = false;
          break;
        }
        const uint8_t* src = smem + Pl::kRawRing + r * Pl::kRaw + in0;
        uint8_t* dst = smem + Pl::kRing + s * Pl::kTile;
        const int k0 = (it.t0 + i) * kKT, slot = tiles % kSlots;
        const unsigned none = *reinterpret_cast<volatile uint32_t*>(&info[slot].bad);
        const bool masked = k0 + kKT > it.vmin, look = (e & 1) && (masked || none);
        bool found = false;
#pragma unroll 1
        for (int k = 0; k < 128 / RPI; ++k) {
          uint4 w[NB];
#pragma unroll
          for (int v = 0; v < NB; ++v) w[v] = *reinterpret_cast<const uint4*>(src + k * (RPI * D) + (NB == 2 ? (v ^ pair) * 64 : 0));
          if (look) {     // values that some row does not see: NaN to 0, all of what lies past the end or outside the cache
            const int row = row0 + k * RPI;
            const bool gone = row >= it.nk - k0 || (none >> (row / 16)) & 1;
#pragma unroll
            for (int v = 0; v < NB; ++v) {
              if (gone) w[v] = make_uint4(0, 0, 0, 0);
              if (masked && (any_nan4(w[v].x) || any_nan4(w[v].y) || any_nan4(w[v].z) || any_nan4(w[v].w))) {
                found = true;
                w[v].x = drop_nan4(w[v].x);
                w[v].y = drop_nan4(w[v].y);
                w[v].z = drop_nan4(w[v].z);
                w[v].w = drop_nan4(w[v].w);
              }
            }
          }
#pragma unroll
          for (int v = 0; v < NB; ++v) {
            uint8_t* o = dst + k * (RPI * 128) + (NB == 2 ? (v ^ pair) * kBoxBytes : 0);
            *reinterpret_cast<uint4*>(o + out0) =
                make_uint4(f16x2_of(w[v].x), f16x2_of_hi(w[v].x), f16x2_of(w[v].y), f16x2_of_hi(w[v].y));
            *reinterpret_cast<uint4*>(o + out1) =
                make_uint4(f16x2_of(w[v].z), f16x2_of_hi(w[v].z), f16x2_of(w[v].w), f16x2_of_hi(w[v].w));
          }
        }
        if (look) found = __any_sync(0xFFFFFFFFu, found);
        if ((e & 1) && lane == 0) info[slot].poison[warp - kWConv] = found;
        fence_async_smem();
        __threadfence_block();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&full[s]);
          mbar_arrive(&raw_empty[r]);
          if (e & 1) mbar_arrive(&v_done[tiles % kSlots]);
        }
        tiles += e & 1;
        ++loads;
        if (++s == NS) s = 0;
        if (++r == NR) r = 0;
      }
    }
  } else {
    // ---- softmax ------------------------------------------------------------------------
    const int j = (warp - kWSoft) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    const uint32_t ts = tmem + lanes + j * kKT, to = tmem + lanes + 256 + j * D;
    int st = 0;                        // ring stage of the next key tile's keys
    int nsf = 0, nof = 0, tiles = 0;   // scores and outputs awaited; key tiles of all items
    bool ok = true;
    Item it;
    for (int t = 0; ok && take_item(t, &it); ++t) {
      const int nkt = it.nkt[j], rows = it.rows[j];
      const int64_t grow = (int64_t)it.r0 + j * kQT + row;       // row of the sequence and head
      const int tok = int(grow / G), head = it.hk * G + int(grow % G);
      const int vis = min(max(tok + it.off + 1, 0), it.nk);
      const int vis_w = __shfl_sync(0xFFFFFFFFu, vis, 0);        // the warp's fewest
      int ce = P.ce;
      if (nkt > 0) {
        // this row of Q to f16; its tile's products of the last item have been read
        uint4 w[D / 8];
        const __nv_bfloat16* q = a.q + (int64_t)(it.q0 + tok) * a.q_ts + (int64_t)head * a.q_hs;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) w[x] = row < rows ? *reinterpret_cast<const uint4*>(q + x * 8) : make_uint4(0, 0, 0, 0);
        uint32_t m2 = 0;
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
          m2 = __vmaxu2(__vmaxu2(m2, __vmaxu2(w[x].x & 0x7FFF7FFFu, w[x].y & 0x7FFF7FFFu)),
                        __vmaxu2(w[x].z & 0x7FFF7FFFu, w[x].w & 0x7FFF7FFFu));
        const uint32_t top = max(m2 & 0xFFFFu, m2 >> 16);
        const int ex = min(max(int(top >> 7) - 127, -112), 127);
        ce += ex - 14;
        // 2^(14 - ex). A row that is not finite becomes NaN as a whole, and so do the scores of what it sees: those of an
        // infinity may all be -inf, which a mask leaves too.
        const float f = __uint_as_float((uint32_t(141 - ex) << 23) | (P.negate ? 0x80000000u : 0u) | (top >= 0x7F80u ? 0x7FC00000u : 0u));
        const uint32_t dst = row * 128;
        uint8_t* qs = smem + Pl::kQ + j * Pl::kTile;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          const uint32_t u[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
          uint32_t h[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) h[y] = f16x2_bits(bf16_lo(u[y]) * f, bf16_hi(u[y]) * f);
          *reinterpret_cast<uint4*>(qs + (x / 8) * kBoxBytes + dst + (((x % 8) ^ (row & 7)) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[j]);
      }
      // references: score sr of a page with scale byte kr (none yet: have = false), its factor cr, so the score m in
      // log2; value reference rv above m; sum l in units of 2^m, O in units of 2^(m + rv - 8)
      bool have = false;
      float sr = 0.0f, cr = 0.0f, m = 0.0f, l = 0.0f, rv = 0.0f;
      int kr = 0;              // of a scale byte below all, so that above() takes scores as they are
      unsigned bad = 0;                // masked tiles with NaN (an item's rows span at most 256 tokens)
      for (int i = 0; i < nkt; ++i) {
        const int k0 = (it.t0 + i) * kKT, slot = (tiles + i) % kSlots;
        const uint32_t slot_ph = uint32_t((tiles + i) / kSlots) & 1u;
        const bool masked = k0 + kKT > it.vmin;
        const uint32_t ph = uint32_t(nsf) & 1u, ta = ts + 64 * ph, tb = ts + 64 - 64 * ph;
        ++nsf;
        const int n_vis = vis - k0;
        const bool cut = k0 + kKT > vis_w;   // some lane of the warp does not see the whole tile
        uint32_t s[2][32];
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (!bar_wait(&s_full[2 * j + half], ph, abort, status)) ok = false;
          // complete by now, and for this tile: a warp that had nothing to do for an item is far ahead of its ring
          if (!bar_wait(&info_full[slot], slot_ph, abort, status)) ok = false;
          const uint32_t kb4 = info[slot].k[half];
          const unsigned none = info[slot].bad;
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
          if (cut || none) {   // places that this row does not see
            uint64_t seen = n_vis - 64 * half >= 64 ? ~0ull : n_vis > 64 * half ? (1ull << (n_vis - 64 * half)) - 1 : 0ull;
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if ((none >> (4 * half + g)) & 1) seen &= ~(0xFFFFull << (16 * g));
            const uint32_t seen2[2] = {uint32_t(seen), uint32_t(seen >> 32)};
#pragma unroll
            for (int y = 0; y < 64; ++y)
              if (!((seen2[y / 32] >> (y % 32)) & 1)) s[y / 32][y % 32] = 0xFF800000u;
          }
          // a group of keys: factor of its scores, its largest score, how far that is above the reference
          constexpr int GK = 64 / NG, GB = 4 / NG;      // keys, scale bytes of a group
          float ck[NG], mx[NG], d[NG];
          int kb[NG];
          float ve[NG];
          float dm = -INFINITY, dy = -INFINITY;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            kb[g] = int(kb4 >> (8 * GB * g)) & 255;
            ve[g] = info[slot].v[4 * half + GB * g];
            float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
            for (int z = g * GK; z < (g + 1) * GK; z += 16) {
              uint32_t* x = &s[z / 32][z % 32];
#pragma unroll
              for (int y = 0; y < 16; y += 4) {
                a0 = max3(a0, __uint_as_float(x[y]), __uint_as_float(x[y + 1]));
                a1 = max3(a1, __uint_as_float(x[y + 2]), __uint_as_float(x[y + 3]));
              }
            }
            mx[g] = fmaxf(a0, a1);
            ck[g] = __uint_as_float(__float_as_uint(P.cm) + (uint32_t(min(max(ce + kb[g] - 127, -100), 126)) << 23));
          }
          // Short pages: whether one's largest lies too far above the references is seen from fp32 differences first,
          // which tell it to 2^-6 while a reference is not far.
          bool look = true;
          if (NG > 1) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              d[g] = fmaf(mx[g], ck[g], -m);
              dm = fmaxf(dm, d[g]);
              dy = fmaxf(dy, d[g] + ve[g]);
            }
            look = __any_sync(0xFFFFFFFFu, !have || fabsf(m) > kFar || dm > kRaiseSum || dy > rv + kRaiseOut);
            dm = dy = -INFINITY;
          }
          bool raise = false;
          if (look) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              d[g] = above(mx[g], kb[g], ck[g], sr, kr, cr);
              dm = fmaxf(dm, d[g]);
              dy = fmaxf(dy, d[g] + ve[g]);
            }
            raise = have ? dm > kRaiseSum || dy > rv + kRaiseOut : dm > -INFINITY;
          }
          if (look && __any_sync(0xFFFFFFFFu, raise)) {
            float fl = 1.0f, fo = 1.0f;
            if (raise) {
              float top = have ? 0.0f : -INFINITY;     // of the new reference above the old one
              float nsr = sr, ncr = cr;
              int nkr = kr;
#pragma unroll
              for (int g = 0; g < NG; ++g)
                if (d[g] > top) top = d[g], nsr = mx[g], ncr = ck[g], nkr = kb[g];
              sr = nsr, cr = ncr, kr = nkr;
              m = sr * cr;
              float y = have ? rv - top : -INFINITY;
#pragma unroll
              for (int g = 0; g < NG; ++g) y = fmaxf(y, above(mx[g], kb[g], ck[g], sr, kr, cr) + ve[g]);
              const float nrv = ceilf(fminf(fmaxf(y, -1000.0f), 1000.0f));
              fl = have ? pf_ex2(-top) : 0.0f;
              fo = have ? pf_ex2(rv - nrv - top) : 0.0f;
              rv = nrv;
              have = true;
            }
            l *= fl;
            // what is in O: the earlier tiles' products, which have finished
            // when this tile's second scores have, since these were issued after
            // them; in the second half this tile's first product too, after
            // which the next tile's first scores are issued
            if (half == 1 || i > 0) {
              if (!bar_wait(half ? &h_done[j] : &s_full[2 * j + 1], ph, abort, status)) ok = false;
              tc_fence_after();
#pragma unroll 1
              for (int z = 0; z < D; z += 16) {
                uint32_t o[16];
                tmem_ld16(to + z, o);
#pragma unroll
                for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * fo);
                tmem_st16(to + z, o);
              }
            }
          }
          const bool far = fabsf(m) > kFar;
          const float ref = far ? 0.0f : m;
          if (__any_sync(0xFFFFFFFFu, far)) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              const int dk = kr - kb[g];     // as above()
              const float fs = far ? -sr * pow2c(min(dk, 0)) : 0.0f, fx = far ? pow2c(min(-dk, 0)) : 1.0f;
              if (far && dk > 0) ck[g] = cr;
#pragma unroll
              for (int y = g * GK; y < (g + 1) * GK; ++y)
                s[y / 32][y % 32] = __float_as_uint(fmaf(__uint_as_float(s[y / 32][y % 32]), fx, fs));
            }
          }
          // A probability comes out in the units of O, 2^t times itself; what that makes of 16 at most is 2^15 at most,
          // and below t = -60 it is 0 in f16 either way. The sum takes the 2^t back.
          constexpr int SB = GK < 32 ? GK : 32;         // keys of one group in a row
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint32_t pb[16];
#pragma unroll
            for (int u = 0; u < 32; u += SB) {
              const int g = (32 * b + u) / GK;
              const float t = fminf(fmaxf(ve[g] - rv + kPBias, -60.0f), 126.0f);
              const uint64_t c2 = pack2(ck[g], ck[g]), r2 = pack2(t - ref, t - ref);
              uint32_t* x = &s[b][u];
              float e[SB];
#pragma unroll
              for (int y = 0; y < SB; y += 2)
                unpack2(fma2(pack2(__uint_as_float(x[y]), __uint_as_float(x[y + 1])), c2, r2), e[y], e[y + 1]);
#pragma unroll
              for (int y = 0; y < SB; ++y) e[y] = pf_ex2(e[y]);
#pragma unroll
              for (int y = 0; y < SB; y += 2) pb[(u + y) / 2] = f16x2_bits(e[y], e[y + 1]);
              uint64_t sum[4];
#pragma unroll
              for (int z = 0; z < 4; ++z) sum[z] = add2(pack2(e[2 * z], e[2 * z + 1]), pack2(e[2 * z + 8], e[2 * z + 9]));
#pragma unroll
              for (int y = 16; y < SB; y += 8)
#pragma unroll
                for (int z = 0; z < 4; ++z) sum[z] = add2(sum[z], pack2(e[y + 2 * z], e[y + 2 * z + 1]));
              float a0, a1;
              unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), a0, a1);
              l = fmaf(a0 + a1, pf_ex2(-t), l);
            }
            tmem_st16(ta + 32 * half + 16 * b, pb);
          }
          if (half == 0) tmem_wait_st();
        }
        if (masked) {
          if (!bar_wait(&v_done[slot], slot_ph, abort, status)) ok = false;
          if (*reinterpret_cast<volatile uint32_t*>(info[slot].poison)) bad |= 1u << (it.t0 + i - it.vmin / kKT);
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
      tiles += it.n;
      const int st_end = (st + 2 * (it.n - nkt)) % NS;
      if (rows == 0) {
        st = st_end;
        continue;
      }
      const bool mine = row < rows;
      if (nkt > 0) {
        if (!bar_wait_warp(&o_full[j], uint32_t(nof++) & 1u, abort, status)) break;
        if (warp == kWSoft + 4 * j && lane == 0) mbar_arrive(&empty[st == 0 ? NS - 1 : st - 1]);
        tc_fence_after();
      }
      const int64_t orow = (int64_t)(it.q0 + tok) * a.n_heads + head;
      __nv_bfloat16* out = a.out + orow * D;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int ov = int(rv) - int(kPBias);
      const float f0 = pow2c(ov >> 1), f1 = pow2c(ov - (ov >> 1));
      float4* part = P.parts + (size_t)(it.slot < 0 ? 0 : it.slot) * (256 * (D / 4 + 1)) + j * kQT + row;
#pragma unroll 1
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
          for (int k = k0; k < min(k0 + kKT, vis); ++k) {
            const int pg = __ldg(a.table + (size_t)it.b * a.width + (k >> P.log2_page));
            if (pg < 0 || pg >= a.c.n_pages) continue;
            const uint4* v = reinterpret_cast<const uint4*>(
                static_cast<const uint8_t*>(a.c.v_codes) + ((((size_t)pg * H + it.hk) << P.log2_page) + (k & (page - 1))) * D + x);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint4 c4 = v[y];
              const uint32_t c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
              for (int z = 0; z < 16; ++z)
                if (((c[z >> 2] >> (8 * (z & 3))) & 0x7Fu) == 0x7Fu) o[16 * y + z] = 0x7FC00000u;
            }
          }
        }
        if (it.slot >= 0) {
          if (mine) {
#pragma unroll
            for (int y = 0; y < 8; ++y)
              part[(size_t)(x / 4 + y) * 256] = make_float4(__uint_as_float(o[4 * y]), __uint_as_float(o[4 * y + 1]),
                                                            __uint_as_float(o[4 * y + 2]), __uint_as_float(o[4 * y + 3]));
          }
        } else if (mine) {
          uint32_t b[16];
#pragma unroll
          for (int y = 0; y < 16; ++y)
            b[y] = l == 0.0f ? 0u : bf16x2_bits(__uint_as_float(o[2 * y]) * inv * f0 * f1, __uint_as_float(o[2 * y + 1]) * inv * f0 * f1);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            *reinterpret_cast<uint4*>(out + x + y * 8) = make_uint4(b[4 * y], b[4 * y + 1], b[4 * y + 2], b[4 * y + 3]);
        }
      }
      st = st_end;
      if (mine) {
        if (it.slot >= 0)
          part[(size_t)(D / 4) * 256] = make_float4(sr, cr, l, __int_as_float((int(rv) << 8) | kr));
        else if (a.lse)
          a.lse[orow] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2f;
      }
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

// Joins the parts of an item that was cut, in order of position: block (c, x)
// channels 4 x .. 4 x + 3 of the item that begins in CTA c and ends in a later one,
// thread = row, so parts are read coalesced over the rows.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const Params P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, x = blockIdx.y, row = threadIdx.x;
  const Desc d = P.desc[c];
  if (!d.last) return;
  constexpr size_t kSlot = 256 * (D / 4 + 1);
  int last = c + 1;                // the last CTA with a part
  for (unsigned ends = 0; !ends; last += ends ? __ffs(ends) - 1 : 32) {
    const int i = last + (threadIdx.x & 31);
    ends = __ballot_sync(0xFFFFFFFFu, i > int(gridDim.x) || !(P.desc[i].first & 2));
  }
  if (row >= d.rows) return;
  auto slot = [&](int k) { return P.parts + (size_t)(k == c ? 2 * c + 1 : 2 * k) * kSlot + row; };
  // the parts one after another, two on their way at once (with eight the code is longer, and 37 tokens took 3 us
  // more); so far: reference sr, kr, cr, sum l in its units, outputs o
  // and their reference rm above it
  float sr = 0.0f, cr = 0.0f, l = 0.0f, rm = -INFINITY;
  int kr = 0;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k0 = c; k0 <= last; k0 += 2) {
    float4 h[2], v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      h[i] = k0 + i <= last ? slot(k0 + i)[(size_t)(D / 4) * 256] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      v[i] = k0 + i <= last ? slot(k0 + i)[(size_t)x * 256] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (h[i].z == 0.0f) continue;            // nothing seen there
      const int kb = __float_as_int(h[i].w) & 255, rv = __float_as_int(h[i].w) >> 8;
      float up = l == 0.0f ? 0.0f : above(h[i].x, kb, h[i].y, sr, kr, cr);
      float f = 1.0f;                          // of what is there
      if (l == 0.0f || up > 0.0f) {
        f = l == 0.0f ? 0.0f : pf_ex2(-up);
        rm -= up;
        sr = h[i].x, kr = kb, cr = h[i].y;
        up = 0.0f;
      }
      l = fmaf(h[i].z, pf_ex2(up), l * f);
      const float r = up + float(rv), rn = fmaxf(rm, r), fo = rm == -INFINITY ? 0.0f : pf_ex2(rm - rn), fv = pf_ex2(r - rn);
      o.x = fmaf(v[i].x, fv, o.x * fo), o.y = fmaf(v[i].y, fv, o.y * fo);
      o.z = fmaf(v[i].z, fv, o.z * fo), o.w = fmaf(v[i].w, fv, o.w * fo);
      rm = rn;
    }
  }
  const float m = sr * cr;
  const int G = P.G, r = d.r0 + row;
  const int64_t orow = (int64_t)(d.q0 + r / G) * P.a.n_heads + d.hk * G + r % G;
  const float inv = 1.0f / l, f = pf_ex2(0.5f * (rm - kPBias));
  uint2 w = make_uint2(0, 0);
  if (l != 0.0f) w = make_uint2(bf16x2_bits(o.x * inv * f * f, o.y * inv * f * f), bf16x2_bits(o.z * inv * f * f, o.w * inv * f * f));
  *reinterpret_cast<uint2*>(P.a.out + orow * D + 4 * x) = w;
  if (x == 0 && P.a.lse) P.a.lse[orow] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2f;
}

template <int D, int NG>
int launch_chunk(const Params& P, int grid, const DeviceInfo& di, cudaStream_t s) {
  constexpr uint32_t smem = Plan<D>::kTotal;
  if (smem > di.smem_optin) return MOE_ERR_UNSUPPORTED_SHAPE;
  MOE_CUDA_TRY(cudaFuncSetAttribute(chunk_kernel<D, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)));
  chunk_kernel<D, NG><<<grid, kThreads, smem, s>>>(P);
  if (grid > 1) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid - 1, D / 4);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute pdl;
    pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &pdl;
    cfg.numAttrs = 1;
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, chunk_join_kernel<D>, P));
  }
  return launch_status();
}

size_t desc_bytes(const DeviceInfo& di) { return round_up(size_t(di.sm_count) * sizeof(Desc), 256); }

}  // namespace

size_t attn_chunk_ws_bytes(const moe_kv_cache& c, int, int, int, const DeviceInfo& di) {
  return desc_bytes(di) + size_t(2 * di.sm_count) * 256 * (c.head_dim + 4) * 4;
}

int launch_attn_chunk(const ChunkArgs& a, const DeviceInfo& di, cudaStream_t s) {
  Params P{};
  P.a = a;
  P.G = a.n_heads / a.c.n_kv_heads;
  while ((1 << P.log2_page) < a.c.page_size) ++P.log2_page;
  const double c = fabs(double(a.scale)) * 1.4426950408889634;      // beyond fp32 for the largest scales
  if (c > 0.0) {
    int e;
    P.cm = float(2.0 * frexp(c, &e));
    P.ce = e - 1;
  } else {   // every score counts the same
    P.cm = 1.0f;
    P.ce = -1000;
  }
  P.negate = a.scale < 0.0f;
  // work is counted in 64 bits: items times positions and heads of a group
  const double items = double(a.total_q) * P.G / 256 + a.n_seq;
  if (items * a.c.n_kv_heads * P.G * (double(a.width) * a.c.page_size + 1024) > 4e18) return MOE_ERR_UNSUPPORTED_SHAPE;
  P.desc = static_cast<Desc*>(a.ws);
  P.parts = reinterpret_cast<float4*>(static_cast<char*>(a.ws) + desc_bytes(di));
  const int ng = a.c.page_size == 16 ? 4 : a.c.page_size == 32 ? 2 : 1;
  if (a.c.head_dim == 128)
    return ng == 4 ? launch_chunk<128, 4>(P, di.sm_count, di, s)
                   : ng == 2 ? launch_chunk<128, 2>(P, di.sm_count, di, s) : launch_chunk<128, 1>(P, di.sm_count, di, s);
  return ng == 4 ? launch_chunk<64, 4>(P, di.sm_count, di, s)
                 : ng == 2 ? launch_chunk<64, 2>(P, di.sm_count, di, s) : launch_chunk<64, 1>(P, di.sm_count, di, s);
}

}  // namespace moe
