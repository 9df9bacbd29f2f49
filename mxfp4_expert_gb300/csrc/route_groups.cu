// Routing by groups: scores (sigmoid or softmax of the logits), a bias that only
// the selection sees, the best groups of experts, the k best experts in them,
// weights from the scores without the bias.
//
// One warp per token, its keys in registers. Lane (g, u) = lane / L, lane % L
// holds experts g * size + u, g * size + u + L, ... of group g (L = 32 / the
// power of two not below the number of groups), so a group's best keys are
// merged by log2 L shuffles and a group is dropped by its own lanes.
//
// Selection must not hang on the rounding of an exponential: with a bias two
// keys may lie closer than fp32 tells. A score therefore is a pair of fp32
// numbers (high, low; about 2^-42 of it), keys are compared by both, and without
// a bias the logits themselves are, of which the scores are monotone. The
// exponential: exp(x) = 2^n exp(j/32) exp(r), |r| <= 1/64, exp(j/32) from a table
// of pairs that the lanes hold (P. T. P. Tang, "Table-driven implementation of the
// exponential function", 1989), exp(r) its Taylor series, of which the terms up
// to r^2 are pairs.
#include <math.h>

#include "block.h"
#include "common.cuh"
#include "topk.cuh"

namespace moe {
namespace {

constexpr int kGrpWarps = 4;
constexpr float kFmax = 3.4028235e38f;

struct F2 {      // hi + lo, |lo| <= half a step of hi
  float hi, lo;
};
__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}
__device__ __forceinline__ F2 quick_sum(float a, float b) {   // |a| >= |b|, or a = 0
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ F2 add(const F2& a, const F2& b) {
  const F2 s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
  const F2 u = quick_sum(s.hi, __fadd_rn(s.lo, t.hi));
  return quick_sum(u.hi, __fadd_rn(u.lo, t.lo));
}
__device__ __forceinline__ F2 mul(const F2& a, const F2& b) {
  const float p = __fmul_rn(a.hi, b.hi), e = fmaf(a.hi, b.hi, -p);
  return quick_sum(p, fmaf(a.hi, b.lo, fmaf(a.lo, b.hi, e)));
}
// a / b, b normal
__device__ __forceinline__ F2 div(const F2& a, const F2& b) {
  const float q = __fdiv_rn(a.hi, b.hi);
  float r = fmaf(-q, b.hi, a.hi);
  r = __fadd_rn(r, fmaf(-q, b.lo, a.lo));
  return quick_sum(q, __fdiv_rn(r, b.hi));
}
__device__ __forceinline__ bool less(const F2& a, const F2& b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }

// exp(j / 32) for j = -12 .. 12, to 2^-50: high and low parts, made at compile time.
struct ExpTable {
  float hi[32], lo[32];
};
constexpr double exp_taylor(double x) {
  double s = 1.0, t = 1.0;
  for (int i = 1; i < 24; ++i) t *= x / i, s += t;
  return s;
}
constexpr ExpTable make_exp_table() {
  ExpTable t{};
  for (int i = 0; i < 32; ++i) {
    const double v = i < 25 ? exp_taylor((i - 12) / 32.0) : 1.0;
    t.hi[i] = float(v);
    t.lo[i] = float(v - double(float(v)));
  }
  return t;
}
__constant__ const ExpTable kExpTable = make_exp_table();

// exp(x) for x = hi + lo <= 0 (whole warp; tab: entry `lane` of the table). Below
// 2^-100 it loses low bits, below 2^-126 it is 0.
__device__ __forceinline__ F2 exp_pair(const F2& x, const F2& tab) {
  const float n = rintf(fmaxf(x.hi, -200.0f) * 1.4426950408889634f);
  // log 2 in three parts, the first of 12 bits: n times it is exact
  constexpr double kLog2 = 0.693147180559945309417232;
  constexpr float c1 = 0.693115234375f, c2 = float(kLog2 - 0.693115234375),
                  c3 = float(kLog2 - 0.693115234375 - double(float(kLog2 - 0.693115234375)));
  F2 r = two_sum(fmaf(-n, c1, x.hi), x.lo);          // the product is exact, and so is the difference
  const float p = __fmul_rn(n, c2), e = fmaf(n, c2, -p);
  r = add(r, {-p, -fmaf(n, c3, e)});
  const float jf = fminf(fmaxf(rintf(r.hi * 32.0f), -12.0f), 12.0f);
  r = two_sum(fmaf(jf, -0.03125f, r.hi), r.lo);
  const int j = int(jf) + 12;
  const F2 t{__shfl_sync(0xFFFFFFFFu, tab.hi, j), __shfl_sync(0xFFFFFFFFu, tab.lo, j)};
  // exp(r) - 1
  const float q = __fmul_rn(r.hi, r.hi), qe = fmaf(r.hi, r.hi, -q) + 2.0f * r.hi * r.lo;
  const float rest = q * r.hi * fmaf(r.hi, fmaf(r.hi, 1.0f / 120.0f, 1.0f / 24.0f), 1.0f / 6.0f);
  F2 v = two_sum(r.hi, 0.5f * q);
  v = quick_sum(v.hi, v.lo + (r.lo + 0.5f * qe + rest));
  v = add({1.0f, 0.0f}, v);
  v = mul(v, t);
  const int ni = int(n);
  if (ni < -140) return {0.0f, 0.0f};
  const float f1 = exp2i(ni / 2), f2 = exp2i(ni - ni / 2);
  return {v.hi * f1 * f2, v.lo * f1 * f2};
}

// PL: experts a lane holds.
template <int PL>
__global__ void __launch_bounds__(kGrpWarps * 32) route_groups_kernel(const GroupArgs a, int L) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kGrpWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int size = a.E / a.n_groups, g = lane / L, u = lane % L;
  const F2 tab{kExpTable.hi[lane], kExpTable.lo[lane]};
  const float* row = a.logits + (size_t)t * a.E;
  auto expert = [&](int j) { return g * size + u + j * L; };
  auto held = [&](int j) { return g < a.n_groups && u + j * L < size; };

  float l[PL];
  bool nan[PL];
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    l[j] = held(j) ? row[expert(j)] : -kFmax;
    nan[j] = isnan(l[j]);
    l[j] = nan[j] ? -kFmax : fminf(fmaxf(l[j], -kFmax), kFmax);
  }
  const bool scores = a.bias || a.best > 1 || a.softmax;   // else only those of the selected
  F2 s[PL];
  float top_l = 0.0f;
  F2 sum{0.0f, 0.0f};
  if (a.softmax) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < PL; ++j) m = max(m, held(j) && !nan[j] ? rank_key(l[j]) : 0u);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    top_l = m ? rank_value(m) : 0.0f;
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      s[j] = exp_pair(two_sum(l[j], -top_l), tab);
      if (nan[j] || !held(j)) s[j] = {0.0f, 0.0f};
      sum = add(sum, s[j]);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const F2 other{__shfl_xor_sync(0xFFFFFFFFu, sum.hi, o), __shfl_xor_sync(0xFFFFFFFFu, sum.lo, o)};
      // the same two numbers in the same order in both lanes
      sum = (lane & o) ? add(other, sum) : add(sum, other);
    }
    if (sum.hi == 0.0f) sum = {1.0f, 0.0f};
  }
  auto sigmoid = [&](float x) {
    const F2 e = exp_pair({-fabsf(x), 0.0f}, tab);
    const F2 d = add({1.0f, 0.0f}, e);
    return x >= 0.0f ? div({1.0f, 0.0f}, d) : div(e, d);
  };
  if (scores) {
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      s[j] = a.softmax ? div(s[j], sum) : sigmoid(l[j]);
      if (nan[j]) s[j] = {0.0f, 0.0f};
    }
  }
  // keys: high part 0 stands for "no candidate"
  uint32_t kh[PL], kl[PL];
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    F2 key{l[j], 0.0f};
    if (a.bias) {
      const float b = held(j) ? a.bias[expert(j)] : 0.0f;
      key = add({b, 0.0f}, s[j]);
      if (!(fabsf(b) <= kFmax)) key = {b, 0.0f};
      if (nan[j]) key = {-INFINITY, 0.0f};
    }
    kh[j] = held(j) ? rank_key(nan[j] ? -INFINITY : key.hi) : 0u;
    kl[j] = kh[j] ? rank_key(key.lo) : 0u;
  }

  if (a.top < a.n_groups) {
    // a group's score: its best key, or the sum of its two best (without a bias, of their scores)
    F2 b0{-INFINITY, 0.0f}, b1{-INFINITY, 0.0f};
    auto take = [&](const F2& v) {
      if (less(b0, v)) b1 = b0, b0 = v;
      else if (less(b1, v)) b1 = v;
    };
#pragma unroll
    for (int j = 0; j < PL; ++j)
      if (kh[j]) take(a.best > 1 && !a.bias ? (nan[j] ? F2{-INFINITY, 0.0f} : s[j]) : F2{rank_value(kh[j]), rank_value(kl[j])});
    for (int o = 1; o < L; o <<= 1) {
      const F2 o0{__shfl_xor_sync(0xFFFFFFFFu, b0.hi, o), __shfl_xor_sync(0xFFFFFFFFu, b0.lo, o)};
      const F2 o1{__shfl_xor_sync(0xFFFFFFFFu, b1.hi, o), __shfl_xor_sync(0xFFFFFFFFu, b1.lo, o)};
      take(o0);
      take(o1);
    }
    F2 score = b0;
    if (a.best > 1) score = fabsf(b0.hi) <= kFmax && fabsf(b1.hi) <= kFmax ? add(b0, b1) : F2{b0.hi + b1.hi, 0.0f};
    int better = 0;
    for (int i = 0; i < a.n_groups; ++i) {
      const F2 v{__shfl_sync(0xFFFFFFFFu, score.hi, i * L), __shfl_sync(0xFFFFFFFFu, score.lo, i * L)};
      better += less(score, v) || (!less(v, score) && i < g);
    }
    if (better >= a.top) {
#pragma unroll
      for (int j = 0; j < PL; ++j) kh[j] = 0u;
    }
  }

  // the k best keys, equal ones by the lower expert
  uint32_t bh, bl;
  int bj;
  auto local_best = [&]() {
    bh = bl = 0u;
    bj = 0;
#pragma unroll
    for (int j = 0; j < PL; ++j)
      if (kh[j] > bh || (kh[j] == bh && kh[j] && kl[j] > bl)) bh = kh[j], bl = kl[j], bj = j;
  };
  local_best();
  int my_e = 0;
  float my_s = 0.0f, my_l = 0.0f;
  for (int r = 0; r < a.k; ++r) {
    const uint32_t h = __reduce_max_sync(0xFFFFFFFFu, bh);
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, bh == h ? bl : 0u);
    const int mine = bh == h && bl == lo ? expert(bj) : 0x7FFFFFFF;
    const int e = __reduce_min_sync(0xFFFFFFFFu, mine);
    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, mine == e)) - 1;
    float sv = 0.0f, lv = 0.0f;
    if (lane == src) {
#pragma unroll
      for (int j = 0; j < PL; ++j)
        if (j == bj) {
          if (scores) sv = s[j].hi;
          lv = nan[j] ? -INFINITY : l[j];
          kh[j] = 0u;
        }
      local_best();
    }
    sv = __shfl_sync(0xFFFFFFFFu, sv, src);
    lv = __shfl_sync(0xFFFFFFFFu, lv, src);
    if (lane == r) my_e = e, my_s = sv, my_l = lv;
  }
  if (!scores) {
    const F2 v = sigmoid(fmaxf(my_l, -kFmax));
    my_s = v.hi;
  }
  if (lane >= a.k || my_l == -INFINITY) my_s = 0.0f;
  float all = my_s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  if (lane < a.k) {
    a.idx[(size_t)t * a.k + lane] = my_e;
    a.w[(size_t)t * a.k + lane] = (a.renorm ? my_s / (all + 1e-20f) : my_s) * a.scale;
  }
}

int lanes_of(int n_groups) {
  int p = 1;
  while (p < n_groups) p *= 2;
  return 32 / p;
}

}  // namespace

bool groups_ok(int E, int k, int n_groups, int top, int best) {
  if (E > 1024 || k > 32 || n_groups > 32 || E % n_groups) return false;
  const int size = E / n_groups;
  return size >= best && k <= size * top && (size + lanes_of(n_groups) - 1) / lanes_of(n_groups) <= 32;
}

int launch_route_groups(const GroupArgs& a, cudaStream_t s) {
  const int L = lanes_of(a.n_groups), pl = (a.E / a.n_groups + L - 1) / L;
  const int grid = (a.T + kGrpWarps - 1) / kGrpWarps;
#define MOE_GRP_CASE(P)                                                 \
  route_groups_kernel<P><<<grid, kGrpWarps * 32, 0, s>>>(a, L);         \
  break;
  switch (pl <= 1 ? 1 : pl <= 2 ? 2 : pl <= 4 ? 4 : pl <= 8 ? 8 : pl <= 16 ? 16 : 32) {
    case 1: MOE_GRP_CASE(1)
    case 2: MOE_GRP_CASE(2)
    case 4: MOE_GRP_CASE(4)
    case 8: MOE_GRP_CASE(8)
    case 16: MOE_GRP_CASE(16)
    default: MOE_GRP_CASE(32)
  }
#undef MOE_GRP_CASE
  return launch_status();
}

}  // namespace moe
