// Routing by groups: scores (sigmoid or softmax of the logits), a bias that only
// the selection sees, the best groups of experts, the k best experts in them,
// weights from the scores without the bias. One token, by a warp: for the routing
// kernel and for the layer's single launch.
//
// The keys are in registers. Lane (g, u) = lane / L, lane % L
// holds experts g * size + u, g * size + u + L, ... of group g (L = 32 / the
// power of two not below the number of groups), so a group's best keys are
// merged by log2 L shuffles and a group is dropped by its own lanes.
//
// Selection must not hang on the rounding of an exponential: with a bias two
// keys may lie closer than fp32 tells. Keys are taken in fp32 first; what lies so
// close to a neighbour in rank, or to the cut, that their errors could turn it
// (doubt()) is ranked once more by pairs of fp32 numbers (high, low; about 2^-42 of a
// score): the few candidates mostly (and a softmax's sum), all of a token where it is
// not clear which experts make a group's score.
// Without a bias the logits themselves rank, of which the scores are monotone. The
// exponential of a pair: exp(x) = 2^n exp(j/32) exp(r), |r| <= 1/64, exp(j/32) from a
// table of pairs that the lanes hold (P. T. P. Tang, "Table-driven implementation of
// the exponential function", 1989), exp(r) its Taylor series, of which the terms up
// to r^2 are pairs.
#pragma once

#include <math.h>

#include "block.h"
#include "common.cuh"
#include "topk.cuh"

namespace moe {
namespace {

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

// Distance up to which two fp32 keys may stand in the wrong order. The exponential
// errs by 2^-22 (ex2.approx) and 2^-23, the quotient by 2^-22, the sum with one by
// 2^-24: a sigmoid by less than 7e-7 of itself, a key by a rounding more; a softmax's
// sum of up to 1,024 terms adds 2^-21, which all scores share.
__device__ __forceinline__ float doubt(bool softmax, float s_max, float key) {
  return s_max * (softmax ? 2.4e-6f : 1.4e-6f) + 2.4e-7f * fabsf(key);
}
__device__ __forceinline__ F2 pair_sigmoid(float x, const F2& tab) {
  const F2 e = exp_pair({-fabsf(x), 0.0f}, tab), d = add({1.0f, 0.0f}, e);
  return x >= 0.0f ? div({1.0f, 0.0f}, d) : div(e, d);
}
__device__ __forceinline__ F2 pair_score(bool softmax, float x, float top, const F2& sum, const F2& tab) {
  return softmax ? div(exp_pair(two_sum(x, -top), tab), sum) : pair_sigmoid(x, tab);
}
// Finite logit; *nan.
__device__ __forceinline__ float logit(float x, bool* nan) {
  *nan = isnan(x);
  return *nan ? -kFmax : fminf(fmaxf(x, -kFmax), kFmax);
}
// A key as a pair, by the definition.
__device__ __forceinline__ F2 pair_key(const F2& s, float b, bool nan) {
  if (nan) return {-INFINITY, 0.0f};
  return fabsf(b) <= kFmax ? add({b, 0.0f}, s) : F2{isnan(b) ? -INFINITY : b, 0.0f};
}

// Sum of exp(l - top) over a token's experts (whole warp, all lanes the same); top is the largest logit. Two terms at a
// time, since one is a long chain.
__device__ __noinline__ F2 pair_sum(const float* row, int E, float top) {
  const int lane = threadIdx.x & 31;
  const F2 tab{kExpTable.hi[lane], kExpTable.lo[lane]};
  F2 s0{0.0f, 0.0f}, s1{0.0f, 0.0f};
#pragma unroll 1
  for (int e0 = 0; e0 < E; e0 += 64) {
    bool nan0 = true, nan1 = true;
    const int e = e0 + lane;
    const float l0 = e < E ? logit(row[e], &nan0) : 0.0f, l1 = e + 32 < E ? logit(row[e + 32], &nan1) : 0.0f;
    const F2 v0 = exp_pair(two_sum(l0, -top), tab), v1 = exp_pair(two_sum(l1, -top), tab);
    if (!nan0) s0 = add(s0, v0);
    if (!nan1) s1 = add(s1, v1);
  }
  F2 sum = add(s0, s1);
  for (int o = 1; o < 32; o <<= 1) {
    const F2 other{__shfl_xor_sync(0xFFFFFFFFu, sum.hi, o), __shfl_xor_sync(0xFFFFFFFFu, sum.lo, o)};
    sum = (lane & o) ? add(other, sum) : add(sum, other);   // the same in both lanes
  }
  return sum.hi == 0.0f ? F2{1.0f, 0.0f} : sum;
}

// One token with every score as a pair (whole warp): keys to shared memory [n][32]
// twice, high and low parts; lane r < k gets its expert. Taken where fp32 cannot tell
// groups apart, or too many experts.
__device__ __noinline__ int route_in_pairs(const GroupArgs& a, const float* row, int L, uint32_t* kh, uint32_t* kl) {
  const int lane = threadIdx.x & 31, size = a.E / a.n_groups, g = lane / L, u = lane % L;
  const int n = g < a.n_groups ? (size - u + L - 1) / L : 0;         // experts of this lane
  const F2 tab{kExpTable.hi[lane], kExpTable.lo[lane]};
  const int all = (size + L - 1) / L;
  float top_l = -kFmax;
  F2 sum{0.0f, 0.0f};
  if (a.softmax) {
    for (int j = 0; j < n; ++j) {
      bool nan;
      const float l = logit(row[g * size + u + j * L], &nan);
      if (!nan) top_l = fmaxf(top_l, l);
    }
    for (int o = 16; o > 0; o >>= 1) top_l = fmaxf(top_l, __shfl_xor_sync(0xFFFFFFFFu, top_l, o));
    sum = pair_sum(row, a.E, top_l);
  }
  F2 b0{-INFINITY, 0.0f}, b1{-INFINITY, 0.0f};                 // the two best of this lane's, for its group
  auto take = [&](const F2& v) {
    if (less(b0, v)) b1 = b0, b0 = v;
    else if (less(b1, v)) b1 = v;
  };
#pragma unroll 1
  for (int j = 0; j < all; ++j) {
    bool nan = true;
    const int e = g * size + u + j * L;
    const float l = j < n ? logit(row[e], &nan) : 0.0f;
    F2 s = a.softmax ? div(exp_pair(two_sum(l, -top_l), tab), sum) : pair_sigmoid(l, tab);
    if (nan) s = {0.0f, 0.0f};
    const F2 key = a.bias ? pair_key(s, j < n ? a.bias[e] : 0.0f, nan) : F2{nan ? -INFINITY : l, 0.0f};
    if (j < n) {
      kh[j * 32 + lane] = rank_key(key.hi);
      kl[j * 32 + lane] = rank_key(key.lo);
      take(a.bias || a.best == 1 || nan ? key : s);
    }
  }
  bool in = g < a.n_groups;
  if (a.top < a.n_groups) {
    for (int o = 1; o < L; o <<= 1) {
      const F2 o0{__shfl_xor_sync(0xFFFFFFFFu, b0.hi, o), __shfl_xor_sync(0xFFFFFFFFu, b0.lo, o)};
      const F2 o1{__shfl_xor_sync(0xFFFFFFFFu, b1.hi, o), __shfl_xor_sync(0xFFFFFFFFu, b1.lo, o)};
      take(o0);
      take(o1);
    }
    // a sum of two keys in halves, so that it does not leave fp32; with an infinite one it is that, the larger of two
    F2 score = b0;
    if (a.best > 1) {
      auto half = [](const F2& v) { return F2{0.5f * v.hi, 0.5f * v.lo}; };
      if (fabsf(b0.hi) <= kFmax) score = fabsf(b1.hi) <= kFmax ? add(half(b0), half(b1)) : b1;
    }
    int better = 0;
    for (int i = 0; i < a.n_groups; ++i) {
      const F2 v{__shfl_sync(0xFFFFFFFFu, score.hi, i * L), __shfl_sync(0xFFFFFFFFu, score.lo, i * L)};
      better += less(score, v) || (!less(v, score) && i < g);
    }
    in = in && better < a.top;
  }
  int my_e = 0;
  for (int r = 0; r < a.k; ++r) {
    uint32_t bh = 0u, bl = 0u;
    int bj = 0;
    if (in)
      for (int j = 0; j < n; ++j) {
        const uint32_t h = kh[j * 32 + lane], w = kl[j * 32 + lane];
        if (h > bh || (h == bh && h && w > bl)) bh = h, bl = w, bj = j;
      }
    const uint32_t h = __reduce_max_sync(0xFFFFFFFFu, bh);
    const uint32_t w = __reduce_max_sync(0xFFFFFFFFu, bh == h ? bl : 0u);
    const int mine = bh == h && bl == w ? g * size + u + bj * L : 0x7FFFFFFF;
    const int e = __reduce_min_sync(0xFFFFFFFFu, mine);
    if (mine == e) kh[bj * 32 + lane] = 0u;
    if (lane == r) my_e = e;
  }
  return my_e;
}

// One token's experts and weights to the lanes below k, in descending key order (whole
// warp). PL: experts a lane holds, of group lane / L. scratch: PL * 64 words of shared
// memory.
template <int PL>
__device__ __forceinline__ void route_token(const GroupArgs& a, const float* row, int L, uint32_t* scratch, int* e_out,
                                            float* w_out) {
  const int lane = threadIdx.x & 31;
  const int size = a.E / a.n_groups, g = lane / L, u = lane % L;
  auto expert = [&](int j) { return g * size + u + j * L; };
  auto held = [&](int j) { return g < a.n_groups && u + j * L < size; };

  // ---- keys in fp32 --------------------------------------------------------------
  float l[PL], s[PL], b[PL];
  float l_max = -INFINITY;
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    l[j] = held(j) ? row[expert(j)] : -INFINITY;
    b[j] = a.bias && held(j) ? a.bias[expert(j)] : 0.0f;
  }
  bool odd = false;              // a logit or a bias that is not finite
#pragma unroll
  for (int j = 0; j < PL; ++j) {
    l_max = fmaxf(l_max, l[j]);
    odd |= held(j) && !(fabsf(l[j]) <= kFmax && fabsf(b[j]) <= kFmax);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l_max = fmaxf(l_max, __shfl_xor_sync(0xFFFFFFFFu, l_max, o));
  const bool scores = a.bias || a.best > 1;      // else the logits rank
  float s_max = 1.0f;
  bool unsure = __any_sync(0xFFFFFFFFu, odd);
  int my_e = 0;
  if (!unsure) {
    if (scores) {
      const float from = a.softmax ? l_max : 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < PL; ++j) {
        // 2^(x log2 e), with what the product's rounding leaves out
        const float x = a.softmax ? l[j] - from : -l[j], y = x * 1.4426950408889634f;
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
        if (fabsf(x) < 100.0f) e = fmaf(e, fmaf(x, 1.4426950408889634f, -y) * 0.6931472f, e);
        s[j] = a.softmax ? e : __fdividef(1.0f, 1.0f + e);
        if (!a.softmax && l[j] < -80.0f) s[j] = 0.0f;
        sum += s[j];
      }
      if (a.softmax) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        s_max = 1.0f / sum;
#pragma unroll
        for (int j = 0; j < PL; ++j) s[j] *= s_max;
      } else {
        s_max = 1.0f / (1.0f + expf(-l_max));
        unsure = l_max < -80.0f;                 // scores that fp32 hardly holds
      }
    }
    uint32_t key[PL];
#pragma unroll
    for (int j = 0; j < PL; ++j) {
      const float v = a.bias ? s[j] + b[j] : l[j];
      key[j] = held(j) ? rank_key(v) : 0u;
      s[j] = a.bias || a.best == 1 ? v : s[j];       // from here on: what counts for the group
    }

    if (a.top < a.n_groups) {
      // a group's score: its best key, or the sum of its two best (without a bias, of their scores)
      float b0 = -INFINITY, b1 = -INFINITY;
      auto take = [&](float v) {
        b1 = fmaxf(b1, fminf(b0, v));
        b0 = fmaxf(b0, v);
      };
#pragma unroll
      for (int j = 0; j < PL; ++j)
        if (held(j)) take(s[j]);
      for (int o = 1; o < L; o <<= 1) {
        const float o0 = __shfl_xor_sync(0xFFFFFFFFu, b0, o), o1 = __shfl_xor_sync(0xFFFFFFFFu, b1, o);
        take(o0);
        take(o1);
      }
      const float score = a.best > 1 ? b0 + b1 : b0;
      int better = 0;
      for (int i = 0; i < a.n_groups; ++i) {
        const float v = __shfl_sync(0xFFFFFFFFu, score, i * L);
        better += v > score || (v == score && i < g);
      }
      if (scores) {        // the last group that is in and the first that is not: does their order stand?
        const int in = __ffs(__ballot_sync(0xFFFFFFFFu, g < a.n_groups && better == a.top - 1)) - 1;
        const int out = __ffs(__ballot_sync(0xFFFFFFFFu, g < a.n_groups && better == a.top)) - 1;
        const float v = __shfl_sync(0xFFFFFFFFu, score, in), w = __shfl_sync(0xFFFFFFFFu, score, out);
        if (!(v - w > 2.0f * doubt(a.softmax, s_max, fabsf(v) + fabsf(w)))) {     // where sums leave fp32, too
          // Rank the groups by sums of pairs, where it is clear of which experts.
          const float from_key = (a.best > 1 ? b1 : b0) - doubt(a.softmax, s_max, fabsf(b0) + fabsf(b1));
          int n = 0, e0 = -1, e1 = -1;           // this lane's experts that may count
#pragma unroll
          for (int j = 0; j < PL; ++j)
            if (held(j) && s[j] >= from_key) {
              e1 = n ? expert(j) : -1;
              if (!n) e0 = expert(j);
              ++n;
            }
          int of_group = n;
          for (int o = 1; o < L; o <<= 1) of_group += __shfl_xor_sync(0xFFFFFFFFu, of_group, o);
          unsure = __any_sync(0xFFFFFFFFu, g < a.n_groups && (of_group != a.best || !(fabsf(score) <= kFmax)));
          if (!unsure) {
            const F2 tab{kExpTable.hi[lane], kExpTable.lo[lane]};
            const F2 of_all = a.softmax ? pair_sum(row, a.E, l_max) : F2{1.0f, 0.0f};
            F2 sum{0.0f, 0.0f};
            for (int i = 0; i < a.best; ++i) {
              const int e = i ? e1 : e0;
              const F2 x = pair_score(a.softmax, e >= 0 ? row[e] : l_max, l_max, of_all, tab);
              if (e >= 0) sum = add(sum, a.bias ? add({a.bias[e], 0.0f}, x) : x);
            }
            for (int o = 1; o < L; o <<= 1) {
              const F2 other{__shfl_xor_sync(0xFFFFFFFFu, sum.hi, o), __shfl_xor_sync(0xFFFFFFFFu, sum.lo, o)};
              sum = (lane & o) ? add(other, sum) : add(sum, other);   // the same in both lanes
            }
            better = 0;
            for (int i = 0; i < a.n_groups; ++i) {
              const F2 x{__shfl_sync(0xFFFFFFFFu, sum.hi, i * L), __shfl_sync(0xFFFFFFFFu, sum.lo, i * L)};
              better += less(sum, x) || (!less(x, sum) && i < g);
            }
          }
        }
      }
      if (better >= a.top) {
#pragma unroll
        for (int j = 0; j < PL; ++j) key[j] = 0u;
      }
    }

    // ---- the best keys, equal ones by the lower expert -------------------------------
    // a lane's two best, for it is seldom asked for a third
    uint32_t bk, ck, gone = 0u;
    int bj, cj;
    auto local_best = [&]() {
      bk = ck = 0u;
      bj = cj = 0;
#pragma unroll
      for (int j = 0; j < PL; ++j) {
        const uint32_t v = (gone >> j) & 1u ? 0u : key[j];
        const bool first = v > bk, second = v > ck;
        ck = first ? bk : second ? v : ck;
        cj = first ? bj : second ? j : cj;
        bk = first ? v : bk;
        bj = first ? j : bj;
      }
    };
    local_best();
    bool two = true;
    uint32_t my_key = 0u;
    auto next_best = [&](int r) {      // to lane r; false: there is none
      const uint32_t h = __reduce_max_sync(0xFFFFFFFFu, bk);
      const int e = __reduce_min_sync(0xFFFFFFFFu, bk == h ? expert(bj) : 0x7FFFFFFF);
      if (bk == h && expert(bj) == e) {
        gone |= 1u << bj;
        bk = ck, bj = cj;
        if (!two) local_best();
        two = !two;
      }
      if (lane == r) my_e = e, my_key = h;
      return h != 0u;
    };
    int n = 0;
    while (n < a.k && next_best(n)) ++n;
    if (a.bias && !unsure) {
      // Does the order stand? Candidates are all keys that may be as large as the last one wanted, of one logit and bias
      // with it or not, and one more, which shows that there are no others.
      for (bool more = true; more;) {
        if (n == 32) {
          unsure = true;
          break;
        }
        more = next_best(n);
        if (more) ++n;
        const float v = rank_value(my_key), last = __shfl_sync(0xFFFFFFFFu, v, a.k - 1);
        more = more && last - __shfl_sync(0xFFFFFFFFu, v, n - 1) <= doubt(a.softmax, s_max, fabsf(last));
      }
      const float v = rank_value(my_key), w = __shfl_down_sync(0xFFFFFFFFu, v, 1);
      const float ml = lane < n ? row[my_e] : 0.0f, mb = lane < n ? a.bias[my_e] : 0.0f;
      const float wl = __shfl_down_sync(0xFFFFFFFFu, ml, 1), wb = __shfl_down_sync(0xFFFFFFFFu, mb, 1);
      // keys of one logit and bias are equal, whatever their rounding: their order stands
      const bool close = __any_sync(
          0xFFFFFFFFu, lane + 1 < n && v - w <= doubt(a.softmax, s_max, fabsf(v)) && !(ml == wl && mb == wb));
      if (close && !unsure) {       // rank the candidates by their keys as pairs
        const F2 tab{kExpTable.hi[lane], kExpTable.lo[lane]};
        const F2 of_all = a.softmax ? pair_sum(row, a.E, l_max) : F2{1.0f, 0.0f};
        const F2 e = add({mb, 0.0f}, pair_score(a.softmax, lane < n ? ml : l_max, l_max, of_all, tab));
        int before = 0;
        for (int i = 0; i < n; ++i) {
          const F2 v{__shfl_sync(0xFFFFFFFFu, e.hi, i), __shfl_sync(0xFFFFFFFFu, e.lo, i)};
          const int id = __shfl_sync(0xFFFFFFFFu, my_e, i);
          before += less(e, v) || (!less(v, e) && id < my_e);
        }
        int mine = 0;
        for (int i = 0; i < n; ++i) {
          const int at = __shfl_sync(0xFFFFFFFFu, before, i), id = __shfl_sync(0xFFFFFFFFu, my_e, i);
          if (at == lane) mine = id;
        }
        my_e = mine;
      }
    }
  }
  if (unsure) my_e = route_in_pairs(a, row, L, scratch, scratch + PL * 32);

  // ---- weights ------------------------------------------------------------------------
  if (a.softmax && __any_sync(0xFFFFFFFFu, odd)) {     // the largest finite logit, or what an infinite one counts as
    l_max = -kFmax;
    for (int e = lane; e < a.E; e += 32) {
      bool nan;
      const float x = logit(row[e], &nan);
      if (!nan) l_max = fmaxf(l_max, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l_max = fmaxf(l_max, __shfl_xor_sync(0xFFFFFFFFu, l_max, o));
  }
  float my_s = 0.0f;
  if (lane < a.k) {
    bool nan;
    const float x = logit(row[my_e], &nan);
    if (a.softmax) {
      my_s = expf(x - l_max);        // times the sum of all, as yet
    } else {
      const float e = expf(-fabsf(x));
      my_s = (x >= 0.0f ? 1.0f : e) / (1.0f + e);
    }
    if (nan) my_s = 0.0f;
  }
  float all = my_s, sum = 1.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  // in a quotient of scores the sum of all drops out, but for the 1e-20, which is less than 2^-26 of more than 1e-9
  if (a.softmax && !(a.renorm && all > 1e-9f)) {
    sum = 0.0f;
#pragma unroll 4
    for (int e = lane; e < a.E; e += 32) {
      bool nan;
      const float x = logit(row[e], &nan);
      if (!nan) sum += expf(x - l_max);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (sum == 0.0f) sum = 1.0f;
  }
  *e_out = my_e;
  *w_out = (a.renorm ? my_s / fmaf(1e-20f, sum, all) : my_s / sum) * a.scale;
}

}  // namespace
}  // namespace moe
