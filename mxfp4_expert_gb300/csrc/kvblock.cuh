// Where the tokens that a call appends to the paged cache go: shared by the two
// append kernels.
#pragma once

#include "attn.h"
#include "fp8kv.cuh"

namespace moe {

// Blocks of positions (page-sized, aligned) that a sequence's new tokens touch.
struct Block {
  int b;         // sequence, -1 for none
  int blk;       // page-table column
  int s0, s1;    // slots of new tokens
  int t0;        // row of the first of them
};

// Whole warp: which block is number x, counting over the sequences in order.
__device__ __forceinline__ Block find_block(const AppendArgs& a, int x, bool* bad) {
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

}  // namespace moe
