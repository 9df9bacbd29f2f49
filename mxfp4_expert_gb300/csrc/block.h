// Launchers of the operators around a block's halves (norms, routing by groups),
// shared between their translation units and the C-ABI entry points.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "host_util.h"

namespace moe {

// norm.cu
struct NormArgs {
  const void* x;                 // residual stream, bf16 or fp32
  const __nv_bfloat16* a;        // block output, or null
  const __nv_bfloat16* wp;       // weight of its norm, or null: none
  const __nv_bfloat16* gate;     // [d] or [T][d], or null
  const __nv_bfloat16* wn;       // weight of the norm of y, or null: 1
  void* y;                       // as x, or null (without a)
  __nv_bfloat16* h;              // or null
  int64_t x_rs, a_rs, g_rs, y_rs, h_rs;   // row strides, elements
  int T, d, fp32;
  float scale, eps, offset;
};
int launch_block_norm(const NormArgs& a, const DeviceInfo& di, cudaStream_t s);

// route_groups.cu
struct GroupArgs {
  const float* logits;           // [T][E]
  const float* bias;             // [E] or null
  int T, E, k;
  int softmax, n_groups, top, best, renorm;
  float scale;
  int32_t* idx;                  // [T][k]
  float* w;                      // [T][k]
};
// Lanes of a warp that hold a group's experts, and how many of them each holds.
inline int group_lanes(int n_groups) {
  int p = 1;
  while (p < n_groups) p *= 2;
  return 32 / p;
}
inline int group_keys(int E, int n_groups) { return (E / n_groups + group_lanes(n_groups) - 1) / group_lanes(n_groups); }
// Checks a rule and fills all of *g but logits, idx and w.
int group_args(const moe_group_rule* r, int T, int E, int k, const float* bias, GroupArgs* g);
bool groups_ok(int E, int k, int n_groups, int top, int best);
int launch_route_groups(const GroupArgs& a, cudaStream_t s);

}  // namespace moe
