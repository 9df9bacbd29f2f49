// C-ABI entry points of the operators around a block's halves: argument checks,
// then the launchers. Nothing is enqueued when a check fails.
#include <math.h>

#include "block.h"
#include "host_util.h"
#include "moe_mxfp4.h"

using namespace moe;

extern "C" int moe_block_norm(const void* x_dev, int64_t x_stride, int x_is_fp32, const void* a_dev, int64_t a_stride,
                              int T, int d, const void* post_weight_dev, const void* gate_dev, int64_t gate_stride,
                              float residual_scale, const void* pre_weight_dev, float eps, float weight_offset,
                              void* y_dev, int64_t y_stride, void* h_dev, int64_t h_stride, moe_stream_t stream) {
  MOE_CHECK_ARG(T >= 0 && d >= 1 && (x_is_fp32 == 0 || x_is_fp32 == 1), MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(isfinite(residual_scale) && isfinite(weight_offset) && isfinite(eps) && eps >= 0.0f, MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(d % 8 == 0 && d <= 32768, MOE_ERR_UNSUPPORTED_SHAPE);
  if (T == 0) return MOE_OK;
  MOE_CHECK_ARG((a_dev != nullptr) == (y_dev != nullptr) && (y_dev || h_dev), MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(a_dev || (!post_weight_dev && !gate_dev), MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(h_dev || !pre_weight_dev, MOE_ERR_INVALID_ARG);
  // one row of the gate may serve all; the strides of absent operands do not count
  const int64_t strides[5] = {x_stride, a_dev ? a_stride : d, gate_dev && gate_stride ? gate_stride : d,
                              y_dev ? y_stride : d, h_dev ? h_stride : d};
  for (int64_t s : strides) MOE_CHECK_ARG(s % 8 == 0 && (s >= d || T <= 1), MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(x_dev, MOE_ERR_INVALID_ARG);
  for (const void* p : {x_dev, a_dev, post_weight_dev, gate_dev, pre_weight_dev, (const void*)y_dev, (const void*)h_dev})
    MOE_CHECK_ARG(aligned(p, 16), MOE_ERR_INVALID_ARG);
  DeviceInfo di;
  const int st = current_device(&di);
  if (st != MOE_OK) return st;
  NormArgs n{};
  n.x = x_dev;
  n.a = static_cast<const __nv_bfloat16*>(a_dev);
  n.wp = static_cast<const __nv_bfloat16*>(post_weight_dev);
  n.gate = static_cast<const __nv_bfloat16*>(gate_dev);
  n.wn = static_cast<const __nv_bfloat16*>(pre_weight_dev);
  n.y = y_dev;
  n.h = static_cast<__nv_bfloat16*>(h_dev);
  n.x_rs = x_stride;
  n.a_rs = a_stride;
  n.g_rs = gate_stride;
  n.y_rs = y_stride;
  n.h_rs = h_stride;
  n.T = T;
  n.d = d;
  n.fp32 = x_is_fp32;
  n.scale = residual_scale;
  n.eps = eps;
  n.offset = weight_offset;
  return launch_block_norm(n, di, (cudaStream_t)stream);
}

namespace moe {

int group_args(const moe_group_rule* r, int T, int E, int k, const float* bias, GroupArgs* g) {
  MOE_CHECK_ARG(T >= 0 && E >= 1 && k >= 1 && r->n_groups >= 1 && r->top_groups >= 1 && r->top_groups <= r->n_groups,
                MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(r->score == MOE_SCORE_SIGMOID || r->score == MOE_SCORE_SOFTMAX, MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG((r->group_best == 1 || r->group_best == 2) && (r->renormalise == 0 || r->renormalise == 1) &&
                    isfinite(r->scale),
                MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(groups_ok(E, k, r->n_groups, r->top_groups, r->group_best), MOE_ERR_UNSUPPORTED_SHAPE);
  *g = GroupArgs{nullptr, bias, T, E, k, r->score == MOE_SCORE_SOFTMAX, r->n_groups, r->top_groups, r->group_best,
                 r->renormalise, r->scale, nullptr, nullptr};
  return MOE_OK;
}

}  // namespace moe

extern "C" int moe_route_groups(const float* logits_dev, int T, int E, int k, const float* bias_dev,
                                const moe_group_rule* rule, int32_t* idx_dev, float* w_dev, moe_stream_t stream) {
  MOE_CHECK_ARG(rule, MOE_ERR_INVALID_ARG);
  GroupArgs g{};
  int st = group_args(rule, T, E, k, bias_dev, &g);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  MOE_CHECK_ARG(logits_dev && idx_dev && w_dev, MOE_ERR_INVALID_ARG);
  DeviceInfo di;
  if ((st = current_device(&di))) return st;
  g.logits = logits_dev;
  g.idx = idx_dev;
  g.w = w_dev;
  return launch_route_groups(g, (cudaStream_t)stream);
}
