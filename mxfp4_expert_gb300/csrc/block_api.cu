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

extern "C" int moe_route_groups(const float* logits_dev, int T, int E, int k, const float* bias_dev, int score,
                                int n_groups, int top_groups, int group_best, int renormalise, float scale,
                                int32_t* idx_dev, float* w_dev, moe_stream_t stream) {
  MOE_CHECK_ARG(T >= 0 && E >= 1 && k >= 1 && n_groups >= 1 && top_groups >= 1 && top_groups <= n_groups,
                MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(score == MOE_SCORE_SIGMOID || score == MOE_SCORE_SOFTMAX, MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG((group_best == 1 || group_best == 2) && (renormalise == 0 || renormalise == 1) && isfinite(scale),
                MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(groups_ok(E, k, n_groups, top_groups, group_best), MOE_ERR_UNSUPPORTED_SHAPE);
  if (T == 0) return MOE_OK;
  MOE_CHECK_ARG(logits_dev && idx_dev && w_dev, MOE_ERR_INVALID_ARG);
  DeviceInfo di;
  const int st = current_device(&di);
  if (st != MOE_OK) return st;
  const GroupArgs a{logits_dev, bias_dev, T, E, k, score == MOE_SCORE_SOFTMAX, n_groups, top_groups, group_best,
                    renormalise, scale, idx_dev, w_dev};
  return launch_route_groups(a, (cudaStream_t)stream);
}
