// Launchers of the attention operators, shared between their translation units
// and the C-ABI entry points (attn_api.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "host_util.h"

namespace moe {

struct PrefillArgs {
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;   // token and head strides, elements
  int n_heads, n_kv, D;
  const int32_t *cu_q, *cu_k;
  int n_seq, total_q, total_k;
  int causal;
  float scale;
  __nv_bfloat16* out;   // [total_q][n_heads][D]
  float* lse;           // [total_q][n_heads] or null
  int* status;
};
int launch_attn_prefill(const PrefillArgs& a, const DeviceInfo& di, cudaStream_t s);

struct AppendArgs {
  moe_kv_cache c;
  const __nv_bfloat16 *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;
  const int32_t *cu, *start, *table;
  int n_seq, total, width;
  int* status;
};
int launch_kv_append(const AppendArgs& a, cudaStream_t s);

struct DecodeArgs {
  moe_kv_cache c;
  const __nv_bfloat16* q;
  int64_t q_ts, q_hs;
  int n_heads, n_seq, n_new;
  const int32_t *lengths, *table;
  int width;
  float scale;
  __nv_bfloat16* out;
  float* lse;
  float* weights;
  int64_t w_stride;
  void* ws;
  int* status;
};
size_t attn_decode_ws_bytes(const moe_kv_cache& c, int n_seq, int n_new, int n_heads, int width, bool weights,
                            const DeviceInfo& di);
int launch_attn_decode(const DecodeArgs& a, const DeviceInfo& di, cudaStream_t s);

struct EvictArgs {
  moe_kv_cache c;
  const int32_t *table, *lengths;
  int width, n_seq;
  const float* weights;
  int64_t w_stride;
  int keep, recent;
  const int32_t* dst;
  int dst_width;
  int32_t* kept;
  float* kept_w;
  int32_t* new_lengths;
  int* status;
};
int launch_kv_evict(const EvictArgs& a, const DeviceInfo& di, cudaStream_t s);

}  // namespace moe
