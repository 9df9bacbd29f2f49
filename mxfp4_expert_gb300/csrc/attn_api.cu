// C-ABI entry points of the attention operators: argument checks, then the
// launchers. Nothing is enqueued when a check fails.
#include <cuda_bf16.h>
#include <math.h>

#include "attn.h"
#include "host_util.h"
#include "moe_mxfp4.h"

namespace moe {
namespace {

int check_rows(const moe_rows* r) {
  if (!r || !r->data || !aligned(r->data, 16)) return MOE_ERR_INVALID_ARG;
  if (r->token_stride < 0 || r->head_stride < 0 || r->token_stride % 8 || r->head_stride % 8) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Sizes of a cache; its pointers too if `buffers`.
int check_cache(const moe_kv_cache* c, bool buffers) {
  if (!c || c->n_pages < 0 || c->n_kv_heads < 1) return MOE_ERR_INVALID_ARG;
  const int p = c->page_size, d = c->head_dim;
  if ((p != 16 && p != 32 && p != 64 && p != 128) || (d != 64 && d != 128)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (c->n_kv_heads > 1024) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!buffers) return MOE_OK;
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return MOE_ERR_INVALID_ARG;
  return aligned(c->k_codes, 16) && aligned(c->v_codes, 16) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

// The kernels count rows and positions in an int and step past the last one by
// tiles (of 16,384 positions at most, in the eviction).
constexpr int64_t kMaxRows = INT32_MAX - 65535;
bool table_ok(int width, int page) { return width >= 0 && (int64_t)width * page <= kMaxRows; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

int check_decode_shape(const moe_kv_cache* c, int n_seq, int n_new, int n_heads, int width) {
  int st = check_cache(c, false);
  if (st != MOE_OK) return st;
  if (n_seq < 0 || n_new < 1 || n_heads < 1 || !table_ok(width, c->page_size)) return MOE_ERR_INVALID_ARG;
  if (n_heads % c->n_kv_heads || n_new > 8 || n_new * (n_heads / c->n_kv_heads) > 64 || n_seq > 4096)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  // and the chunks of 32 positions of all sequences in one, at the longest that the tables hold
  return ((int64_t)width * c->page_size / 32 + 1) * n_seq <= INT32_MAX ? MOE_OK : MOE_ERR_UNSUPPORTED_SHAPE;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_attn_prefill(const moe_rows* q, const moe_rows* k, const moe_rows* v, int n_heads,
                                int n_kv_heads, int head_dim, const int32_t* cu_q_dev, const int32_t* cu_k_dev,
                                int n_seq, int total_q, int total_k, int causal, float scale, void* out_dev,
                                float* lse_dev, int* dev_status, moe_stream_t stream) {
  MOE_CHECK_ARG(n_seq >= 0 && total_q >= 0 && total_k >= 0 && n_heads >= 1 && n_kv_heads >= 1, MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG((causal == 0 || causal == 1) && isfinite(scale), MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG((head_dim == 64 || head_dim == 128) && n_heads % n_kv_heads == 0 && n_heads <= 65535 && n_seq <= 65536 &&
                    total_q <= kMaxRows && total_k <= kMaxRows,
                MOE_ERR_UNSUPPORTED_SHAPE);
  if (n_seq == 0 || total_q == 0) return MOE_OK;
  int st;
  if ((st = check_rows(q))) return st;
  // keys may be absent altogether: every query then sees nothing
  if (total_k > 0 && ((st = check_rows(k)) || (st = check_rows(v)))) return st;
  // a tensor map has no rows that lie on one another
  MOE_CHECK_ARG((total_q <= 1 || q->token_stride) && (total_k <= 1 || (k->token_stride && v->token_stride)),
                MOE_ERR_UNSUPPORTED_SHAPE);
  MOE_CHECK_ARG(cu_q_dev && cu_k_dev && out_dev && aligned(out_dev, 16), MOE_ERR_INVALID_ARG);
  DeviceInfo di;
  if ((st = current_device(&di))) return st;
  PrefillArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q->data);
  a.q_ts = q->token_stride;
  a.q_hs = q->head_stride;
  if (total_k > 0) {
    a.k = static_cast<const __nv_bfloat16*>(k->data);
    a.k_ts = k->token_stride;
    a.k_hs = k->head_stride;
    a.v = static_cast<const __nv_bfloat16*>(v->data);
    a.v_ts = v->token_stride;
    a.v_hs = v->head_stride;
  }
  a.n_heads = n_heads;
  a.n_kv = n_kv_heads;
  a.D = head_dim;
  a.cu_q = cu_q_dev;
  a.cu_k = cu_k_dev;
  a.n_seq = n_seq;
  a.total_q = total_q;
  a.total_k = total_k;
  a.causal = causal;
  a.scale = scale;
  a.out = static_cast<__nv_bfloat16*>(out_dev);
  a.lse = lse_dev;
  a.status = dev_status;
  return launch_attn_prefill(a, di, (cudaStream_t)stream);
}

extern "C" int moe_kv_append_fp8(const moe_kv_cache* cache, const moe_rows* k, const moe_rows* v,
                                 const int32_t* cu_dev, const int32_t* start_dev, int n_seq, int total,
                                 const int32_t* page_table_dev, int table_width, int* dev_status,
                                 moe_stream_t stream) {
  int st;
  if ((st = check_cache(cache, true))) return st;
  MOE_CHECK_ARG(n_seq >= 0 && total >= 0 && table_ok(table_width, cache->page_size), MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(n_seq <= 65536 && total <= kMaxRows, MOE_ERR_UNSUPPORTED_SHAPE);
  if (n_seq == 0 || total == 0) return MOE_OK;
  if ((st = check_rows(k)) || (st = check_rows(v))) return st;
  MOE_CHECK_ARG(cu_dev && start_dev && page_table_dev, MOE_ERR_INVALID_ARG);
  DeviceInfo di;
  if ((st = current_device(&di))) return st;
  AppendArgs a{};
  a.c = *cache;
  a.k = static_cast<const __nv_bfloat16*>(k->data);
  a.v = static_cast<const __nv_bfloat16*>(v->data);
  a.k_ts = k->token_stride;
  a.k_hs = k->head_stride;
  a.v_ts = v->token_stride;
  a.v_hs = v->head_stride;
  a.cu = cu_dev;
  a.start = start_dev;
  a.table = page_table_dev;
  a.n_seq = n_seq;
  a.total = total;
  a.width = table_width;
  a.status = dev_status;
  return launch_kv_append(a, (cudaStream_t)stream);
}

extern "C" size_t moe_attn_decode_workspace_bytes(const moe_kv_cache* cache, int n_seq, int n_new, int n_heads,
                                                  int table_width, int with_weights) {
  if (check_decode_shape(cache, n_seq, n_new, n_heads, table_width) != MOE_OK) return 0;
  DeviceInfo di;
  if (current_device(&di) != MOE_OK) return 0;
  return attn_decode_ws_bytes(*cache, n_seq, n_new, n_heads, table_width, with_weights != 0, di);
}

extern "C" int moe_attn_decode_fp8(const moe_kv_cache* cache, const moe_rows* q, int n_heads, int n_seq, int n_new,
                                   const int32_t* lengths_dev, const int32_t* page_table_dev, int table_width,
                                   float scale, void* out_dev, float* lse_dev, float* weights_dev,
                                   int64_t weights_stride, void* workspace_dev, size_t workspace_bytes,
                                   int* dev_status, moe_stream_t stream) {
  int st;
  if ((st = check_decode_shape(cache, n_seq, n_new, n_heads, table_width))) return st;
  if ((st = check_cache(cache, true))) return st;
  MOE_CHECK_ARG(isfinite(scale) && (!weights_dev || weights_stride >= 0), MOE_ERR_INVALID_ARG);
  if (n_seq == 0) return MOE_OK;
  if ((st = check_rows(q))) return st;
  MOE_CHECK_ARG(lengths_dev && (page_table_dev || table_width == 0) && out_dev && aligned(out_dev, 16), MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(workspace_dev && aligned(workspace_dev, 256), MOE_ERR_INVALID_ARG);
  DeviceInfo di;
  if ((st = current_device(&di))) return st;
  MOE_CHECK_ARG(workspace_bytes >= attn_decode_ws_bytes(*cache, n_seq, n_new, n_heads, table_width,
                                                        weights_dev != nullptr, di),
                MOE_ERR_WORKSPACE_TOO_SMALL);
  DecodeArgs a{};
  a.c = *cache;
  a.q = static_cast<const __nv_bfloat16*>(q->data);
  a.q_ts = q->token_stride;
  a.q_hs = q->head_stride;
  a.n_heads = n_heads;
  a.n_seq = n_seq;
  a.n_new = n_new;
  a.lengths = lengths_dev;
  a.table = page_table_dev;
  a.width = table_width;
  a.scale = scale;
  a.out = static_cast<__nv_bfloat16*>(out_dev);
  a.lse = lse_dev;
  a.weights = weights_dev;
  a.w_stride = weights_stride;
  a.ws = workspace_dev;
  a.status = dev_status;
  return launch_attn_decode(a, di, (cudaStream_t)stream);
}

extern "C" int moe_kv_evict_fp8(const moe_kv_cache* cache, const int32_t* page_table_dev, int table_width,
                                const int32_t* lengths_dev, int n_seq, const float* weights_dev,
                                int64_t weights_stride, int keep, int recent, const int32_t* dst_table_dev,
                                int dst_width, int32_t* kept_dev, float* kept_weights_dev, int32_t* new_lengths_dev,
                                int* dev_status, moe_stream_t stream) {
  int st;
  if ((st = check_cache(cache, true))) return st;
  const int page = cache->page_size;
  MOE_CHECK_ARG(n_seq >= 0 && table_ok(table_width, page) && table_ok(dst_width, page), MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(keep >= 1 && keep <= kMaxRows && recent >= 0 && recent <= keep && weights_stride >= 0, MOE_ERR_INVALID_ARG);
  MOE_CHECK_ARG(n_seq <= 65535, MOE_ERR_UNSUPPORTED_SHAPE);
  const int64_t most = (int64_t)table_width * page < keep ? (int64_t)table_width * page : keep;
  MOE_CHECK_ARG((int64_t)dst_width * page >= most, MOE_ERR_BUFFER_TOO_SMALL);
  if (n_seq == 0) return MOE_OK;
  MOE_CHECK_ARG(lengths_dev && kept_dev && new_lengths_dev, MOE_ERR_INVALID_ARG);
  // other heads still read the inputs when one writes its outputs
  const size_t pairs = (size_t)n_seq * cache->n_kv_heads, n_kept = pairs * keep * 4, n_len = (size_t)n_seq * 4;
  const struct { const void* p; size_t bytes; }
      outs[3] = {{kept_dev, n_kept}, {kept_weights_dev, n_kept}, {new_lengths_dev, n_len}},
      ins[4] = {{lengths_dev, n_len}, {weights_dev, pairs * weights_stride * 4},
                {page_table_dev, (size_t)n_seq * table_width * 4}, {dst_table_dev, (size_t)n_seq * dst_width * 4}};
  for (const auto& o : outs) {
    for (const auto& i : ins) MOE_CHECK_ARG(!overlap(o.p, o.bytes, i.p, i.bytes), MOE_ERR_INVALID_ARG);
    for (const auto& q : outs) MOE_CHECK_ARG(&o == &q || !overlap(o.p, o.bytes, q.p, q.bytes), MOE_ERR_INVALID_ARG);
  }
  MOE_CHECK_ARG(table_width == 0 || (page_table_dev && dst_table_dev && weights_dev), MOE_ERR_INVALID_ARG);
  DeviceInfo di;
  if ((st = current_device(&di))) return st;
  EvictArgs a{};
  a.c = *cache;
  a.table = page_table_dev;
  a.lengths = lengths_dev;
  a.width = table_width;
  a.n_seq = n_seq;
  a.weights = weights_dev;
  a.w_stride = weights_stride;
  a.keep = keep;
  a.recent = recent;
  a.dst = dst_table_dev;
  a.dst_width = dst_width;
  a.kept = kept_dev;
  a.kept_w = kept_weights_dev;
  a.new_lengths = new_lengths_dev;
  a.status = dev_status;
  return launch_kv_evict(a, di, (cudaStream_t)stream);
}
