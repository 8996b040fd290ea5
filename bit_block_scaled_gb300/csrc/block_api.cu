// The C ABI of the calls around the layer (grouped routing, norms, key-value
// cache, attention): argument checks, all before anything is launched.
#include "checks.h"
#include "common.cuh"
#include "kernels.h"
#include "kvcache.cuh"
#include "types.cuh"

using namespace moe4;

namespace {

moe_status_t check_router(const moe_router_t *r, int E, int k) {
  if (!r) return MOE_ERR_INVALID_ARG;
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (r->group_score != MOE_GROUP_MAX && r->group_score != MOE_GROUP_TOP2) return MOE_ERR_INVALID_ARG;
  if (r->n_group < 1 || r->n_group > 32 || E % r->n_group) return MOE_ERR_INVALID_ARG;
  if (r->topk_group < 1 || r->topk_group > r->n_group) return MOE_ERR_INVALID_ARG;
  const int gs = E / r->n_group;
  if (k > r->topk_group * gs) return MOE_ERR_INVALID_ARG;
  if (r->group_score == MOE_GROUP_TOP2 && r->topk_group < r->n_group && gs < 2) return MOE_ERR_INVALID_ARG;
  if (!(r->scale == r->scale)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status_t check_norm(const moe_norm_t *n) {
  if (!n) return MOE_OK;
  if (n->kind != MOE_NORM_RMS && n->kind != MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
  if (!valid_dtype(n->type) || !(n->eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if ((n->weight && !aligned16(n->weight)) || (n->bias && !aligned16(n->bias))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status_t moe_route_grouped(const void *logits, int logits_type, int64_t ld, const float *sel_bias, int T, int E,
                               int k, const moe_router_t *router, int32_t *topk_ids, float *topk_weights, void *ws,
                               moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  if (T < 0 || T > 1 << 28 || E < 1 || E > 256 || k < 1 || k > 8 || k > E) return MOE_ERR_INVALID_ARG;
  if (!valid_dtype(logits_type) || ld < E) return MOE_ERR_INVALID_ARG;
  const moe_status_t s = check_router(router, E, k);
  if (s != MOE_OK) return s;
  if (!aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!aligned16(logits) || !aligned16(topk_ids) || !aligned16(topk_weights)) return MOE_ERR_INVALID_ARG;
  if (sel_bias && !aligned16(sel_bias)) return MOE_ERR_INVALID_ARG;
  return launch_group_route(logits, logits_type, ld, sel_bias, T, E, k, *router, topk_ids, topk_weights,
                            (cudaStream_t)stream, n);
}

moe_status_t moe_residual_norm(const void *z, int64_t z_stride, const void *residual, int64_t residual_stride,
                               const void *gate, int64_t gate_stride_t, int64_t gate_stride_h, int T, int H, int type,
                               int res_type, const moe_norm_t *post, float alpha, void *h_out, int64_t h_stride,
                               const moe_norm_t *pre, void *y_out, int64_t y_stride, moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  if (T < 0 || H < 1 || H > 16384 || !valid_dtype(type)) return MOE_ERR_INVALID_ARG;
  if (res_type != type && res_type != MOE_FP32) return MOE_ERR_INVALID_ARG;
  moe_status_t s = check_norm(post);
  if (s == MOE_OK) s = check_norm(pre);
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  if ((pre == nullptr) != (y_out == nullptr) || (!h_out && !y_out)) return MOE_ERR_INVALID_ARG;
  if (!z && (post || gate || !residual)) return MOE_ERR_INVALID_ARG;
  const void *ptr[5] = {z, residual, gate, h_out, y_out};
  for (const void *p : ptr)
    if (p && !aligned16(p)) return MOE_ERR_INVALID_ARG;
  if ((z && z_stride < 0) || (residual && residual_stride < 0)) return MOE_ERR_INVALID_ARG;
  if ((h_out && T > 1 && h_stride < H) || (y_out && T > 1 && y_stride < H)) return MOE_ERR_INVALID_ARG;
  if (gate && ((gate_stride_h != 0 && gate_stride_h != 1) || gate_stride_t < 0)) return MOE_ERR_INVALID_ARG;
  return launch_residual_norm(z, z_stride, residual, residual_stride, gate, gate_stride_t, gate_stride_h, T, H, type,
                              res_type, post, alpha, h_out, h_stride, pre, y_out, y_stride, (cudaStream_t)stream, n);
}

int64_t moe_kv_record_bytes(int fmt, int head_dim) { return built(fmt, head_dim) ? kv_record(fmt, head_dim) : 0; }

moe_status_t moe_kv_write(const void *k, const void *v, int type, int64_t k_stride_t, int64_t k_stride_h,
                          int64_t v_stride_t, int64_t v_stride_h, const int32_t *slots, int T,
                          const moe_kv_cache_t *cache, void *ws, moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  if (T < 0 || !valid_dtype(type) || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  const moe_status_t s = check_cache(cache);
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  if (!aligned16(k) || !aligned16(v) || !aligned4(slots)) return MOE_ERR_INVALID_ARG;
  if (!strides8(k_stride_t, k_stride_h) || !strides8(v_stride_t, v_stride_h)) return MOE_ERR_INVALID_ARG;
  if (k_stride_t < 0 || k_stride_h < 0 || v_stride_t < 0 || v_stride_h < 0) return MOE_ERR_INVALID_ARG;
  return launch_kv_write(k, v, type, k_stride_t, k_stride_h, v_stride_t, v_stride_h, slots, T, *cache, status_of(ws),
                         (cudaStream_t)stream, n);
}

moe_status_t moe_kv_read(const moe_kv_cache_t *cache, const int32_t *slots, int num, void *k_out, void *v_out, int type,
                         int64_t k_stride_t, int64_t k_stride_h, int64_t v_stride_t, int64_t v_stride_h, void *ws,
                         moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  if (num < 0 || !valid_dtype(type) || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  const moe_status_t s = check_cache(cache);
  if (s != MOE_OK) return s;
  if (num == 0 || (!k_out && !v_out)) return MOE_OK;
  if ((k_out && !aligned16(k_out)) || (v_out && !aligned16(v_out)) || !aligned4(slots)) return MOE_ERR_INVALID_ARG;
  const int H = cache->kv_heads, D = cache->head_dim;
  if (k_out && (!strides8(k_stride_t, k_stride_h) || !apart(num, k_stride_t, H, k_stride_h, D)))
    return MOE_ERR_INVALID_ARG;
  if (v_out && (!strides8(v_stride_t, v_stride_h) || !apart(num, v_stride_t, H, v_stride_h, D)))
    return MOE_ERR_INVALID_ARG;
  return launch_kv_read(*cache, slots, num, k_out, v_out, type, k_stride_t, k_stride_h, v_stride_t, v_stride_h,
                        status_of(ws), (cudaStream_t)stream, n);
}

moe_status_t moe_attn_workspace_size(int q_heads, int kv_heads, int head_dim, size_t *bytes) {
  if (!bytes || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads || q_heads / kv_heads > 128)
    return MOE_ERR_INVALID_ARG;
  if (!built(MOE_KV_BF16, head_dim)) return MOE_ERR_UNSUPPORTED;
  *bytes = attn_workspace(q_heads / kv_heads, head_dim);
  return MOE_OK;
}

moe_status_t moe_attn_decode(const void *q, int q_type, int64_t q_stride_b, int64_t q_stride_h,
                             const moe_kv_cache_t *cache, const int32_t *block_table, int64_t table_stride,
                             int max_pages, const int32_t *seq_lens, int B, int q_heads, float scale, int window,
                             const float *sinks, void *out, int64_t out_stride_b, int64_t out_stride_h, float *lse,
                             void *ws, size_t ws_bytes, moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  const moe_status_t s = check_cache(cache);
  if (s != MOE_OK) return s;
  size_t need = 0;
  const moe_status_t w = moe_attn_workspace_size(q_heads, cache->kv_heads, cache->head_dim, &need);
  if (w != MOE_OK) return w;
  if (B < 0 || max_pages < 0 || window < 0 || (q_type != MOE_BF16 && q_type != MOE_FP16)) return MOE_ERR_INVALID_ARG;
  if (!(scale == scale) || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (B > 4096) return MOE_ERR_UNSUPPORTED;
  if ((cache->fmt == MOE_KV_BF16 && q_type != MOE_BF16) || (cache->fmt == MOE_KV_FP16 && q_type != MOE_FP16))
    return MOE_ERR_UNSUPPORTED;
  if ((int64_t)max_pages * cache->page_size >= (int64_t)1 << 31) return MOE_ERR_INVALID_ARG;
  // records of all sequences and heads, the most there can be, in 32 bits a CTA
  if ((int64_t)max_pages * (cache->page_size / 16) * B >= (int64_t)1 << 31) return MOE_ERR_INVALID_ARG;
  if ((int64_t)B * q_heads * 8 >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  if (B == 0) return MOE_OK;
  if (!aligned16(q) || !aligned16(out) || !aligned4(seq_lens) || (max_pages > 0 && !aligned4(block_table)))
    return MOE_ERR_INVALID_ARG;
  if ((sinks && !aligned4(sinks)) || (lse && !aligned4(lse))) return MOE_ERR_INVALID_ARG;
  if (!strides8(q_stride_b, q_stride_h) || !strides8(out_stride_b, out_stride_h)) return MOE_ERR_INVALID_ARG;
  if (q_stride_b < 0 || q_stride_h < 0 || (B > 1 && table_stride < max_pages)) return MOE_ERR_INVALID_ARG;
  if (!apart(B, out_stride_b, q_heads, out_stride_h, cache->head_dim)) return MOE_ERR_INVALID_ARG;
  return launch_attn_decode(q, q_type, q_stride_b, q_stride_h, *cache, block_table, table_stride, max_pages, seq_lens,
                            B, q_heads, scale, window, sinks, out, out_stride_b, out_stride_h, lse, ws,
                            (cudaStream_t)stream, n);
}

}  // extern "C"
