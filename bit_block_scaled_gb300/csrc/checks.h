// Argument checks that several of the C entry points share.
#pragma once

#include <stdint.h>

#include "kvcache.cuh"
#include "types.cuh"

namespace moe4 {

inline bool aligned16(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline unsigned int *status_of(void *ws) { return static_cast<unsigned int *>(ws); }

inline bool built(int fmt, int D) { return fmt >= MOE_KV_BF16 && fmt <= MOE_KV_NVFP4 && (D == 64 || D == 128 || D == 256); }

inline moe_status_t check_cache(const moe_kv_cache_t *c) {
  if (!c || c->fmt < MOE_KV_BF16 || c->fmt > MOE_KV_NVFP4) return MOE_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->kv_heads < 1 || c->head_dim < 1) return MOE_ERR_INVALID_ARG;
  if (c->page_size < 16 || c->page_size % 16 || c->page_size > 4096) return MOE_ERR_INVALID_ARG;
  if ((int64_t)c->num_pages * c->page_size >= (int64_t)1 << 31) return MOE_ERR_INVALID_ARG;
  if (!aligned16(c->data)) return MOE_ERR_INVALID_ARG;
  return built(c->fmt, c->head_dim) ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// rows of D values, 16-byte aligned
inline bool strides8(int64_t t, int64_t h) { return t % 8 == 0 && h % 8 == 0; }
// No two of the rows of D values at o * outer + i * inner (o < n_outer, i < n_inner) share an element.
inline bool apart(int n_outer, int64_t outer, int n_inner, int64_t inner, int D) {
  if (outer < 0 || inner < 0) return false;
  if ((n_outer > 1 && outer < D) || (n_inner > 1 && inner < D)) return false;
  if (n_outer <= 1 || n_inner <= 1) return true;
  // one dimension within the other's step, as in nearly all layouts
  if ((outer - D) / (n_inner - 1) >= inner || (inner - D) / (n_outer - 1) >= outer) return true;
  for (int i = 1; i < n_inner; ++i) {  // rows i apart in one dimension and o or o + 1 in the other
    const __int128 x = (__int128)i * inner, o = x / outer;
    if ((o < n_outer && x - o * outer < D) || (o + 1 < n_outer && (o + 1) * outer - x < D)) return false;
  }
  return true;
}

}  // namespace moe4
