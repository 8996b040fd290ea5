// The C ABI of the batch plan and of rotary positions: argument checks, all before
// anything is launched, and the table of frequencies, on the host.
#include <math.h>

#include "checks.h"
#include "common.cuh"
#include "kernels.h"

using namespace moe4;

namespace {

constexpr double kTwoPi = 6.283185307179586476925, kTwoPiRest = 2.4492935982947064e-16;  // 2 pi is their sum

// A frequency in radians a position as a 64-bit fraction of a turn, to the nearest: the quotient by 2 pi in two doubles,
// whose fractions are exact.
uint64_t turns_of(double f) {
  if (f < 0.0) return 0 - turns_of(-f);
  const double t = f / kTwoPi, low = (fma(-t, kTwoPi, f) - t * kTwoPiRest) / kTwoPi;
  const double high = ldexp(t - floor(t), 64), rest = floor(high - floor(high) + ldexp(low - nearbyint(low), 64) + 0.5);
  return (uint64_t)high + (rest < 0.0 ? 0 - (uint64_t)-rest : (uint64_t)rest);
}

bool valid_rope(const moe_rope_t *r, int D) {
  if (!r || r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > D) return false;
  if (r->layout != MOE_ROPE_HALF && r->layout != MOE_ROPE_INTERLEAVED) return false;
  return isfinite((float)r->amplitude) && r->turns && (reinterpret_cast<uintptr_t>(r->turns) & 7u) == 0;
}

bool fits(const void *p, int type) { return p && reinterpret_cast<uintptr_t>(p) % dtype_bytes(type) == 0; }

// One of the rotated tensors: where it goes to must be apart, or be itself.
bool valid_tensor(const void *in, int64_t its, int64_t ith, void *out, int64_t ots, int64_t oth, int T, int heads, int D,
                  int type) {
  if (!fits(in, type) || !fits(out, type) || its < 0 || ith < 0 || !apart(T, ots, heads, oth, D)) return false;
  return in != out || ((T == 1 || its == ots) && (heads == 1 || ith == oth));
}

}  // namespace

extern "C" {

moe_status_t moe_batch_plan(const int32_t *new_lens, const int32_t *seq_lens, int B, int page_size, int num_pages,
                            int32_t *block_table, int64_t table_stride, int max_pages, int32_t *free_pages,
                            const int32_t *free_count, int32_t *seq_lens_out, int32_t *free_count_out, int32_t *offsets,
                            int T, int rows_each, int32_t *slots, int32_t *positions, int32_t *seq_ids, void *ws,
                            moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  if (B < 0 || T < 0 || T > 1 << 28 || rows_each < 0 || rows_each > 1 << 28 || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (page_size < 16 || page_size % 16 || page_size > 4096) return MOE_ERR_INVALID_ARG;
  if (num_pages < 1 || (int64_t)num_pages * page_size >= (int64_t)1 << 31) return MOE_ERR_INVALID_ARG;
  if (max_pages < 0 || ((int64_t)max_pages + 1) * page_size >= (int64_t)1 << 31) return MOE_ERR_INVALID_ARG;
  if (B > 4096) return MOE_ERR_UNSUPPORTED;
  if (B == 0 && T == 0) return MOE_OK;
  if (B > 1 && table_stride < max_pages) return MOE_ERR_INVALID_ARG;
  if (B > 0 && (!aligned4(new_lens) || !aligned4(seq_lens) || !aligned4(seq_lens_out))) return MOE_ERR_INVALID_ARG;
  if ((B > 0 && max_pages > 0 && !aligned4(block_table)) || (T > 0 && !aligned4(slots))) return MOE_ERR_INVALID_ARG;
  if (!aligned4(free_pages) || !aligned4(free_count) || !aligned4(free_count_out)) return MOE_ERR_INVALID_ARG;
  if ((offsets && !aligned4(offsets)) || (positions && !aligned4(positions)) || (seq_ids && !aligned4(seq_ids)))
    return MOE_ERR_INVALID_ARG;
  return launch_batch_plan(new_lens, seq_lens, B, page_size, num_pages, block_table, table_stride, max_pages, free_pages,
                           free_count, seq_lens_out, free_count_out, offsets, T, rows_each, slots, positions, seq_ids, status_of(ws),
                           (cudaStream_t)stream, n);
}

moe_status_t moe_rope_turns(const double *frequencies, int n, uint64_t *turns) {
  if (n < 0 || (n > 0 && (!frequencies || !turns))) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!isfinite(frequencies[i])) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) turns[i] = turns_of(frequencies[i]);
  return MOE_OK;
}

moe_status_t moe_rope_table(const moe_rope_config_t *c, uint64_t *turns, double *amplitude) {
  if (!c || !turns || !amplitude) return MOE_ERR_INVALID_ARG;
  const int R = c->rot_dim;
  if (R < 2 || R % 2 || R > 256 || !(c->base > 1.0) || !isfinite(c->base)) return MOE_ERR_INVALID_ARG;
  if (c->scaling < MOE_ROPE_PLAIN || c->scaling > MOE_ROPE_WAVELENGTH) return MOE_ERR_INVALID_ARG;
  const bool scaled = c->scaling != MOE_ROPE_PLAIN, bands = c->scaling == MOE_ROPE_YARN || c->scaling == MOE_ROPE_WAVELENGTH;
  if (scaled && (!(c->factor > 0.0) || !isfinite(c->factor))) return MOE_ERR_INVALID_ARG;
  if (bands && (c->original_len < 1 || !(c->high > c->low) || !(c->low > 0.0) || !isfinite(c->high))) return MOE_ERR_INVALID_ARG;
  if (c->scaling == MOE_ROPE_NTK && R == 2) return MOE_ERR_INVALID_ARG;
  if (!(c->amplitude >= 0.0) || !isfinite(c->amplitude)) return MOE_ERR_INVALID_ARG;
  const double L = c->original_len;
  double base = c->base, a = 1.0, lo = 0.0, hi = 0.0;
  if (c->scaling == MOE_ROPE_NTK) base *= pow(c->factor, (double)R / (R - 2));
  if (c->scaling == MOE_ROPE_YARN) {
    // the pairs that turn `high` and `low` times over the original length
    lo = R * log(L / (kTwoPi * c->high)) / (2.0 * log(base));
    hi = R * log(L / (kTwoPi * c->low)) / (2.0 * log(base));
    if (c->truncate) lo = floor(lo), hi = ceil(hi);
    lo = fmax(lo, 0.0);
    hi = fmin(hi, R - 1.0);
    if (c->factor > 1.0) a = 0.1 * log(c->factor) + 1.0;
  }
  for (int i = 0; i < R / 2; ++i) {
    double f = pow(base, -2.0 * i / R);
    double keep = 1.0;  // the share that is not stretched
    if (c->scaling == MOE_ROPE_LINEAR) keep = 0.0;
    if (c->scaling == MOE_ROPE_YARN) keep = 1.0 - fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
    if (c->scaling == MOE_ROPE_WAVELENGTH) keep = fmin(fmax((L * f / kTwoPi - c->low) / (c->high - c->low), 0.0), 1.0);
    if (keep < 1.0) f = f / c->factor * (1.0 - keep) + f * keep;
    turns[i] = turns_of(f);
  }
  *amplitude = c->amplitude > 0.0 ? c->amplitude : a;
  return MOE_OK;
}

moe_status_t moe_rope(const moe_rope_t *rope, const int32_t *positions, int T, int head_dim, const void *q, int64_t q_stride_t,
                      int64_t q_stride_h, int q_heads, void *q_out, int64_t q_out_stride_t, int64_t q_out_stride_h,
                      const void *k, int64_t k_stride_t, int64_t k_stride_h, int k_heads, void *k_out, int64_t k_out_stride_t,
                      int64_t k_out_stride_h, int type, moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  if (T < 0 || head_dim < 2 || head_dim > 256 || q_heads < 1 || k_heads < 0 || !valid_dtype(type)) return MOE_ERR_INVALID_ARG;
  if (q_heads > 4096 || k_heads > 4096) return MOE_ERR_UNSUPPORTED;
  if (!valid_rope(rope, head_dim)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!aligned4(positions)) return MOE_ERR_INVALID_ARG;
  if (!valid_tensor(q, q_stride_t, q_stride_h, q_out, q_out_stride_t, q_out_stride_h, T, q_heads, head_dim, type))
    return MOE_ERR_INVALID_ARG;
  if (k_heads && !valid_tensor(k, k_stride_t, k_stride_h, k_out, k_out_stride_t, k_out_stride_h, T, k_heads, head_dim, type))
    return MOE_ERR_INVALID_ARG;
  return launch_rope(*rope, positions, T, head_dim, q, q_stride_t, q_stride_h, q_heads, q_out, q_out_stride_t, q_out_stride_h,
                     k, k_stride_t, k_stride_h, k_heads, k_out, k_out_stride_t, k_out_stride_h, type, (cudaStream_t)stream, n);
}

moe_status_t moe_rope_kv_write(const moe_rope_t *rope, const int32_t *positions, const void *q, int64_t q_stride_t,
                               int64_t q_stride_h, int q_heads, void *q_out, int64_t q_out_stride_t, int64_t q_out_stride_h,
                               const void *k, int64_t k_stride_t, int64_t k_stride_h, const void *v, int64_t v_stride_t,
                               int64_t v_stride_h, int type, const int32_t *slots, int T, const moe_kv_cache_t *cache,
                               void *ws, moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  if (T < 0 || !valid_dtype(type) || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  const moe_status_t s = check_cache(cache);
  if (s != MOE_OK) return s;
  if (!valid_rope(rope, cache->head_dim) || (q != nullptr && q_heads < 1)) return MOE_ERR_INVALID_ARG;
  if (q && q_heads > 4096) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!aligned4(positions) || !aligned16(k) || !aligned16(v) || !aligned4(slots)) return MOE_ERR_INVALID_ARG;
  if (!strides8(k_stride_t, k_stride_h) || !strides8(v_stride_t, v_stride_h)) return MOE_ERR_INVALID_ARG;
  if (k_stride_t < 0 || k_stride_h < 0 || v_stride_t < 0 || v_stride_h < 0) return MOE_ERR_INVALID_ARG;
  if (q && (!aligned16(q) || !aligned16(q_out) || !strides8(q_stride_t, q_stride_h) ||
            !strides8(q_out_stride_t, q_out_stride_h) ||
            !valid_tensor(q, q_stride_t, q_stride_h, q_out, q_out_stride_t, q_out_stride_h, T, q_heads, cache->head_dim, type)))
    return MOE_ERR_INVALID_ARG;
  return launch_rope_kv_write(*rope, positions, T, q, q_stride_t, q_stride_h, q_heads, q_out, q_out_stride_t, q_out_stride_h,
                              k, k_stride_t, k_stride_h, v, v_stride_t, v_stride_h, type, slots, *cache, status_of(ws),
                              (cudaStream_t)stream, n);
}

}  // extern "C"
