// The C ABI of the dense projections in 4 bits: argument checks, all before
// anything is launched.
#include "checks.h"
#include "common.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "types.cuh"

using namespace moe4;

namespace {

bool valid_sizes(int fmt, int rows, int K) {
  return (fmt == MOE_FMT_NVFP4 || fmt == MOE_FMT_MXFP4) && rows >= 0 && rows < 1 << 24 && K >= 32 && K % 32 == 0 && K <= 1 << 20;
}

// Sizes first, so that an operand without rows needs no memory.
moe_status_t check_fp4(const moe_fp4_t *f) {
  if (!f || !valid_sizes(f->fmt, f->rows, f->K)) return MOE_ERR_INVALID_ARG;
  if (f->row_scale_stride != 0 && f->row_scale_stride != 1) return MOE_ERR_INVALID_ARG;
  if (f->row_scale && (f->fmt != MOE_FMT_NVFP4 || !aligned4(f->row_scale))) return MOE_ERR_INVALID_ARG;
  if (f->rows && (!aligned16(f->q) || !aligned16(f->scales))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

int64_t moe_fp4_scale_bytes(int fmt, int rows, int K) {
  return valid_sizes(fmt, rows, K) ? fp4_tiles_r(rows) * fp4_tiles_k(fmt, K) * kFp4Tile : 0;
}

moe_status_t moe_fp4_quantize(const void *x, int type, int64_t x_stride, const moe_fp4_t *out, moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  const moe_status_t s = check_fp4(out);
  if (s != MOE_OK) return s;
  if (!valid_dtype(type)) return MOE_ERR_INVALID_ARG;
  if (out->K > 32768) return MOE_ERR_UNSUPPORTED;
  if (out->rows == 0) return MOE_OK;
  if (!aligned16(x) || x_stride < 0 || x_stride % 8) return MOE_ERR_INVALID_ARG;
  if (out->fmt == MOE_FMT_NVFP4 && (!out->row_scale || (out->row_scale_stride != 1 && out->rows > 1)))
    return MOE_ERR_INVALID_ARG;
  return launch_fp4_quantize(x, type, x_stride, *out, (cudaStream_t)stream, n);
}

moe_status_t moe_fp4_dequantize(const moe_fp4_t *f, void *out, int type, int64_t out_stride, moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  const moe_status_t s = check_fp4(f);
  if (s != MOE_OK) return s;
  if (!valid_dtype(type)) return MOE_ERR_INVALID_ARG;
  if (f->rows == 0) return MOE_OK;
  if (!aligned16(out) || out_stride % 8 || out_stride < 0 || (f->rows > 1 && out_stride < f->K)) return MOE_ERR_INVALID_ARG;
  return launch_fp4_dequantize(*f, out, type, out_stride, (cudaStream_t)stream, n);
}

moe_status_t moe_fp4_pack_scales(const uint8_t *plain, int fmt, int rows, int K, uint8_t *scales, moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  if (!valid_sizes(fmt, rows, K)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!plain || !aligned16(scales)) return MOE_ERR_INVALID_ARG;
  return launch_fp4_pack_scales(plain, fmt, rows, K, scales, (cudaStream_t)stream, n);
}

moe_status_t moe_fp4_linear(const moe_fp4_t *x, const moe_fp4_t *w, const void *bias, void *out, int type, int64_t ldo,
                            void *ws, moe_stream_t stream) {
  int *n = launch_counter();
  *n = 0;
  moe_status_t s = check_fp4(x);
  if (s == MOE_OK) s = check_fp4(w);
  if (s != MOE_OK) return s;
  if (x->fmt != w->fmt || x->K != w->K || !valid_dtype(type) || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (x->rows == 0 || w->rows == 0) return MOE_OK;
  if (!aligned16(out) || (bias && !aligned16(bias)) || ldo < 0 || (x->rows > 1 && ldo < w->rows)) return MOE_ERR_INVALID_ARG;
  return launch_fp4_linear(*x, *w, bias, out, type, ldo, status_of(ws), (cudaStream_t)stream, n);
}

}  // extern "C"
