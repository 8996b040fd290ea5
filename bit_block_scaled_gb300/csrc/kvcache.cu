// Writing tokens into the paged key-value cache, quantised, and reading them
// back.
//
// D / 8 lanes take one (token, head): each holds 8 values of the key and 8 of
// the value, so a row's largest magnitude is log2(D / 8) shuffles, a block of
// 16 is two lanes, and a lane's codes are one 4-, 8- or 16-byte store.
//
// Row scales are powers of two: x / r is exact, so an FP8 code is one rounding
// of x / r, and an NVFP4 code one rounding of the quotient x / r / s by the
// E4M3 scale. Quotients of a 16-bit x that lie on a tie of E2M1 are exact in
// fp32 and others cannot round onto one (x and the tie times s both have at
// most 11 significant bits), so the codes are those of real arithmetic.
#include "common.cuh"
#include "kernels.h"
#include "kvcache.cuh"
#include "types.cuh"

namespace moe4 {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 128;

struct KvArgs {
  uint8_t *data;
  const void *k, *v;
  void *ko, *vo;
  const int32_t *slots;
  unsigned int *status;
  int64_t kst, ksh, vst, vsh;
  int64_t rows;  // T * heads
  int type, T, heads, D, page, pages;
};

// 2^e for e in -63..64 (half of any row exponent), exactly.
__device__ __forceinline__ float pow2_half(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// x * 2^e for |e| <= 127, one step at a time so that 2^127 and 2^-127 work.
__device__ __forceinline__ float times_pow2(float x, int e) {
  const int h = e >> 1;
  return x * pow2_half(h) * pow2_half(e - h);
}

// Least e in -127..127 with amax * 2^-e <= top = m 2^x (m in [1/2, 1)); 0 gives -127.
__device__ __forceinline__ int row_exponent(float amax, float m, int x) {
  if (amax == 0.f) return -127;
  int e;
  const float f = frexpf(amax, &e);
  e += (f > m ? 1 : 0) - x;
  return min(max(e, -127), 127);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_f32(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

__device__ __forceinline__ void e2m1x8_f32(uint32_t w, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// Quantises a lane's 8 values x of a row and stores its codes (and the scales
// that fall to this lane). rec: the record; i: token in it; part: 0 keys, 1
// values; j: lane of the row; n: lanes of the row.
template <int FMT>
__device__ __forceinline__ void put8(uint8_t *rec, int i, int part, int j, int n, int D, float (&x)[8], bool live) {
  const int row = kv_row(FMT, D);
  uint8_t *codes = rec + part * 16 * row;
  if (FMT == MOE_KV_BF16 || FMT == MOE_KV_FP16) {
    const Raw8 r = f32_to_raw8(x, FMT == MOE_KV_BF16 ? MOE_BF16 : MOE_FP16);
    if (live) *reinterpret_cast<uint4 *>(codes + kv_place(row, i, 16 * j)) = r.a;
    return;
  }
  float m = 0.f;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m = fmaxf(m, fabsf(x[e]));
    bad = bad || !(fabsf(x[e]) <= 3.402823466e38f);
  }
  if (bad) m = INFINITY;
  float amax = m;
  for (int o = 1; o < n; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
  bad = !(amax <= 3.402823466e38f);
  const int e = bad ? 0 : FMT == MOE_KV_FP8 ? row_exponent(amax, 448.f / 512.f, 9) : row_exponent(amax, 2688.f / 4096.f, 12);
#pragma unroll
  for (int q = 0; q < 8; ++q) x[q] = bad ? 0.f : times_pow2(x[q], -e);
  if (FMT == MOE_KV_FP8) {
    uint2 c;
    c.x = e4m3x2(x[0], x[1]) | (e4m3x2(x[2], x[3]) << 16);
    c.y = e4m3x2(x[4], x[5]) | (e4m3x2(x[6], x[7]) << 16);
    if (live) *reinterpret_cast<uint2 *>(codes + kv_place(row, i, 8 * j)) = c;
  } else {
    m = bad ? 0.f : times_pow2(m, -e);
    m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));  // two lanes hold a block of 16
    const uint32_t sb = e4m3x2(m / 6.0f, 0.f) & 0xFFu;
    const float s = e4m3x2_f32(sb).x;
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = s > 0.f ? x[q] / s : 0.f;
    const uint32_t c = e2m1x8(x);
    if (live) {
      *reinterpret_cast<uint32_t *>(codes + kv_place(row, i, 4 * j)) = c;
      if ((j & 1) == 0) rec[kv_scales_at(FMT, D) + part * D + (j >> 1) * 16 + i] = (uint8_t)sb;
    }
  }
  if (live && j == 0) rec[kv_exps_at(FMT, D) + part * 16 + i] = (uint8_t)(bad ? 255 : e + 127);
}

template <int FMT>
__device__ __forceinline__ void get8(const uint8_t *rec, int i, int part, int j, int D, float (&x)[8]) {
  const int row = kv_row(FMT, D);
  const uint8_t *codes = rec + part * 16 * row;
  if (FMT == MOE_KV_BF16 || FMT == MOE_KV_FP16) {
    Raw8 r;
    r.a = *reinterpret_cast<const uint4 *>(codes + kv_place(row, i, 16 * j));
    raw8_to_f32(r, FMT == MOE_KV_BF16 ? MOE_BF16 : MOE_FP16, x);
    return;
  }
  const int e8 = rec[kv_exps_at(FMT, D) + part * 16 + i];
  if (FMT == MOE_KV_FP8) {
    const uint2 c = *reinterpret_cast<const uint2 *>(codes + kv_place(row, i, 8 * j));
    const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = e4m3x2_f32(w[q]);
      x[2 * q] = f.x;
      x[2 * q + 1] = f.y;
    }
  } else {
    e2m1x8_f32(*reinterpret_cast<const uint32_t *>(codes + kv_place(row, i, 4 * j)), x);
    const float s = e4m3x2_f32(rec[kv_scales_at(FMT, D) + part * D + (j >> 1) * 16 + i]).x;
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] *= s;
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) x[q] = e8 == 255 ? __int_as_float(0x7fc00000) : times_pow2(x[q], e8 - 127);
}

// The record of a slot, or null.
__device__ __forceinline__ uint8_t *record_of(const KvArgs &a, int fmt, int slot, int head) {
  const int page = slot / a.page, off = slot % a.page;
  return a.data + (((int64_t)page * a.heads + head) * (a.page >> 4) + (off >> 4)) * kv_record(fmt, a.D);
}

// grid: every lane one (token, head, 8 columns) of the keys and of the values
template <int FMT, bool WRITE>
__global__ void __launch_bounds__(kThreads) kv_kernel(const KvArgs a) {
  pdl_wait();
  pdl_trigger();
  const int n = a.D >> 3;  // lanes of a row: 8, 16 or 32
  const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t r = at / n;
  const int j = (int)(at % n);
  bool live = r < a.rows;
  const int t = live ? (int)(r / a.heads) : 0, head = live ? (int)(r % a.heads) : 0;
  int slot = a.slots[t];
  if (slot >= a.pages * a.page) {
    if (live && j == 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
    slot = -1;
  }
  const bool held = slot >= 0;
  uint8_t *rec = held ? record_of(a, FMT, slot, head) : nullptr;
  const int i = held ? slot % a.page & 15 : 0;
  float x[8];
  if (WRITE) {
    live = live && held;
    float y[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = y[q] = 0.f;
    if (live) {
      raw8_to_f32(load_raw8(a.k, t * a.kst + head * a.ksh + 8 * j, a.type), a.type, x);
      raw8_to_f32(load_raw8(a.v, t * a.vst + head * a.vsh + 8 * j, a.type), a.type, y);
    }
    put8<FMT>(rec, i, 0, j, n, a.D, x, live);
    put8<FMT>(rec, i, 1, j, n, a.D, y, live);
  } else if (live) {
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      void *o = part ? a.vo : a.ko;
      if (!o) continue;
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = 0.f;
      if (held) get8<FMT>(rec, i, part, j, a.D, x);
      store_raw8(o, part ? t * a.vst + head * a.vsh + 8 * j : t * a.kst + head * a.ksh + 8 * j, a.type,
                 f32_to_raw8(x, a.type));
    }
  }
}

template <bool WRITE>
moe_status_t launch(const KvArgs &a, int fmt, cudaStream_t stream, int *launches) {
  const int64_t lanes = a.rows * (a.D >> 3);
  const int64_t ctas = (lanes + kThreads - 1) / kThreads;
  if (ctas == 0) return MOE_OK;
  if (ctas > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ctas), block(kThreads);
  cudaError_t err;
  if (fmt == MOE_KV_BF16)
    err = launch_pdl(kv_kernel<MOE_KV_BF16, WRITE>, grid, block, 0, stream, a);
  else if (fmt == MOE_KV_FP16)
    err = launch_pdl(kv_kernel<MOE_KV_FP16, WRITE>, grid, block, 0, stream, a);
  else if (fmt == MOE_KV_FP8)
    err = launch_pdl(kv_kernel<MOE_KV_FP8, WRITE>, grid, block, 0, stream, a);
  else
    err = launch_pdl(kv_kernel<MOE_KV_NVFP4, WRITE>, grid, block, 0, stream, a);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

KvArgs args_of(const moe_kv_cache_t &c, const int32_t *slots, int T, int type, int64_t kst, int64_t ksh, int64_t vst,
               int64_t vsh, unsigned int *status) {
  KvArgs a = {};
  a.data = static_cast<uint8_t *>(c.data);
  a.slots = slots;
  a.status = status;
  a.kst = kst;
  a.ksh = ksh;
  a.vst = vst;
  a.vsh = vsh;
  a.rows = (int64_t)T * c.kv_heads;
  a.type = type;
  a.T = T;
  a.heads = c.kv_heads;
  a.D = c.head_dim;
  a.page = c.page_size;
  a.pages = c.num_pages;
  return a;
}

}  // namespace

moe_status_t launch_kv_write(const void *k, const void *v, int type, int64_t kst, int64_t ksh, int64_t vst,
                             int64_t vsh, const int32_t *slots, int T, const moe_kv_cache_t &c, unsigned int *status,
                             cudaStream_t stream, int *launches) {
  KvArgs a = args_of(c, slots, T, type, kst, ksh, vst, vsh, status);
  a.k = k;
  a.v = v;
  return launch<true>(a, c.fmt, stream, launches);
}

moe_status_t launch_kv_read(const moe_kv_cache_t &c, const int32_t *slots, int n, void *ko, void *vo, int type,
                            int64_t kst, int64_t ksh, int64_t vst, int64_t vsh, unsigned int *status,
                            cudaStream_t stream, int *launches) {
  KvArgs a = args_of(c, slots, n, type, kst, ksh, vst, vsh, status);
  a.ko = ko;
  a.vo = vo;
  return launch<false>(a, c.fmt, stream, launches);
}

}  // namespace moe4
