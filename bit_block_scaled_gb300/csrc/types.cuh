// Reading and writing values of a run-time type (moe_dtype_t) as fp32.
#pragma once

#include "common.cuh"

namespace moe4 {

__host__ __device__ constexpr int dtype_bytes(int type) { return type == MOE_FP32 ? 4 : 2; }
inline bool valid_dtype(int type) { return type >= MOE_BF16 && type <= MOE_FP32; }

__device__ __forceinline__ float load_as_f32(const void *p, int64_t i, int type) {
  if (type == MOE_BF16) return __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
  if (type == MOE_FP16) return __half2float(static_cast<const __half *>(p)[i]);
  return static_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_from_f32(void *p, int64_t i, int type, float v) {
  if (type == MOE_BF16)
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else if (type == MOE_FP16)
    static_cast<__half *>(p)[i] = __float2half_rn(v);
  else
    static_cast<float *>(p)[i] = v;
}

// Eight consecutive values as they lie in memory; a 16-bit type uses a alone.
struct Raw8 {
  uint4 a, b;
};

__device__ __forceinline__ Raw8 load_raw8(const void *p, int64_t i, int type) {
  Raw8 r;
  if (type == MOE_FP32) {
    const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
    r.a = q[0];
    r.b = q[1];
  } else {
    r.a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
    r.b = make_uint4(0, 0, 0, 0);
  }
  return r;
}

__device__ __forceinline__ void raw8_to_f32(const Raw8 &r, int type, float (&v)[8]) {
  const uint32_t a[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  if (type == MOE_FP32) {
    const uint32_t b[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else if (type == MOE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ Raw8 f32_to_raw8(const float (&v)[8], int type) {
  Raw8 r;
  uint32_t a[4], b[4] = {0, 0, 0, 0};
  if (type == MOE_FP32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = __float_as_uint(v[i]);
      b[i] = __float_as_uint(v[4 + i]);
    }
  } else if (type == MOE_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      a[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      a[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
  }
  r.a = make_uint4(a[0], a[1], a[2], a[3]);
  r.b = make_uint4(b[0], b[1], b[2], b[3]);
  return r;
}

__device__ __forceinline__ void store_raw8(void *p, int64_t i, int type, const Raw8 &r) {
  if (type == MOE_FP32) {
    uint4 *q = reinterpret_cast<uint4 *>(static_cast<float *>(p) + i);
    q[0] = r.a;
    q[1] = r.b;
  } else {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = r.a;
  }
}

}  // namespace moe4
