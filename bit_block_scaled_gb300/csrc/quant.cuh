// Conversions to and from the 4- and 8-bit formats, and the exponents of
// power-of-two scales.
#pragma once

#include "common.cuh"
#include "types.cuh"

namespace moe4 {

// 2^e for e in -127..127, exactly (2^-127 is a subnormal).
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(e == -127 ? 0x00400000u : (uint32_t)(e + 127) << 23); }

// Least e in -127..127 with amax * 2^-e <= top, 2^x > top >= 2^(x - 1); amax
// below fp32's normal range gives -127, as 0 does.
__device__ __forceinline__ int row_exponent(float amax, float top, int x) {
  const uint32_t a = __float_as_uint(amax);
  const int over = (a & 0x7fffffu) > (__float_as_uint(top) & 0x7fffffu) ? 1 : 0;
  return max((int)(a >> 23) - 126 - x + over, -127);
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

// Largest magnitude of a lane's 8 values, as the bits of that type: they order
// as the magnitudes do, with infinities and NaN above all numbers.
template <int TYPE>
__device__ __forceinline__ uint32_t abs_max(const Raw8 &r) {
  const uint32_t a[4] = {r.a.x, r.a.y, r.a.z, r.a.w}, b[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
  if (TYPE == MOE_FP32) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(a[i] & 0x7fffffffu, b[i] & 0x7fffffffu));
    return m;
  }
  const uint32_t m = __vmaxu2(__vmaxu2(a[0] & 0x7fff7fffu, a[1] & 0x7fff7fffu),
                              __vmaxu2(a[2] & 0x7fff7fffu, a[3] & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}
// The bits of infinity of a type: what is not below is no number.
template <int TYPE>
__device__ __forceinline__ constexpr uint32_t inf_bits() {
  return TYPE == MOE_FP32 ? 0x7f800000u : TYPE == MOE_BF16 ? 0x7f80u : 0x7c00u;
}
template <int TYPE>
__device__ __forceinline__ float from_bits(uint32_t b) {
  if (TYPE == MOE_FP32) return __uint_as_float(b);
  if (TYPE == MOE_BF16) return __uint_as_float(b << 16);
  return __half2float(__ushort_as_half((unsigned short)b));
}

}  // namespace moe4
