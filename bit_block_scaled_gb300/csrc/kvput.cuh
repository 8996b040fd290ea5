// Quantising one lane's share of a cache row into its record.
#pragma once

#include "kvcache.cuh"
#include "quant.cuh"

namespace moe4 {

// Quantises a lane's 8 values of a row and stores its codes (and the scales
// that fall to this lane). rec: the record; i: token in it; part: 0 keys, 1
// values; j: lane of the row; n: lanes of the row.
template <int FMT, int TYPE>
__device__ __forceinline__ void put8(uint8_t *rec, int i, int part, int j, int n, int D, const Raw8 &raw, bool live) {
  const int row = kv_row(FMT, D);
  uint8_t *codes = rec + part * 16 * row;
  float x[8];
  if (FMT == MOE_KV_BF16 || FMT == MOE_KV_FP16) {
    constexpr int kTo = FMT == MOE_KV_BF16 ? MOE_BF16 : MOE_FP16;
    Raw8 r = raw;
    if (TYPE != kTo) {
      raw8_to_f32(raw, TYPE, x);
      r = f32_to_raw8(x, kTo);
    }
    if (live) *reinterpret_cast<uint4 *>(codes + kv_place(row, i, 16 * j)) = r.a;
    return;
  }
  const uint32_t own = abs_max<TYPE>(raw);
  uint32_t top = own;
  for (int o = 1; o < n; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool bad = top >= inf_bits<TYPE>();
  const int e = FMT == MOE_KV_FP8 ? row_exponent(from_bits<TYPE>(top), 448.f, 9) : row_exponent(from_bits<TYPE>(top), 2688.f, 12);
  const float up = pow2(-e);  // e is at most 120 for finite values; a bad row's codes are not used
  raw8_to_f32(raw, TYPE, x);
#pragma unroll
  for (int q = 0; q < 8; ++q) x[q] *= up;
  if (FMT == MOE_KV_FP8) {
    uint2 c;
    c.x = e4m3x2(x[0], x[1]) | (e4m3x2(x[2], x[3]) << 16);
    c.y = e4m3x2(x[4], x[5]) | (e4m3x2(x[6], x[7]) << 16);
    if (bad) c = make_uint2(0, 0);
    if (live) *reinterpret_cast<uint2 *>(codes + kv_place(row, i, 8 * j)) = c;
  } else {
    // two lanes hold a block of 16
    const float m = from_bits<TYPE>(max(own, __shfl_xor_sync(0xffffffffu, own, 1))) * up;
    const uint32_t sb = bad ? 0u : e4m3x2(m / 6.0f, 0.f) & 0xFFu;
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

}  // namespace moe4
