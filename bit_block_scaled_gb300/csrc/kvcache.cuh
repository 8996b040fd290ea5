// Record layout of the paged key-value cache (include/moe4.h): 16 tokens of
// one head in one contiguous piece, so that a reader fetches keys, values and
// all their scales with a single bulk copy.
#pragma once

#include "common.cuh"

namespace moe4 {

// Bytes of one token's codes.
__host__ __device__ constexpr int kv_row(int fmt, int D) {
  return fmt == MOE_KV_FP8 ? D : fmt == MOE_KV_NVFP4 ? D / 2 : 2 * D;
}
// Offset of the block scales, of the row exponents, and the record's size.
__host__ __device__ constexpr int kv_scales_at(int fmt, int D) { return 32 * kv_row(fmt, D); }
__host__ __device__ constexpr int kv_exps_at(int fmt, int D) {
  return kv_scales_at(fmt, D) + (fmt == MOE_KV_NVFP4 ? 2 * D : 0);
}
__host__ __device__ constexpr int kv_record(int fmt, int D) {
  return kv_exps_at(fmt, D) + (fmt >= MOE_KV_FP8 ? 32 : 0);
}
// Place of byte p of token i's codes within a section of codes: the 16-byte
// pieces of every 128-byte line are permuted by an exclusive or, so that eight
// rows read at the same column lie in different banks.
__host__ __device__ __forceinline__ int kv_place(int row, int i, int p) {
  const int f = row >= 128 ? (i & 7) : row == 64 ? (i & 6) : ((i >> 1) & 2);
  return (i * row + p) ^ (f << 4);
}

}  // namespace moe4
