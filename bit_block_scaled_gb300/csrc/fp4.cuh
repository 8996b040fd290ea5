// Layout of 4-bit operands (moe_fp4_t in include/moe4.h): packed codes row by
// row, block scales in tiles of 128 rows by 4 blocks.
#pragma once

#include "common.cuh"

namespace moe4 {

// Values a block scale covers.
__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == MOE_FMT_NVFP4 ? 16 : 32; }
// Tiles of 4 blocks along K, and of 128 rows.
__host__ __device__ constexpr int fp4_tiles_k(int fmt, int K) { return (K / fp4_block(fmt) + 3) / 4; }
__host__ __device__ constexpr int64_t fp4_tiles_r(int rows) { return ((int64_t)rows + 127) / 128; }
constexpr int kFp4Tile = 512;  // bytes
// Place of the scale of (row, block): the 4 blocks of a row are 4 consecutive
// bytes, rows 32 apart lie side by side in 16 bytes, and 32 such rows of 16
// bytes are a tile. That is the order in which tensor memory holds them (32
// lanes of 4 columns of 4 bytes), so a tile is copied there as it lies.
__host__ __device__ __forceinline__ int64_t fp4_scale_at(int row, int block, int tiles_k) {
  return ((int64_t)(row >> 7) * tiles_k + (block >> 2)) * kFp4Tile + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (block & 3);
}

}  // namespace moe4
