// Product of two 4-bit operands: out[t][n] = rx[t] rw[n] sum_k x[t][k] w[n][k] +
// bias[n] on the block-scaled tensor cores. Codes (128-byte swizzle) and block
// scales come by TMA; the scales go on into tensor memory (tcgen05.cp, each
// 512-byte tile spread over 32 lanes and repeated for the four warps), from where
// tcgen05.mma applies them: the products of a block are exact, sums fp32.
//
// Two kernels:
//  * narrow (few tokens): the weights are the 128 rows of the MMA, the tokens
//    its columns. K is split over a cluster of CTAs whose partial sums are
//    joined through distributed shared memory in the order of K. Bound by
//    latency for one token (3.8 us at 5120 x 2880), then by what an SM can take
//    in, 64 bytes a cycle (333 x 2880 x 4096 7.4 us).
//  * wide (many tokens): pairs of CTAs (cta_group::2) share 256 tokens x 256
//    weight rows, persistent, two accumulators so that one tile is written
//    while the next is summed. A stage of 256 values of K is 38 KB an SM, 600
//    cycles at 64 bytes, and its MMAs take 512 (16384 products a cycle): bound by
//    the way into the SMs. 256 columns instead of 192, whose two accumulators
//    need no sharing of columns, take 19% fewer bytes a product (16384 x 8192 x
//    8192 347 -> 313 us, 7.0 PFLOP/s, 0.92 of four times the measured bf16 rate).
//    Rows of outputs off the 16-byte grid are written value by value (8192 x 5120 x
//    2880 52 us, with rows of 5121 79).
#include <cudaTypedefs.h>
#include <float.h>
#include <math.h>
#include <string.h>

#include "device.cuh"
#include "fp4.cuh"
#include "kernels.h"
#include "quant.cuh"
#include "tmap.cuh"
#include "types.cuh"

namespace moe4 {

namespace {

constexpr int kStageK = 256;  // values of K a stage: 128 bytes of codes a row
constexpr int kThreads = 192;  // warp 0 loads, warp 1 multiplies, warps 2..5 write
constexpr int kEpiThreads = 128;

struct LinArgs {
  CUtensorMap tm_x, tm_w, tm_xs, tm_ws, tm_out;
  const float *xr, *wr;  // row scales, or NULL
  const void *bias;
  void *out;
  unsigned int *status;
  int64_t ldo;
  int T, N, K, xr_stride, wr_stride, type, split, stages, parts_at, tiles_t, tiles_n;
  int bulk_n;  // columns of out that bulk copies write
};

// 512-byte tiles of scales a stage and block of 128 rows, K values a tile.
template <int FMT>
struct Sf {
  static constexpr int kTiles = kStageK / (4 * fp4_block(FMT));  // 4 or 2
  static constexpr int kBytes = kTiles * kFp4Tile;
};

// Instruction descriptor: E2M1 operands, both K-major, fp32 sums, scales UE4M3
// or UE8M0; id: which half of a tile's 4 bytes a lane holds (32-value blocks).
template <int FMT>
__device__ __forceinline__ uint32_t idesc_fp4(int M, int N, int id) {
  return ((uint32_t)id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (FMT == MOE_FMT_MXFP4 ? 1u << 23 : 0u) |
         ((uint32_t)(M >> 7) << 27) | ((uint32_t)id << 29);
}

// Rows of 16 bytes, 8-row groups 128 bytes apart, no swizzle: a tile of scales.
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  if (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

template <int FMT, int CG>
__device__ __forceinline__ void mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
#define MOE4_MMA(group, kind)                                                                                  \
  asm volatile("{\n\t.reg .pred p;\n\t"                                                                        \
               "setp.ne.b32 p, %6, 0;\n\t"                                                                     \
               "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), \
               "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                                 \
               : "memory")
  if (FMT == MOE_FMT_NVFP4) {
    if (CG == 1)
      MOE4_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else
      MOE4_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
  } else {
    if (CG == 1)
      MOE4_MMA("1", "mxf4.block_scale.scale_vec::2X");
    else
      MOE4_MMA("2", "mxf4.block_scale.scale_vec::2X");
  }
#undef MOE4_MMA
}

// The MMAs of one stage, issued by one thread: `steps` of 64 values of K. a, b, sa, sb: descriptors of the stage's
// codes and scales; sfa and sfb: tensor memory of its scales, 4 and 4 * BLOCKS columns a tile;
// sfb_shift: columns of 32 rows by which the tile begins within its first 128 rows of scales.
template <int FMT, int CG, int BLOCKS>
__device__ __forceinline__ void stage_mmas(uint32_t d, int M, int N, uint64_t a, uint64_t b, uint64_t sa, uint64_t sb,
                                           uint32_t sfa, uint32_t sfb, int steps, bool first, uint32_t sfb_shift = 0) {
  constexpr int kSteps = FMT == MOE_FMT_NVFP4 ? 1 : 2;  // MMAs a tile of scales
  auto scales = [&](int t) {
    copy_scales<CG>(sfa + 4 * t, sa + t * (kFp4Tile >> 4));
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j)
      copy_scales<CG>(sfb + 4 * (BLOCKS * t + j), sb + (j * Sf<FMT>::kBytes + t * kFp4Tile) / 16);
  };
  auto multiply = [&](int k) {
    const int t = k / kSteps, id = (k % kSteps) * 2;
    mma_fp4<FMT, CG>(d, a + 2 * k, b + 2 * k, idesc_fp4<FMT>(M, N, id), sfa + 4 * t, sfb + 4 * BLOCKS * t + sfb_shift,
                     !(first && k == 0));
  };
  if (steps == kStageK / 64) {
#pragma unroll
    for (int t = 0; t < Sf<FMT>::kTiles; ++t) scales(t);
#pragma unroll
    for (int k = 0; k < kStageK / 64; ++k) multiply(k);
  } else {
#pragma unroll 1
    for (int t = 0; t * kSteps < steps; ++t) scales(t);
#pragma unroll 1
    for (int k = 0; k < steps; ++k) multiply(k);
  }
}

__device__ __forceinline__ uint32_t at_rank(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float row_scale(const float *r, int stride, int i) { return r ? r[(int64_t)i * stride] : 1.f; }

// A sum of NVFP4 products, 0 or from 2^-20 to 2^43 and a multiple of 2^-20, times a token's row scale is a normal number or
// exact for scales from 2^-60 to 2^61 and for the 2^-127 of a row of zeros: what follows is rounded once.
__device__ __forceinline__ bool is_near(float r) {
  const uint32_t bits = __float_as_uint(r) & 0x7fffffffu;
  return bits - (67u << 23) < 121u << 23 || bits == 0x00400000u;
}
// Any other one as a 2^h, a at that range's end (subnormal ones: from 2^-82 on), 2^h for the weight's scale.
struct Parted {
  float a, up;
  __device__ __forceinline__ explicit Parted(float r) {
    const int e = (int)(__float_as_uint(r) >> 23 & 255u) - 127;  // infinities and NaN stay what they are
    const int h = is_near(r) ? 0 : e - max(-60, min(e, 60));
    a = r * pow2(-h);
    up = pow2(h);
  }
};
// v xr w + bias for any scales. Where w 2^h would pass fp32's range, v a (2^40 at least, or 0) makes an infinity of the
// largest number, too.
__device__ __forceinline__ float scaled_far(float v, const Parted &xr, float w, float bias) {
  const float m = w * xr.up;
  return fmaf(v * xr.a, fabsf(m) > FLT_MAX && fabsf(w) <= FLT_MAX ? copysignf(FLT_MAX, w) : m, bias);
}

// The whole warp waits, and agrees on the outcome. One lane is then elected to issue (elect.sync, not a comparison of
// the lane: only then the compiler knows that one thread runs, and issues each tcgen05 instruction without a loop over
// lanes; 4096 x 6144 x 8192 184 -> 89 us).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

// A ring slot and its parity.
struct Ring {
  int slot = 0, phase = 0;
  __device__ __forceinline__ void advance(int n) {
    if (++slot == n) slot = 0, phase ^= 1;
  }
};

// ------------------------------------------------------------------- narrow
constexpr int kMaxStages = 8, kMaxSplit = 8;

template <int FMT, int TN>
struct Narrow {
  static constexpr int kA = 128 * 128, kB = TN * 128, kBlocks = (TN + 127) / 128;
  static constexpr int kStage = kA + kB + Sf<FMT>::kBytes * (1 + kBlocks);
  static constexpr int kSfCols = Sf<FMT>::kTiles * 4 * (1 + kBlocks);
  static constexpr int kUsed = TN + kSfCols;
  static constexpr int kCols = kUsed <= 32 ? 32 : kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
};

// 8 sums of tokens from c on, whose row scales are any, into the outputs from i on (`put` below takes nearly all tiles).
// Not inline, so that the code of the others stays together: 64 x 5120 x 2880 6.5 us, with it inline 6.7 to 6.8 (this way
// itself 9.6).
__device__ __noinline__ void put8_far(const LinArgs &p, uint8_t *tile_s, const float *xr_s, int i, int c, int count, int t0, int n,
                                      int row, float scale, float bias, float v0, float v1, float v2, float v3, float v4, float v5,
                                      float v6, float v7) {
  const float v[8] = {v0, v1, v2, v3, v4, v5, v6, v7};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = scaled_far(v[j], Parted(xr_s[c + j]), scale, bias);
    if (n < p.bulk_n)
      store_from_f32(tile_s, (i + j) * 128 + row, p.type, f);
    else if (n < p.N && i + j < count)
      store_from_f32(p.out, (t0 + c + j) * p.ldo + n, p.type, f);
  }
}

template <int FMT, int TN>
__global__ void __launch_bounds__(kThreads) narrow_kernel(const __grid_constant__ LinArgs p) {
  using S = Narrow<FMT, TN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 2];
  __shared__ uint32_t tmem_at;
  __shared__ float xr_s[TN + 8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = smem_u32(bars), ring = smem_u32(base);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  const uint32_t done = bar0 + 8u * 2 * kMaxStages, joined = done + 8;
  // cluster rank = part of K; tiles of weight rows, then of tokens
  const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
  const int n0 = tile % p.tiles_n * 128, t0 = tile / p.tiles_n * TN;
  const int all = (p.K + kStageK - 1) / kStageK;
  const int s_begin = (int)((int64_t)all * rank / p.split), s_end = (int)((int64_t)all * (rank + 1) / p.split);

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    mbar_init(done, 1);
    mbar_init(joined, 1);
    fence_mbar_init();
    prefetch_tmap(&p.tm_w);
    prefetch_tmap(&p.tm_ws);
    prefetch_tmap(&p.tm_x);
    prefetch_tmap(&p.tm_xs);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_at), S::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (p.split > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  pdl_wait();
  pdl_trigger();

  bool ok = true;
  if (warp == 0) {
    if (elect_one()) {
      Ring r;
      for (int s = s_begin; s < s_end; ++s) {
        if (s - s_begin >= p.stages && !mbar_wait(empty(r.slot), r.phase ^ 1)) {
          ok = false;
          break;
        }
        const uint32_t a = ring + r.slot * S::kStage, b = a + S::kA, sa = b + S::kB, sb = sa + Sf<FMT>::kBytes;
        mbar_arrive_expect_tx(full(r.slot), S::kStage);
        tma_load_2d(a, &p.tm_w, full(r.slot), s * 128, n0);
        tma_load_2d(b, &p.tm_x, full(r.slot), s * 128, t0);
        tma_load_2d(sa, &p.tm_ws, full(r.slot), s * (Sf<FMT>::kBytes / 8), n0 / 128);
        for (int j = 0; j < S::kBlocks; ++j)
          tma_load_2d(sb + j * Sf<FMT>::kBytes, &p.tm_xs, full(r.slot), s * (Sf<FMT>::kBytes / 8), t0 / 128 + j);
        r.advance(p.stages);
      }
      // where a wait ran out: the copies in flight land before this CTA's memory is given back
      if (!ok)
        for (int s = 0; s < p.stages; ++s) mbar_wait(full(s), s < r.slot ? r.phase : r.phase ^ 1);
    }
    ok = __all_sync(0xffffffffu, ok);
  } else if (warp == 1) {
    if (elect_one()) {
      Ring r;
      const uint64_t a0 = smem_desc_sw128(ring), b0 = smem_desc_sw128(ring + S::kA), sa0 = scale_desc(ring + S::kA + S::kB),
                     sb0 = scale_desc(ring + S::kA + S::kB + Sf<FMT>::kBytes);
      for (int s = s_begin; s < s_end && ok; ++s) {
        ok = mbar_wait(full(r.slot), r.phase);
        if (ok) {
          tc_fence_after();
          const uint32_t at = r.slot * (S::kStage >> 4);
          stage_mmas<FMT, 1, S::kBlocks>(tmem, 128, TN, a0 + at, b0 + at, sa0 + at, sb0 + at, tmem + TN,
                                         tmem + TN + Sf<FMT>::kTiles * 4, (min(p.K - s * kStageK, kStageK) + 63) / 64,
                                         s == s_begin, (t0 & 127) >> 5);
          umma_commit(empty(r.slot));
          if (s + 1 == s_end) umma_commit(done);
        }
        r.advance(p.stages);
      }
    }
    ok = __all_sync(0xffffffffu, ok);
  }
  const int live = min(TN, p.T - t0);  // tokens of this tile
  // the writing warps' rows of tensor memory are 32 weight rows
  const int q = warp & 3, row = q * 32 + lane, n = n0 + row, e = tid - 64;
  float scale = 0.f, bias = 0.f;
  bool near = true;  // all of the tile's row scales are
  if (warp >= 2) {
    for (int i = e; i < live; i += kEpiThreads) {
      xr_s[i] = row_scale(p.xr, p.xr_stride, t0 + i);
      near &= is_near(xr_s[i]);
    }
    if (n < p.N) {
      scale = row_scale(p.wr, p.wr_stride, n);
      bias = p.bias ? load_as_f32(p.bias, n, p.type) : 0.f;
    }
    near = bar_and(1, kEpiThreads, near);  // xr_s is there
    ok = warp_wait(done, 0);
    tc_fence_after();
  }
  // The ring is empty once `done` is: it becomes this CTA's sums [TN][128] (where K is split), then the outputs [TN][128]
  // as they are written, a token's 128 a bulk copy.
  const uint32_t from = tmem + ((uint32_t)(q * 32) << 16);
  const int bytes = dtype_bytes(p.type);
  float *sums = reinterpret_cast<float *>(base);
  uint8_t *tile_s = base + (p.split > 1 ? TN * 512 : 0);
  int first = 0, count = live;  // the tokens that this CTA writes
  // n sums of the tokens from c on into the outputs from i on; what lies past the tile's tokens is not copied out
  auto put = [&](int i, int c, auto &v) {
    constexpr int n_put = sizeof(v) / 4;
    if (FMT == MOE_FMT_NVFP4 && !near) {
#pragma unroll
      for (int j = 0; j < n_put; j += 8)
        put8_far(p, tile_s, xr_s, i + j, c + j, count, t0, n, row, scale, bias, v[j], v[j + 1], v[j + 2], v[j + 3], v[j + 4],
                 v[j + 5], v[j + 6], v[j + 7]);
      return;
    }
    float f[n_put];
#pragma unroll
    for (int j = 0; j < n_put; ++j) f[j] = fmaf(v[j] * xr_s[c + j], scale, bias);
    if (n < p.bulk_n) {
      if (p.type == MOE_FP32) {
#pragma unroll
        for (int j = 0; j < n_put; ++j) reinterpret_cast<float *>(tile_s)[(i + j) * 128 + row] = f[j];
      } else {
#pragma unroll
        for (int j = 0; j < n_put; ++j)
          reinterpret_cast<uint16_t *>(tile_s)[(i + j) * 128 + row] =
              p.type == MOE_BF16 ? float_to_bf16_bits(f[j]) : __half_as_ushort(__float2half_rn(f[j]));
      }
    } else if (n < p.N) {
      for (int j = 0; j < n_put; ++j)
        if (i + j < count) store_from_f32(p.out, (t0 + c + j) * p.ldo + n, p.type, f[j]);
    }
  };
  if (p.split > 1) {
    // rank d sums and writes the tokens from d * share on; the others' parts of them come to [rank][share][128] behind the ring
    const int share = (live + p.split - 1) / p.split;
    first = min(rank * share, live);
    count = min(share, live - first);
    float *parts = reinterpret_cast<float *>(base + p.parts_at);
    // sums of up to 8 tokens from `i` on of those that this CTA writes, in the order of K
    auto join = [&](auto part) {
      for (int i = 0; i < count; i += 8) {
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < p.split; ++k) {
          const float *from_k = part(k) + i * 128 + row;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += from_k[j * 128];
        }
        put(i, first + i, v);
      }
    };
    if (TN == 16) {
      // few values: each lane stores its own where they belong (one token of 5120 x 2880 in 3 parts 3.8 us, by bulk copies
      // the same, in 4 parts 4.1 against 4.3)
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all ranks run
      if (warp >= 2) {
        const uint32_t to = smem_u32(parts + rank * share * 128 + row);
        uint32_t v[16];
        tmem_ld16(from, v);
        tmem_ld_wait();
        int d = 0, i = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j < live) {
            asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(at_rank(to + i * 512, d)), "r"(v[j]) : "memory");
            if (++i == share) i = 0, ++d;
          }
      }
      __syncwarp();
      cluster_sync();
      if (warp >= 2) join([&](int k) { return parts + k * share * 128; });
    } else {
      if (warp >= 2) {
        for (int c = 0; c < live; c += 16) {
          uint32_t v[16];
          tmem_ld16(from + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) sums[(c + j) * 128 + row] = __uint_as_float(v[j]);
        }
        fence_proxy_async_smem();
      }
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all ranks' barriers are there
      if (warp >= 2) {
        asm volatile("bar.sync 1, %0;" ::"r"(kEpiThreads) : "memory");
        if (e < p.split && e != rank) {
          const int c0 = min(e * share, live), size = (min(c0 + share, live) - c0) * 512;
          if (size)
            asm volatile(
                "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                    at_rank(smem_u32(parts + rank * share * 128), e)),
                "r"(smem_u32(sums + c0 * 128)), "r"(size), "r"(at_rank(joined, e))
                : "memory");
        }
        if (e == 0) mbar_arrive_expect_tx(joined, (p.split - 1) * count * 512);
        ok &= warp_wait(joined, 0);
        join([&](int k) { return k == rank ? sums + first * 128 : parts + k * share * 128; });
      }
    }
  } else if (warp >= 2) {
    for (int c = 0; c < live; c += 16) {
      uint32_t u[16];
      float v[16];
      tmem_ld16(from + c, u);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(u[i]);
      put(c, c, v);
    }
  }
  if (warp >= 2 && n0 < p.bulk_n) {
    fence_proxy_async_smem();
    asm volatile("bar.sync 1, %0;" ::"r"(kEpiThreads) : "memory");
    const int size = min(128, p.bulk_n - n0) * bytes;
    uint8_t *to = static_cast<uint8_t *>(p.out) + ((t0 + first) * p.ldo + n0) * bytes;
    for (int i = e; i < count; i += kEpiThreads)
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to + i * p.ldo * bytes),
                   "r"(smem_u32(tile_s + i * 128 * bytes)), "r"(size)
                   : "memory");
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  if (p.split > 1 && TN > 16) cluster_sync();  // what was sent has arrived
  if (!ok && lane == 0) raise_status(p.status, MOE_ERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kCols);
  }
}

constexpr uint32_t kMaxSmem = 227 * 1024 - 1024;  // dynamic; the static part is small

template <int FMT, int TN>
moe_status_t launch_narrow(LinArgs &a, cudaStream_t stream) {
  using S = Narrow<FMT, TN>;
  auto kern = narrow_kernel<FMT, TN>;
  static PerDevice configured;
  const int set = configured.get([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem) == cudaSuccess ? 1 : 0;
  });
  if (set < 1) return MOE_ERR_CUDA;
  const int all = (a.K + kStageK - 1) / kStageK, own = (all + a.split - 1) / a.split;
  const int parts = a.split > 1 ? (a.split * ((TN + a.split - 1) / a.split) + 8) * 512 : 0;  // and 8 that are read in vain
  // sums and outputs, over the ring, and 8 tokens that are written in vain
  const int tail = (TN + 8) * 128 * dtype_bytes(a.type) + (a.split > 1 ? TN * 512 : 0);
  a.stages = (int)(kMaxSmem - 1024 - parts) / S::kStage;
  if (a.stages > own) a.stages = own;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  a.parts_at = a.stages * S::kStage > tail ? a.stages * S::kStage : tail;
  const uint32_t smem = a.parts_at + parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.tiles_t * a.tiles_n * a.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem + 1024;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// --------------------------------------------------------------------- wide
constexpr int kWideN = 256, kWideStages = 5, kWideEpi = 8, kWideThreads = 64 + 32 * kWideEpi;
// The accumulators of two tiles and 48 columns of scales share 512 columns: the second begins 48 before the first ends. A
// tile's MMAs begin when the writing warps have read what it has in common with the tile before, which they do first.
constexpr int kAcc1 = 208, kWideSf = 464;

template <int FMT>
struct Wide {
  static constexpr int kA = 128 * 128, kB = kWideN / 2 * 128;  // this CTA's half of the pair's rows
  static constexpr int kStage = kA + kB + 3 * Sf<FMT>::kBytes;
  static constexpr int kStaging = kWideEpi * 4096;  // 32 rows x 128 bytes a warp
  static constexpr int kSmem = 1024 + kWideStages * kStage + kStaging + 2 * kWideN * 4;
  static_assert(kStage % 1024 == 0 && kWideSf + 12 * Sf<FMT>::kTiles <= 512, "alignment of the swizzle, tensor memory");
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// The outputs leave L2 first: the operands are read again (8192 x 5120 x 2880 53.7 -> 52.2 us).
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int x, int y) {
  uint64_t policy;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%2, %3}], [%1], %4;" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "l"(policy)
               : "memory");
}
// Arrives on the barrier at this address in both CTAs of the pair once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Tiles in groups of 8 along the tokens, so that the CTAs that run at once share rows and columns in L2.
__device__ __forceinline__ void wide_tile(const LinArgs &p, int i, int &t0, int &n0) {
  const int group = i / (8 * p.tiles_n), first = group * 8, in = i - group * 8 * p.tiles_n;
  const int rows = min(8, p.tiles_t - first);
  t0 = (first + in % rows) * 256;
  n0 = in / rows * kWideN;
}

template <int FMT, int TYPE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1) wide_kernel(const __grid_constant__ LinArgs p) {
  using S = Wide<FMT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bars[2 * kWideStages + 3];
  __shared__ uint32_t tmem_at;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const uint32_t bar0 = smem_u32(bars), ring = smem_u32(base);
  auto full = [&](int s) { return bar0 + 8u * s; };  // of the first CTA: both CTAs' copies
  auto empty = [&](int s) { return bar0 + 8u * (kWideStages + s); };
  auto accfull = [&](int s) { return bar0 + 8u * (2 * kWideStages + s); };
  const uint32_t shared_read = bar0 + 8u * (2 * kWideStages + 2);  // of the first CTA: once a tile, by both CTAs' writing warps
  uint8_t *staging = base + kWideStages * S::kStage;
  float *scales = reinterpret_cast<float *>(staging + S::kStaging), *biases = scales + kWideN;  // of the tile's columns

  if (tid == 0) {
    for (int s = 0; s < kWideStages; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    for (int s = 0; s < 2; ++s) mbar_init(accfull(s), 1);
    mbar_init(shared_read, 2 * kWideEpi);
    fence_mbar_init();
    prefetch_tmap(&p.tm_w);
    prefetch_tmap(&p.tm_ws);
    prefetch_tmap(&p.tm_x);
    prefetch_tmap(&p.tm_xs);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_at)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  pdl_wait();
  pdl_trigger();

  const int total = p.tiles_t * p.tiles_n, all = (p.K + kStageK - 1) / kStageK;
  bool ok = true;
  if (warp == 0) {
    Ring r;
    bool lapped = false;
    for (int i = pair; i < total && ok; i += pairs) {
      int t0, n0;
      wide_tile(p, i, t0, n0);
      for (int s = 0; s < all; ++s) {
        if (lapped && !warp_wait(empty(r.slot), r.phase ^ 1)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t a = ring + r.slot * S::kStage, b = a + S::kA, sa = b + S::kB, sb = sa + Sf<FMT>::kBytes;
          const uint32_t bar = at_rank(full(r.slot), 0);
          if (rank == 0) mbar_arrive_expect_tx(full(r.slot), 2 * S::kStage);
          tma_load_pair(a, &p.tm_x, bar, s * 128, t0 + rank * 128);
          tma_load_pair(b, &p.tm_w, bar, s * 128, n0 + rank * (kWideN / 2));
          tma_load_pair(sa, &p.tm_xs, bar, s * (Sf<FMT>::kBytes / 8), t0 / 128 + rank);
          tma_load_pair(sb, &p.tm_ws, bar, s * (Sf<FMT>::kBytes / 8), n0 / 128);
          tma_load_pair(sb + Sf<FMT>::kBytes, &p.tm_ws, bar, s * (Sf<FMT>::kBytes / 8), n0 / 128 + 1);
        }
        __syncwarp();
        r.advance(kWideStages);
        lapped |= r.phase;
      }
    }
    // where a wait ran out: the copies in flight land before the memory is given back
    if (!ok && rank == 0)
      for (int s = 0; s < kWideStages; ++s) mbar_wait(full(s), s < r.slot ? r.phase : r.phase ^ 1);
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      Ring r;
      int n = 0;
      const uint64_t a0 = smem_desc_sw128(ring), b0 = smem_desc_sw128(ring + S::kA), sa0 = scale_desc(ring + S::kA + S::kB),
                     sb0 = scale_desc(ring + S::kA + S::kB + Sf<FMT>::kBytes);
      for (int i = pair; i < total && ok; i += pairs, ++n) {
        int t0, n0;
        wide_tile(p, i, t0, n0);
        const int acc = n & 1;
        if (n >= 1) ok = mbar_wait(shared_read, (n - 1) & 1);
        tc_fence_after();
        for (int s = 0; s < all && ok; ++s) {
          ok = mbar_wait(full(r.slot), r.phase);
          if (ok) {
            tc_fence_after();
            const uint32_t at = r.slot * (S::kStage >> 4);
            stage_mmas<FMT, 2, 2>(tmem + acc * kAcc1, 256, kWideN, a0 + at, b0 + at, sa0 + at, sb0 + at, tmem + kWideSf,
                                  tmem + kWideSf + 4 * Sf<FMT>::kTiles, (min(p.K - s * kStageK, kStageK) + 63) / 64, s == 0);
            commit_pair(empty(r.slot));
            if (s + 1 == all) commit_pair(accfull(acc));
          }
          r.advance(kWideStages);
        }
      }
    }
    ok = __all_sync(0xffffffffu, ok);
  } else {
    // warps 2..9: 32 rows of tensor memory and one half of the columns each, in pieces of 32 columns
    constexpr int kBytes = TYPE == MOE_FP32 ? 4 : 2, kCols = 128 / kBytes;  // columns of the staging memory
    const int q = warp & 3, e = tid - 64, half = (warp - 2) >> 2;
    uint8_t *stage = staging + (warp - 2) * 4096;
    int n = 0;
    for (int i = pair; i < total; i += pairs, ++n) {
      int t0, n0;
      wide_tile(p, i, t0, n0);
      const int acc = n & 1, t = t0 + rank * 128 + q * 32 + lane;
      static_assert(kWideEpi * 32 == kWideN, "a thread a column");
      const bool in = n0 + e < p.N;
      const float wr = in ? row_scale(p.wr, p.wr_stride, n0 + e) : 0.f, bi = in && p.bias ? load_as_f32(p.bias, n0 + e, TYPE) : 0.f;
      if (n) asm volatile("bar.sync 1, %0;" ::"r"(kWideEpi * 32) : "memory");  // the tile before has used them
      scales[e] = wr;
      biases[e] = bi;
      const float xr = t < p.T ? row_scale(p.xr, p.xr_stride, t) : 1.f;
      const bool near = FMT != MOE_FMT_NVFP4 || __all_sync(0xffffffffu, is_near(xr));
      ok = bar_and(1, kWideEpi * 32, mbar_wait(accfull(acc), (n >> 1) & 1));  // all go on, or none; scales and biases are there
      if (!ok) break;
      tc_fence_after();
      // the columns that the next tile has, too, are the first's last 48 and the second's first: the last two pieces of
      // the upper half, the first two of the lower
      const uint32_t from = tmem + ((uint32_t)(q * 32) << 16) + acc * kAcc1 + half * 128;
      const int turn = acc == 0 && half == 1 ? 2 : 0;
#pragma unroll 1
      for (int g = 0; g < 2; ++g) {  // two pieces at a time; the code is kept small, it is not in the instruction cache at first
        const int pc = (2 * g + turn) & 3;
        uint32_t v[2][32];
        tmem_ld32(from + 32 * pc, v[0]);
        tmem_ld32(from + 32 * pc + 32, v[1]);
        tmem_ld_wait();
        if (g == 0) {
          tc_fence_before();
          if (lane == 0) arrive_remote(at_rank(shared_read, 0));
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int c = half * 128 + 32 * (pc + w);
          float f[4][8];
          if (__builtin_expect(near, 1)) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 sc = *reinterpret_cast<const float4 *>(scales + c + j);
              const float4 bs = *reinterpret_cast<const float4 *>(biases + c + j);
              const uint32_t *u = &v[w][j];
              float *x = &f[j >> 3][j & 7];
              x[0] = fmaf(__uint_as_float(u[0]) * xr, sc.x, bs.x);
              x[1] = fmaf(__uint_as_float(u[1]) * xr, sc.y, bs.y);
              x[2] = fmaf(__uint_as_float(u[2]) * xr, sc.z, bs.z);
              x[3] = fmaf(__uint_as_float(u[3]) * xr, sc.w, bs.w);
            }
          } else {
            const Parted r(xr);
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j >> 3][j & 7] = scaled_far(__uint_as_float(v[w][j]), r, scales[c + j], biases[c + j]);
          }
          // rows of 128 bytes in the staging memory, 16-byte pieces in the order of that swizzle: 64 columns of 16 bits (both
          // pieces), 32 of fp32
          constexpr bool kWhole = TYPE == MOE_FP32;
          const int x = lane & 7, at0 = kWhole ? 0 : 4 * w;
          uint8_t *to = stage + lane * 128;
          if (kWhole || w == 0) {
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // what was there has been read
            __syncwarp();
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const Raw8 raw = f32_to_raw8(f[j], TYPE);
            if (kWhole) {
              *reinterpret_cast<uint4 *>(to + (((2 * j) ^ x) << 4)) = raw.a;
              *reinterpret_cast<uint4 *>(to + (((2 * j + 1) ^ x) << 4)) = raw.b;
            } else {
              *reinterpret_cast<uint4 *>(to + (((at0 + j) ^ x) << 4)) = raw.a;
            }
          }
          if (!kWhole && w == 0) continue;
          const int col = n0 + (kWhole ? c : c - 32);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (col < p.bulk_n && t < p.T) tma_store_2d(&p.tm_out, smem_u32(stage), col, t);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
          if (col + kCols > p.bulk_n) {  // columns that no bulk copy writes: a row at a time
            const int rows = min(32, p.T - (t - lane));
#pragma unroll 1
            for (int o = lane; o < kCols; o += 32)
              if (col + o >= p.bulk_n && col + o < p.N)
#pragma unroll 1
                for (int r = 0; r < rows; ++r) {
                  const uint8_t *from_s = stage + r * 128 + ((o * kBytes) ^ ((r & 7) << 4));
                  uint8_t *out = static_cast<uint8_t *>(p.out) + ((t - lane + r) * p.ldo + col + o) * kBytes;
                  if (TYPE == MOE_FP32)
                    *reinterpret_cast<uint32_t *>(out) = *reinterpret_cast<const uint32_t *>(from_s);
                  else
                    *reinterpret_cast<uint16_t *>(out) = *reinterpret_cast<const uint16_t *>(from_s);
                }
            __syncwarp();
          }
        }
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  if (!ok && lane == 0) raise_status(p.status, MOE_ERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int FMT, int TYPE>
moe_status_t launch_wide(const LinArgs &a, cudaStream_t stream) {
  auto kern = wide_kernel<FMT, TYPE>;
  static PerDevice configured;
  const int set = configured.get([&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Wide<FMT>::kSmem) == cudaSuccess ? 1 : 0;
  });
  if (set < 1) return MOE_ERR_CUDA;
  const int64_t tiles = (int64_t)a.tiles_t * a.tiles_n, pairs = sm_count() / 2;
  const dim3 grid((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
  return launch_pdl(kern, grid, dim3(kWideThreads), Wide<FMT>::kSmem, stream, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Codes: [rows][K / 2] bytes, boxes of 128 bytes of `box` rows.
bool map_codes(CUtensorMap *m, const uint8_t *q, int rows, int K, int box) {
  const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows}, strides[1] = {(cuuint64_t)(K / 2)};
  const cuuint32_t b[2] = {128, (cuuint32_t)box};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q, dims, strides, b, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scales: a row of 512-byte tiles for each 128 rows, as 8-byte elements.
bool map_scales(CUtensorMap *m, const uint8_t *s, int fmt, int rows, int K) {
  const cuuint64_t inner = (cuuint64_t)fp4_tiles_k(fmt, K) * (kFp4Tile / 8);
  const cuuint64_t dims[2] = {inner, (cuuint64_t)fp4_tiles_r(rows)}, strides[1] = {inner * 8};
  const cuuint32_t b[2] = {(cuuint32_t)((fmt == MOE_FMT_NVFP4 ? Sf<MOE_FMT_NVFP4>::kBytes : Sf<MOE_FMT_MXFP4>::kBytes) / 8), 1};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_INT64, 2, s, dims, strides, b, CU_TENSOR_MAP_SWIZZLE_NONE);
}

struct Shape {
  int tn, split;  // tokens a tile (256: the wide kernel), CTAs that share a tile's K
};

// The shape of least estimated time, in us beyond what every launch takes. A stage of 256 values of K takes as long as
// its bytes take into an SM (64 a cycle: 0.18 to 0.30 us for 16 to 128 tokens, 0.31 for the pairs' 256). CTAs that fit
// the SMs' shared memory together share that, for 0.5 us more; another round of them takes 3. Clusters are laid into
// groups of about 19 SMs. Joining parts of K takes 0.4 us for 16 tokens, for more 1 (128 tokens: 1.6) and 0.03 a token that a
// CTA sums; the wide kernel's last tile is written in 1 us more. Measured, in us, the chosen first: 1 x 5120 x 2880 16
// tokens in 3 parts 3.8, whole 5.0; 8 x 8192 x 8192 16 in 2 7.3, whole 10.1; 64 x 5120 x 2880 64 in 3 6.5, whole 6.5, too, in
// 4 11.1; 100 x 2688 x 4096 64 in 3 6.5, whole 7.5, 128 in 6 7.3; 333 x 2880 x 4096 (MXFP4) 64 whole 7.4, 128 7.7, wide 9.0;
// 1024 x 4096 x 4096 wide 9.8, 128 16.9.
Shape choose(int T, int N, int K) {
  const int stages = (K + kStageK - 1) / kStageK, sms = sm_count();
  const int64_t wide_tiles = (int64_t)((T + 255) / 256) * ((N + kWideN - 1) / kWideN), pairs = sms / 2;
  Shape best = {256, 1};
  float least = ((wide_tiles + pairs - 1) / pairs) * stages * 0.31f + 1.0f;
  if (T <= 64) least = INFINITY;  // half of a pair's first tile at most
  constexpr int kTn[4] = {16, 32, 64, 128};
  constexpr float kStageUs[4] = {0.18f, 0.20f, 0.235f, 0.30f};
  for (int i = 0; i < 4; ++i) {
    const int tn = kTn[i];
    if (tn < 64 && T > tn) continue;  // a tile's scales begin on an even column of 32 tokens, or the MMA faults
    const int64_t tiles = (int64_t)((T + tn - 1) / tn) * ((N + 127) / 128);
    for (int split = 1; split <= kMaxSplit && split <= stages; ++split) {
      const int own = (stages + split - 1) / split, stage_bytes = 16384 + tn * 128 + 4096;
      int bytes = own * stage_bytes + (split > 1 ? (tn + 8) * 512 : 0);
      if (bytes > (int)kMaxSmem) bytes = kMaxSmem;
      const int together = (int)kMaxSmem / (bytes + 2048) > 1 ? (int)kMaxSmem / (bytes + 2048) : 1;
      const int64_t ctas = tiles * split, held = (split == 1 || sms < 19 ? sms : sms / 19 * (19 / split) * split) * together;
      const int share = ((tn < T ? tn : T) + split - 1) / split;
      const float join = split == 1 ? 0.f : tn == 16 ? 0.4f : (tn == 128 ? 1.6f : 1.0f) + 0.03f * share;
      const float us = ((ctas + sms - 1) / sms) * own * kStageUs[i] + ((ctas + held - 1) / held - 1) * 3.0f +
                       (ctas > sms ? 0.5f : 0.f) + join + 0.005f * tn;
      if (us < least) least = us, best = {tn, split};
    }
    if (tn >= T) break;
  }
  return best;
}

}  // namespace

moe_status_t launch_fp4_linear(const moe_fp4_t &x, const moe_fp4_t &w, const void *bias, void *out, int type, int64_t ldo,
                               unsigned int *status, cudaStream_t stream, int *launches) {
  LinArgs a;
  memset(&a, 0, sizeof(a));
  a.xr = x.row_scale;
  a.wr = w.row_scale;
  a.xr_stride = x.row_scale_stride;
  a.wr_stride = w.row_scale_stride;
  a.bias = bias;
  a.out = out;
  a.status = status;
  a.ldo = ldo;
  a.T = x.rows;
  a.N = w.rows;
  a.K = x.K;
  a.type = type;
  const Shape shape = choose(a.T, a.N, a.K);
  const int tn = shape.tn;
  if (tn < 64 && a.T > tn) return MOE_ERR_UNSUPPORTED;
  const bool wide = tn == 256;
  const int wn = wide ? kWideN : 128;
  a.tiles_t = (a.T + tn - 1) / tn;
  a.tiles_n = (a.N + wn - 1) / wn;
  if ((int64_t)a.tiles_t * a.tiles_n * shape.split >= (int64_t)1 << 30) return MOE_ERR_UNSUPPORTED;
  if (!map_codes(&a.tm_x, x.q, a.T, a.K, wide ? 128 : tn) || !map_codes(&a.tm_w, w.q, a.N, a.K, wide ? kWideN / 2 : 128) ||
      !map_scales(&a.tm_xs, x.scales, x.fmt, a.T, a.K) || !map_scales(&a.tm_ws, w.scales, w.fmt, a.N, a.K))
    return MOE_ERR_CUDA;
  const int bytes = dtype_bytes(type);
  // Rows on the 16-byte grid go out by bulk copies, as far as a row is a multiple of 16 bytes (a tensor store that is cut
  // off at the tensor's edge was seen to write up to the next such multiple); the rest goes value by value.
  a.bulk_n = ldo * bytes % 16 == 0 ? a.N / (16 / bytes) * (16 / bytes) : 0;
  if (wide) {
    if (a.bulk_n) {
      const cuuint64_t dims[2] = {(cuuint64_t)a.bulk_n, (cuuint64_t)a.T}, strides[1] = {(cuuint64_t)ldo * bytes};
      const cuuint32_t box[2] = {(cuuint32_t)(128 / bytes), 32};
      const CUtensorMapDataType t = type == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : type == MOE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
      if (!encode_tiled(&a.tm_out, t, 2, out, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B)) return MOE_ERR_CUDA;
    }
    if (launches) ++*launches;
#define MOE4_WIDE(F)                                                       \
  if (x.fmt == F) {                                                        \
    if (type == MOE_BF16) return launch_wide<F, MOE_BF16>(a, stream);      \
    if (type == MOE_FP16) return launch_wide<F, MOE_FP16>(a, stream);      \
    return launch_wide<F, MOE_FP32>(a, stream);                            \
  }
    MOE4_WIDE(MOE_FMT_NVFP4)
    MOE4_WIDE(MOE_FMT_MXFP4)
#undef MOE4_WIDE
  }
  a.split = shape.split;
  if (launches) ++*launches;
#define MOE4_NARROW(F)                                         \
  if (x.fmt == F) {                                            \
    if (tn == 16) return launch_narrow<F, 16>(a, stream);      \
    if (tn == 32) return launch_narrow<F, 32>(a, stream);      \
    if (tn == 64) return launch_narrow<F, 64>(a, stream);      \
    return launch_narrow<F, 128>(a, stream);                   \
  }
  MOE4_NARROW(MOE_FMT_NVFP4)
  MOE4_NARROW(MOE_FMT_MXFP4)
#undef MOE4_NARROW
  return MOE_ERR_UNSUPPORTED;
}

}  // namespace moe4
