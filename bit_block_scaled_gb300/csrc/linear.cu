// Product of two 4-bit operands: out[t][n] = rx[t] rw[n] sum_k x[t][k] w[n][k] +
// bias[n] on the block-scaled tensor cores. Codes (128-byte swizzle) and block
// scales come by TMA; the scales go on into tensor memory (tcgen05.cp, each
// 512-byte tile spread over 32 lanes and repeated for the four warps), from where
// tcgen05.mma applies them: the products of a block are exact, sums fp32.
//
// Two kernels:
//  * narrow (few tokens): the weights are the 128 rows of the MMA, the tokens
//    its columns. K is split over a cluster of CTAs whose partial sums are
//    joined through distributed shared memory in the order of K.
//  * wide (many tokens): pairs of CTAs (cta_group::2) share 256 tokens x 192
//    weight rows, persistent, two accumulators so that one tile is written
//    while the next is summed.
#include <cudaTypedefs.h>
#include <string.h>

#include "device.cuh"
#include "fp4.cuh"
#include "kernels.h"
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
  int T, N, K, xr_stride, wr_stride, type, split, stages, tiles_t, tiles_n;
  int bulk_n;  // columns of out that are stored by TMA
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
// codes and scales; sfa and sfb: tensor memory of its scales, 4 and 4 * BLOCKS columns a tile.
template <int FMT, int CG, int BLOCKS>
__device__ __forceinline__ void stage_mmas(uint32_t d, int M, int N, uint64_t a, uint64_t b, uint64_t sa, uint64_t sb,
                                           uint32_t sfa, uint32_t sfb, uint32_t sfb_at, int steps, bool first) {
  constexpr int kSteps = FMT == MOE_FMT_NVFP4 ? 1 : 2;  // MMAs a tile of scales
  auto scales = [&](int t) {
    copy_scales<CG>(sfa + 4 * t, sa + t * (kFp4Tile >> 4));
#pragma unroll
    for (int j = 0; j < BLOCKS; ++j)
      copy_scales<CG>(sfb + 4 * (BLOCKS * t + j), sb + (j * Sf<FMT>::kBytes + t * kFp4Tile) / 16);
  };
  auto multiply = [&](int k) {
    const int t = k / kSteps, id = (k % kSteps) * 2;
    mma_fp4<FMT, CG>(d, a + 2 * k, b + 2 * k, idesc_fp4<FMT>(M, N, id), sfa + 4 * t, sfb + 4 * BLOCKS * t + sfb_at,
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
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float row_scale(const float *r, int stride, int i) { return r ? r[(int64_t)i * stride] : 1.f; }

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
  static constexpr int kJoin = TN * 128 * 4;  // partial sums, over the ring when it is drained
  static constexpr int kSfCols = Sf<FMT>::kTiles * 4 * (1 + kBlocks);
  static constexpr int kUsed = TN + 2 * kSfCols;
  static constexpr int kCols = kUsed <= 32 ? 32 : kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
};

template <int FMT, int TN>
__global__ void __launch_bounds__(kThreads) narrow_kernel(const __grid_constant__ LinArgs p) {
  using S = Narrow<FMT, TN>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 1];
  __shared__ uint32_t tmem_at;
  __shared__ int failed;
  __shared__ float xr_s[TN];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = smem_u32(bars), ring = smem_u32(base);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  const uint32_t done = bar0 + 8u * 2 * kMaxStages;
  // cluster rank = part of K; tiles of weight rows, then of tokens
  const int rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
  const int n0 = tile % p.tiles_n * 128, t0 = tile / p.tiles_n * TN;
  const int all = (p.K + kStageK - 1) / kStageK;
  const int s_begin = (int)((int64_t)all * rank / p.split), s_end = (int)((int64_t)all * (rank + 1) / p.split);

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    mbar_init(done, 1);
    failed = 0;
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
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  pdl_trigger();
  pdl_wait();

  bool ok = true;
  if (warp == 0) {
    Ring r;
    for (int s = s_begin; s < s_end; ++s) {
      if (s - s_begin >= p.stages && !warp_wait(empty(r.slot), r.phase ^ 1)) {
        ok = false;
        break;
      }
      if (elect_one()) {
        const uint32_t a = ring + r.slot * S::kStage, b = a + S::kA, sa = b + S::kB, sb = sa + Sf<FMT>::kBytes;
        mbar_arrive_expect_tx(full(r.slot), S::kStage);
        tma_load_2d(a, &p.tm_w, full(r.slot), s * 128, n0);
        tma_load_2d(b, &p.tm_x, full(r.slot), s * 128, t0);
        tma_load_2d(sa, &p.tm_ws, full(r.slot), s * (Sf<FMT>::kBytes / 8), n0 / 128);
        for (int j = 0; j < S::kBlocks; ++j)
          tma_load_2d(sb + j * Sf<FMT>::kBytes, &p.tm_xs, full(r.slot), s * (Sf<FMT>::kBytes / 8), t0 / 128 + j);
      }
      __syncwarp();
      r.advance(p.stages);
    }
    // where a wait ran out: the copies in flight land before this CTA's memory is given back
    if (!ok)
      for (int s = 0; s < p.stages; ++s) mbar_wait(full(s), s < r.slot ? r.phase : r.phase ^ 1);
  } else if (warp == 1) {
    Ring r;
    for (int s = s_begin; s < s_end && ok; ++s) {
      ok = warp_wait(full(r.slot), r.phase);
      if (ok && elect_one()) {
        tc_fence_after();
        const uint32_t a = ring + r.slot * S::kStage, b = a + S::kA, sa = b + S::kB, sb = sa + Sf<FMT>::kBytes;
        const uint32_t sfa = tmem + TN + (s & 1) * S::kSfCols, sfb = sfa + Sf<FMT>::kTiles * 4;
        stage_mmas<FMT, 1, S::kBlocks>(tmem, 128, TN, smem_desc_sw128(a), smem_desc_sw128(b), scale_desc(sa), scale_desc(sb),
                                       sfa, sfb, 0, (min(p.K - s * kStageK, kStageK) + 63) / 64, s == s_begin);
        umma_commit(empty(r.slot));
        if (s + 1 == s_end) umma_commit(done);
      }
      __syncwarp();
      r.advance(p.stages);
    }
  }
  const int q = warp & 3, n = n0 + q * 32 + lane;  // the writing warps' rows of tensor memory
  float scale = 0.f, bias = 0.f;
  if (warp >= 2) {
    const int e = tid - 64;
    for (int i = e; i < TN; i += kEpiThreads) xr_s[i] = t0 + i < p.T ? row_scale(p.xr, p.xr_stride, t0 + i) : 0.f;
    if (n < p.N) {
      scale = row_scale(p.wr, p.wr_stride, n);
      bias = p.bias ? load_as_f32(p.bias, n, p.type) : 0.f;
    }
    ok = warp_wait(done, 0);
    tc_fence_after();
  }
  if (!ok && lane == 0) {
    raise_status(p.status, MOE_ERR_TIMEOUT);
    failed = 1;
  }
  __syncthreads();
  if (p.split == 1) {
    if (warp >= 2 && !failed) {
      for (int c = 0; c < TN && t0 + c < p.T; c += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (t0 + c + i < p.T && n < p.N)
            store_from_f32(p.out, (t0 + c + i) * p.ldo + n, p.type, fmaf(__uint_as_float(v[i]) * xr_s[c + i], scale, bias));
      }
    }
  } else {
    float *join = reinterpret_cast<float *>(base);  // [TN][128]
    if (warp >= 2) {
      for (int c = 0; c < TN; c += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) join[(c + i) * 128 + q * 32 + lane] = __uint_as_float(v[i]);
      }
    }
    cluster_sync();
    if (!failed) {
      // 4 weight rows of a token a thread, the tokens of this rank; sums in the order of K
      const int c_begin = TN * rank / p.split, c_end = TN * (rank + 1) / p.split;
      for (int i = c_begin * 32 + tid; i < c_end * 32; i += kThreads) {
        const int c = i >> 5, m = (i & 31) * 4, t = t0 + c;
        if (t >= p.T) break;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        const uint32_t from = ring + (c * 128 + m) * 4;
        float4 part[kMaxSplit];
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k)
          if (k < p.split) part[k] = ld_cluster4(at_rank(from, k));
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k)
          if (k < p.split) sum.x += part[k].x, sum.y += part[k].y, sum.z += part[k].z, sum.w += part[k].w;
        const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int nn = n0 + m + j;
          if (nn < p.N) {
            const float b = p.bias ? load_as_f32(p.bias, nn, p.type) : 0.f;
            store_from_f32(p.out, t * p.ldo + nn, p.type, fmaf(v[j] * xr_s[c], row_scale(p.wr, p.wr_stride, nn), b));
          }
        }
      }
    }
    cluster_sync();  // the others may still be reading here
  }
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
  const int all = (a.K + kStageK - 1) / kStageK;
  const int own = (all + a.split - 1) / a.split;
  a.stages = own < 4 ? own : 4;
  uint32_t smem = a.stages * S::kStage;
  if (a.split > 1 && smem < S::kJoin) smem = S::kJoin;
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
constexpr int kWideN = 192, kWideStages = 5, kVecs = 2, kWideEpi = 8, kWideThreads = 64 + 32 * kWideEpi;

template <int FMT>
struct Wide {
  static constexpr int kA = 128 * 128, kB = kWideN / 2 * 128;  // this CTA's half of the pair's rows
  static constexpr int kStage = kA + kB + 3 * Sf<FMT>::kBytes;
  static constexpr int kStageAt = (kStage + 1023) / 1024 * 1024;
  static constexpr int kStaging = 8 * 4096;  // a warp's pieces of 32 rows x 32 columns: two of 16 bits, one of 32
  static constexpr int kSmem = 1024 + kWideStages * kStageAt + kStaging + 2 * kVecs * kWideN * 4;
  static constexpr int kSfA = 2 * kWideN, kSfB = kSfA + Sf<FMT>::kTiles * 4;  // columns behind the accumulators
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
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
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
  __shared__ __align__(8) uint64_t bars[2 * kWideStages + 4];
  __shared__ uint32_t tmem_at;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const uint32_t bar0 = smem_u32(bars), ring = smem_u32(base);
  auto full = [&](int s) { return bar0 + 8u * s; };  // of the first CTA: both CTAs' copies
  auto empty = [&](int s) { return bar0 + 8u * (kWideStages + s); };
  auto accfull = [&](int s) { return bar0 + 8u * (2 * kWideStages + s); };
  auto accempty = [&](int s) { return bar0 + 8u * (2 * kWideStages + 2 + s); };  // of the first CTA
  uint8_t *staging = base + kWideStages * S::kStageAt;
  float *vecs = reinterpret_cast<float *>(staging + S::kStaging);  // [buffer][row scales, biases][kWideN]

  if (tid == 0) {
    for (int s = 0; s < kWideStages; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    for (int s = 0; s < 2; ++s) mbar_init(accfull(s), 1), mbar_init(accempty(s), 2 * kWideEpi);
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
  pdl_trigger();
  pdl_wait();

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
          const uint32_t a = ring + r.slot * S::kStageAt, b = a + S::kA, sa = b + S::kB, sb = sa + Sf<FMT>::kBytes;
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
        if (n >= 2) ok = mbar_wait(accempty(acc), ((n >> 1) - 1) & 1);
        tc_fence_after();
        for (int s = 0; s < all && ok; ++s) {
          ok = mbar_wait(full(r.slot), r.phase);
          if (ok) {
            tc_fence_after();
            const uint32_t at = r.slot * (S::kStageAt >> 4);
            stage_mmas<FMT, 2, 2>(tmem + acc * kWideN, 256, kWideN, a0 + at, b0 + at, sa0 + at, sb0 + at, tmem + S::kSfA,
                                  tmem + S::kSfB, (n0 & 127) >> 5, (min(p.K - s * kStageK, kStageK) + 63) / 64, s == 0);
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
    constexpr int kBytes = TYPE == MOE_FP32 ? 4 : 2, kPiece = 32 * 32 * kBytes, kBufs = S::kStaging / (kWideEpi * kPiece);
    const int q = warp & 3, e = tid - 64, half = (warp - 2) >> 2;
    const uint32_t stage = smem_u32(staging) + (warp - 2) * (kBufs * kPiece);
    int n = 0, piece = 0;
    for (int i = pair; i < total; i += pairs, ++n) {
      int t0, n0;
      wide_tile(p, i, t0, n0);
      const int acc = n & 1, t = t0 + rank * 128 + q * 32 + lane, c0 = half * (kWideN / 2);
      float *scales = vecs + acc * kVecs * kWideN, *biases = scales + kWideN;
      if (e < kWideN) {
        const bool in = n0 + e < p.N;
        scales[e] = in ? row_scale(p.wr, p.wr_stride, n0 + e) : 0.f;
        biases[e] = in && p.bias ? load_as_f32(p.bias, n0 + e, TYPE) : 0.f;
      }
      const float xr = t < p.T ? row_scale(p.xr, p.xr_stride, t) : 0.f;
      asm volatile("bar.sync 1, %0;" ::"r"(kWideEpi * 32) : "memory");
      ok = warp_wait(accfull(acc), (n >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const uint32_t from = tmem + ((uint32_t)(q * 32) << 16) + acc * kWideN + c0;
      uint32_t v[2][32];
      tmem_ld32(from, v[0]);
#pragma unroll
      for (int pc = 0; pc < 3; ++pc) {
        const int c = c0 + 32 * pc, col = n0 + c;
        tmem_ld_wait();
        if (pc < 2) {
          tmem_ld32(from + 32 * (pc + 1), v[(pc + 1) & 1]);
        } else {  // the accumulator is read
          tc_fence_before();
          if (lane == 0) arrive_remote(at_rank(accempty(acc), 0));
        }
        const bool bulk = col < p.bulk_n;
        const uint32_t buf = stage + piece % kBufs * kPiece;
        if (bulk) {  // the piece that was there has been read
          if (lane == 0) {
            if (kBufs == 2)
              asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            else
              asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          }
          __syncwarp();
        }
#pragma unroll
        for (int h = 0; h < 32; h += 8) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 sc = *reinterpret_cast<const float4 *>(scales + c + h + j);
            const float4 bi = *reinterpret_cast<const float4 *>(biases + c + h + j);
            f[j] = fmaf(__uint_as_float(v[pc & 1][h + j]) * xr, sc.x, bi.x);
            f[j + 1] = fmaf(__uint_as_float(v[pc & 1][h + j + 1]) * xr, sc.y, bi.y);
            f[j + 2] = fmaf(__uint_as_float(v[pc & 1][h + j + 2]) * xr, sc.z, bi.z);
            f[j + 3] = fmaf(__uint_as_float(v[pc & 1][h + j + 3]) * xr, sc.w, bi.w);
          }
          if (bulk) {
            // rows of 64 or 128 bytes, 16-byte pieces in the order of that swizzle
            const Raw8 raw = f32_to_raw8(f, TYPE);
            const int at = h * kBytes / 16, x = kBytes == 2 ? (lane >> 1) & 3 : lane & 7;
            const uint32_t to = buf + lane * (32 * kBytes);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + ((at ^ x) << 4)), "r"(raw.a.x), "r"(raw.a.y),
                         "r"(raw.a.z), "r"(raw.a.w)
                         : "memory");
            if (TYPE == MOE_FP32)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((at + 1) ^ x) << 4)), "r"(raw.b.x),
                           "r"(raw.b.y), "r"(raw.b.z), "r"(raw.b.w)
                           : "memory");
          }
          if (col + h + 8 > p.bulk_n && t < p.T) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int at = col + h + j;
              if (at >= p.bulk_n && at < p.N) store_from_f32(p.out, t * p.ldo + at, TYPE, f[j]);
            }
          }
        }
        if (bulk) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (t < p.T) tma_store_2d(&p.tm_out, buf, col, t);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
          ++piece;
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
  // TODO rule
  const bool wide = a.T >= 512;
  const int tn = wide ? 256 : a.T <= 16 ? 16 : a.T <= 32 ? 32 : a.T <= 64 ? 64 : 128;
  const int wn = wide ? kWideN : 128;
  a.tiles_t = (a.T + tn - 1) / tn;
  a.tiles_n = (a.N + wn - 1) / wn;
  if (!map_codes(&a.tm_x, x.q, a.T, a.K, wide ? 128 : tn) || !map_codes(&a.tm_w, w.q, a.N, a.K, wide ? kWideN / 2 : 128) ||
      !map_scales(&a.tm_xs, x.scales, x.fmt, a.T, a.K) || !map_scales(&a.tm_ws, w.scales, w.fmt, a.N, a.K))
    return MOE_ERR_CUDA;
  if (wide) {
    const int bytes = dtype_bytes(type);
    // Rows on the 16-byte grid go out by TMA, as far as a row is a multiple of 16 bytes (a store that is cut off at the
    // tensor's edge was seen to write up to the next such multiple); the rest goes value by value.
    a.bulk_n = ldo * bytes % 16 == 0 ? a.N / (16 / bytes) * (16 / bytes) : 0;
    if (a.bulk_n) {
      const cuuint64_t dims[2] = {(cuuint64_t)a.bulk_n, (cuuint64_t)a.T}, strides[1] = {(cuuint64_t)ldo * bytes};
      const cuuint32_t box[2] = {32, 32};
      const CUtensorMapDataType t = type == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : type == MOE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
      const CUtensorMapSwizzle swizzle = bytes == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
      if (!encode_tiled(&a.tm_out, t, 2, out, dims, strides, box, swizzle)) return MOE_ERR_CUDA;
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
  const int64_t tiles = (int64_t)a.tiles_t * a.tiles_n;
  const int all = (a.K + kStageK - 1) / kStageK;
  a.split = 1;
  while (a.split < kMaxSplit && a.split < all && tiles * (a.split + 1) <= sm_count()) ++a.split;
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
