// Writing tokens into the paged key-value cache, quantised, and reading them
// back.
//
// D / 8 lanes take one (token, head): each holds 8 values of the key and 8 of
// the value, so a row's largest magnitude is log2(D / 8) shuffles, a block of
// 16 is two lanes, and a lane's codes are one 4-, 8- or 16-byte store.
//
// Row scales are powers of two: x / r is exact, so an FP8 code is one rounding
// of x / r, and an NVFP4 code one rounding of the quotient x / r / s by the
// E4M3 scale. Quotients that lie on a tie of E2M1 are exact in fp32 and others
// cannot round onto one: x differs from the tie times s, of at most 7 significant
// bits, by a step of fp32 at least, and s < 2 in the units of its leading bit, so
// that the quotient differs from the tie by more than half a step. The same holds
// for m / 6 and the ties of E4M3. So the codes are those of real arithmetic.
#include "common.cuh"
#include "kernels.h"
#include "kvput.cuh"
#include "types.cuh"

namespace moe4 {

namespace {

constexpr int kThreads = 128;

struct KvArgs {
  uint8_t *data;
  const void *k, *v;
  void *ko, *vo;
  const int32_t *slots;
  unsigned int *status;
  int64_t kst, ksh, vst, vsh;
  uint32_t rows;  // T * heads
  int type, heads, D, log_n, page, pages;
};

// A lane's 8 values of a row as they are stored.
template <int FMT>
struct Stored {
  uint4 codes;  // 16, 8 or 4 bytes of it
  uint32_t block_scale, exponent;
  __device__ __forceinline__ void load(const uint8_t *rec, int i, int part, int j, int D) {
    const int row = kv_row(FMT, D);
    const uint8_t *p = rec + part * 16 * row;
    if (FMT == MOE_KV_BF16 || FMT == MOE_KV_FP16) {
      codes = *reinterpret_cast<const uint4 *>(p + kv_place(row, i, 16 * j));
      return;
    }
    exponent = rec[kv_exps_at(FMT, D) + part * 16 + i];
    if (FMT == MOE_KV_FP8) {
      const uint2 c = *reinterpret_cast<const uint2 *>(p + kv_place(row, i, 8 * j));
      codes.x = c.x;
      codes.y = c.y;
    } else {
      codes.x = *reinterpret_cast<const uint32_t *>(p + kv_place(row, i, 4 * j));
      block_scale = rec[kv_scales_at(FMT, D) + part * D + (j >> 1) * 16 + i];
    }
  }
  __device__ __forceinline__ void expand(float (&x)[8]) const {
    if (FMT == MOE_KV_BF16 || FMT == MOE_KV_FP16) {
      raw8_to_f32(Raw8{codes, codes}, FMT == MOE_KV_BF16 ? MOE_BF16 : MOE_FP16, x);
      return;
    }
    float down = exponent == 255u ? __int_as_float(0x7fc00000) : pow2((int)exponent - 127);
    if (FMT == MOE_KV_FP8) {
      const uint32_t w[4] = {codes.x & 0xFFFFu, codes.x >> 16, codes.y & 0xFFFFu, codes.y >> 16};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = e4m3x2_f32(w[q]);
        x[2 * q] = f.x;
        x[2 * q + 1] = f.y;
      }
    } else {
      e2m1x8_f32(codes.x, x);
      const float s = e4m3x2_f32(block_scale).x;
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] *= s;  // apart from 2^e, whose product with s may leave fp32's normal range
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] *= down;
  }
};

// Every lane R (token, head, 8 columns) of the keys and of the values, R * (128
// >> a.log_n) rows a CTA, 1 << a.log_n lanes a row. All loads that do not
// depend on one another come first: with few instructions a row, the time goes
// into waiting for memory.
template <int FMT, int TYPE, bool WRITE, int R>
__global__ void __launch_bounds__(kThreads) kv_kernel(const KvArgs a) {
  pdl_wait();
  pdl_trigger();
  const int n = 1 << a.log_n, j = threadIdx.x & (n - 1);
  const uint32_t per = kThreads >> a.log_n, r0 = blockIdx.x * (per * R) + (threadIdx.x >> a.log_n);
  bool live[R], held[R];
  uint32_t t[R], head[R];
  int slot[R];
  Raw8 k[R], v[R];
#pragma unroll
  for (int x = 0; x < R; ++x) {
    const uint32_t r = r0 + x * per;
    live[x] = r < a.rows;
    t[x] = live[x] ? r / (uint32_t)a.heads : 0;
    head[x] = live[x] ? r - t[x] * a.heads : 0;
    slot[x] = a.slots[t[x]];
    if (WRITE) {
      k[x] = load_raw8(a.k, (int64_t)t[x] * a.kst + (int64_t)head[x] * a.ksh + 8 * j, TYPE);
      v[x] = load_raw8(a.v, (int64_t)t[x] * a.vst + (int64_t)head[x] * a.vsh + 8 * j, TYPE);
    }
  }
  uint8_t *rec[R];
  Stored<FMT> ks[R], vs[R];
#pragma unroll
  for (int x = 0; x < R; ++x) {
    if (slot[x] >= a.pages * a.page) {
      if (live[x] && j == 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
      slot[x] = -1;
    }
    held[x] = live[x] && slot[x] >= 0;
    rec[x] = nullptr;
    if (held[x]) {
      const uint32_t block = (uint32_t)slot[x] >> 4, page16 = (uint32_t)a.page >> 4, page = block / page16;
      rec[x] = a.data + (((int64_t)page * a.heads + head[x]) * page16 + (block - page * page16)) * kv_record(FMT, a.D);
      if (!WRITE) {
        if (a.ko) ks[x].load(rec[x], slot[x] & 15, 0, j, a.D);
        if (a.vo) vs[x].load(rec[x], slot[x] & 15, 1, j, a.D);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < R; ++x) {
    if (WRITE) {
      put8<FMT, TYPE>(rec[x], slot[x] & 15, 0, j, n, a.D, k[x], held[x]);
      put8<FMT, TYPE>(rec[x], slot[x] & 15, 1, j, n, a.D, v[x], held[x]);
    } else if (live[x]) {
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (a.ko) {
        if (held[x]) ks[x].expand(y);
        store_raw8(a.ko, (int64_t)t[x] * a.kst + (int64_t)head[x] * a.ksh + 8 * j, TYPE, f32_to_raw8(y, TYPE));
      }
      if (a.vo) {
        if (held[x]) vs[x].expand(y);
        store_raw8(a.vo, (int64_t)t[x] * a.vst + (int64_t)head[x] * a.vsh + 8 * j, TYPE, f32_to_raw8(y, TYPE));
      }
    }
  }
}

template <bool WRITE>
moe_status_t launch(const KvArgs &a, int fmt, cudaStream_t stream, int *launches) {
  // one row a lane until there are CTAs enough for every SM twice over (304), then four
  const uint32_t per = kThreads >> a.log_n;
  const bool many = a.rows > 4 * 304 * per;
  const uint32_t step = many ? 4 * per : per;
  const dim3 grid(a.rows / step + (a.rows % step != 0)), block(kThreads);
  using Kernel = void (*)(KvArgs);
#define MOE4_KV(F, T) {kv_kernel<F, T, WRITE, 1>, kv_kernel<F, T, WRITE, 4>}
#define MOE4_KV_TYPES(F) {MOE4_KV(F, MOE_BF16), MOE4_KV(F, MOE_FP16), MOE4_KV(F, MOE_FP32)}
  static const Kernel kernels[4][3][2] = {MOE4_KV_TYPES(MOE_KV_BF16), MOE4_KV_TYPES(MOE_KV_FP16),
                                          MOE4_KV_TYPES(MOE_KV_FP8), MOE4_KV_TYPES(MOE_KV_NVFP4)};
#undef MOE4_KV_TYPES
#undef MOE4_KV
  const cudaError_t err = launch_pdl(kernels[fmt][a.type][many], grid, block, 0, stream, a);
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
  a.rows = (uint32_t)((int64_t)T * c.kv_heads);
  a.type = type;
  a.heads = c.kv_heads;
  a.D = c.head_dim;
  a.log_n = c.head_dim == 64 ? 3 : c.head_dim == 128 ? 4 : 5;
  a.page = c.page_size;
  a.pages = c.num_pages;
  return a;
}

}  // namespace

moe_status_t launch_kv_write(const void *k, const void *v, int type, int64_t kst, int64_t ksh, int64_t vst,
                             int64_t vsh, const int32_t *slots, int T, const moe_kv_cache_t &c, unsigned int *status,
                             cudaStream_t stream, int *launches) {
  if ((int64_t)T * c.kv_heads >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  KvArgs a = args_of(c, slots, T, type, kst, ksh, vst, vsh, status);
  a.k = k;
  a.v = v;
  return launch<true>(a, c.fmt, stream, launches);
}

moe_status_t launch_kv_read(const moe_kv_cache_t &c, const int32_t *slots, int n, void *ko, void *vo, int type,
                            int64_t kst, int64_t ksh, int64_t vst, int64_t vsh, unsigned int *status,
                            cudaStream_t stream, int *launches) {
  if ((int64_t)n * c.kv_heads >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  KvArgs a = args_of(c, slots, n, type, kst, ksh, vst, vsh, status);
  a.ko = ko;
  a.vo = vo;
  return launch<false>(a, c.fmt, stream, launches);
}

}  // namespace moe4
