// Quantising rows to 4-bit operands (NVFP4, MXFP4), reading them back, and
// laying out the block scales of a checkpoint.
//
// NVFP4: row scale r = 2^e, the least with amax / r <= 6 * 448; block scales s
// = E4M3(amax16 / r / 6); codes E2M1(x / r / s). MXFP4: s = 2^e, the least with
// amax32 / s <= 6; codes E2M1(x / s). Scaling by powers of two is exact. An fp32
// value's x / r / s is a true quotient (kvcache.cu says why its rounding moves it
// over no tie of E2M1). A 16-bit one is multiplied by 1 / s rounded up, and the
// product cut off: x and a tie times s (4 + 3 bits) are equal or differ by 2^-12 of
// them, the product before the cut is too large by 2^-23 at most, so that no product
// reaches a tie from below, and one on a tie is cut to the tie itself for each of
// the 8 significands of s and 7 ties, as amax16 / r / 6 is for the ties of E4M3
// (tests/test_fp4_rounding.py tries them all).
//
// Bound by memory: 2 bytes of a value are read, 9/16 or 17/32 written (16384 x
// 8192 into MXFP4 at 99% of the copy bandwidth, into NVFP4, which waits for a row's
// largest value first, at 83%). A lane holds 16 consecutive values (an NVFP4 block,
// half an MXFP4 one), a row stays in the registers of 1 to 8 warps, so it is read once.
#include "fp4.cuh"
#include "kernels.h"
#include "quant.cuh"

namespace moe4 {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;

struct QuantArgs {
  const void *x;
  int64_t ld;
  uint8_t *q, *scales;
  float *row_scale;
  int T, K, units, tiles_k, W;  // units of 16 values; W warps a row
};

// x f for pairs of values, cut off towards zero.
__device__ __forceinline__ void scale8_rz(float (&x)[8], float f) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%0, %1};\n\t"
        "mov.b64 b, {%2, %2};\n\t"
        "mul.rz.f32x2 a, a, b;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "+f"(x[i]), "+f"(x[i + 1])
        : "f"(f));
}

template <int TYPE>
__device__ __forceinline__ uint32_t half_max(const Raw8 (&r)[2]) { return max(abs_max<TYPE>(r[0]), abs_max<TYPE>(r[1])); }

template <int FMT, int TYPE, int P>
__global__ void __launch_bounds__(kWarps * 32) fp4_quantize_kernel(const QuantArgs a) {
  __shared__ uint32_t tops[kWarps];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = kWarps / a.W, wr = warp % a.W;  // rows of a CTA, this warp's part of its row
  const int64_t row = (int64_t)blockIdx.x * per + warp / a.W;
  const bool live = row < a.T;
  Raw8 raw[P][2];
  uint32_t top = 0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int u = (p * a.W + wr) * 32 + lane;
    if (live && u < a.units) {
      raw[p][0] = load_raw8(a.x, row * a.ld + 16 * u, TYPE);
      raw[p][1] = load_raw8(a.x, row * a.ld + 16 * u + 8, TYPE);
    } else {
      raw[p][0].a = raw[p][0].b = raw[p][1].a = raw[p][1].b = make_uint4(0, 0, 0, 0);
    }
  }
  float up = 1.f, pre = 1.f;  // the row's factor 1 / r, and what of it is applied ahead so that up / s stays finite
  bool bad = false;
  if (FMT == MOE_FMT_NVFP4) {
#pragma unroll
    for (int p = 0; p < P; ++p) top = max(top, half_max<TYPE>(raw[p]));
    top = __reduce_max_sync(kAll, top);
    if (a.W > 1) {
      if (lane == 0) tops[warp] = top;
      __syncthreads();
      for (int w = 0; w < a.W; ++w) top = max(top, tops[warp - wr + w]);
    }
    bad = top >= inf_bits<TYPE>();
    const int e = row_exponent(from_bits<TYPE>(top), 2688.f, 12);
    // e is at most 117 for finite values (a bad row's codes are not used), so that up / s, s <= 448, is a normal number
    if (TYPE != MOE_FP32 && e < -110) pre = 0x1p64f;
    up = pow2(pre > 1.f ? -e - 64 : -e);
    if (live && wr == 0 && lane == 0) a.row_scale[row] = bad ? __int_as_float(0x7fc00000) : pow2(e);
  }
  if (!live) return;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int u0 = (p * a.W + wr) * 32, u = u0 + lane;
    if (u0 >= a.units) break;
    float x[2][8];
    raw8_to_f32(raw[p][0], TYPE, x[0]);
    raw8_to_f32(raw[p][1], TYPE, x[1]);
    uint32_t sb;
    bool none = bad;
    if (FMT == MOE_FMT_NVFP4) {
      const float top16 = from_bits<TYPE>(half_max<TYPE>(raw[p]));
      if (TYPE == MOE_FP32) {
        sb = e4m3x2(top16 * up / 6.0f, 0.f) & 0xFFu;
      } else {
        constexpr float kSixth = 0.16666667163372039794921875f;  // rounded up
        sb = e4m3x2(__fmul_rz(top16 * pre, kSixth * up), 0.f) & 0xFFu;
      }
      if (bad) sb = 0;
      const float s = e4m3x2_f32(sb).x;
      none = !(s > 0.f);
      if (TYPE == MOE_FP32) {
#pragma unroll
        for (int q = 0; q < 16; ++q) x[q >> 3][q & 7] = none ? 0.f : x[q >> 3][q & 7] * up / s;
      } else {
        if (pre > 1.f) {
#pragma unroll
          for (int q = 0; q < 16; ++q) x[q >> 3][q & 7] *= pre;
        }
        const float f = none ? 0.f : __frcp_ru(s) * up;
        scale8_rz(x[0], f);
        scale8_rz(x[1], f);
      }
    } else {
      const uint32_t own = half_max<TYPE>(raw[p]), m = max(own, __shfl_xor_sync(kAll, own, 1));
      none = m >= inf_bits<TYPE>();
      const int e = row_exponent(from_bits<TYPE>(m), 6.f, 3);
      sb = none ? 255u : (uint32_t)(e + 127);
      const float down = pow2(-e);
#pragma unroll
      for (int q = 0; q < 16; ++q) x[q >> 3][q & 7] *= down;
    }
    uint2 c = make_uint2(e2m1x8(x[0]), e2m1x8(x[1]));
    if (none) c = make_uint2(0, 0);
    if (u < a.units)
      *reinterpret_cast<uint2 *>(a.q + row * (a.K / 2) + 8 * u) = c;
    else
      sb = 0;
    // four blocks' scales are four bytes side by side; blocks past the row are 0
    constexpr int kLanes = FMT == MOE_FMT_NVFP4 ? 1 : 2;
    sb |= __shfl_down_sync(kAll, sb, kLanes) << 8;
    sb |= __shfl_down_sync(kAll, sb, 2 * kLanes) << 16;
    if (lane % (4 * kLanes) == 0 && u < a.units)
      *reinterpret_cast<uint32_t *>(a.scales + fp4_scale_at((int)row, u / kLanes, a.tiles_k)) = sb;
  }
}

struct DequantArgs {
  const uint8_t *q, *scales;
  const float *row_scale;
  void *out;
  int64_t ld;
  int T, K, units, tiles_k, rs_stride;
};

// A lane 16 values: code * s is exact (6 bits), the row scale's factor and the
// output type round once each.
template <int FMT, int TYPE>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(const DequantArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, row = at / a.units;
  const int u = (int)(at - row * a.units);
  if (row >= a.T) return;
  const uint2 c = *reinterpret_cast<const uint2 *>(a.q + row * (a.K / 2) + 8 * u);
  const uint32_t sb = a.scales[fp4_scale_at((int)row, FMT == MOE_FMT_NVFP4 ? u : u >> 1, a.tiles_k)];
  const float r = a.row_scale ? a.row_scale[row * a.rs_stride] : 1.f;
  const float s = FMT == MOE_FMT_NVFP4 ? e4m3x2_f32(sb).x : sb == 255u ? __int_as_float(0x7fc00000) : pow2((int)sb - 127);
  float x[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    e2m1x8_f32(h ? c.y : c.x, x);
#pragma unroll
    for (int q = 0; q < 8; ++q) x[q] = x[q] * s * r;
    store_raw8(a.out, row * a.ld + 16 * u + 8 * h, TYPE, f32_to_raw8(x, TYPE));
  }
}

// A thread the 4 scales of a row in one tile.
__global__ void __launch_bounds__(256) fp4_pack_scales_kernel(const uint8_t *plain, int rows, int blocks, int tiles_k,
                                                              uint8_t *out) {
  pdl_wait();
  pdl_trigger();
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, row = at / tiles_k;
  const int t = (int)(at - row * tiles_k);
  if (row >= rows) return;
  uint32_t w = 0;
  for (int i = 0; i < 4; ++i)
    if (4 * t + i < blocks) w |= (uint32_t)plain[row * blocks + 4 * t + i] << (8 * i);
  *reinterpret_cast<uint32_t *>(out + fp4_scale_at((int)row, 4 * t, tiles_k)) = w;
}

}  // namespace

moe_status_t launch_fp4_quantize(const void *x, int type, int64_t ld, const moe_fp4_t &f, cudaStream_t stream,
                                 int *launches) {
  QuantArgs a = {x, ld, f.q, f.scales, f.row_scale, f.rows, f.K, f.K / 16, fp4_tiles_k(f.fmt, f.K), 1};
  // Few rows: as many warps a row as there are loads for, so that a lane waits for one load. Many rows: one warp a row while
  // 4 loads a lane hold it (2 in fp32, whose values take twice the registers): with 8, registers leave room for half the
  // warps (16384 x 8192 into NVFP4 67 us against 61, into MXFP4 58 against 51), with 2, rows wait for more warps (69, 53).
  const int most = type == MOE_FP32 ? 2 : 4;
  auto units_of = [&](int w) { return (a.units + 32 * w - 1) / (32 * w); };
  if (a.T <= 4 * 152)
    while (a.W < kWarps && units_of(a.W) > 1) a.W *= 2;
  else
    while (a.W < kWarps && units_of(a.W) > most) a.W *= 2;
  const int need = units_of(a.W), p = need <= 4 ? need - 1 : 4;
  if (need > 8) return MOE_ERR_UNSUPPORTED;
  using Kernel = void (*)(QuantArgs);
#define MOE4_Q(F, T) {fp4_quantize_kernel<F, T, 1>, fp4_quantize_kernel<F, T, 2>, fp4_quantize_kernel<F, T, 3>, \
                      fp4_quantize_kernel<F, T, 4>, fp4_quantize_kernel<F, T, 8>}
#define MOE4_Q_TYPES(F) {MOE4_Q(F, MOE_BF16), MOE4_Q(F, MOE_FP16), MOE4_Q(F, MOE_FP32)}
  static const Kernel kernels[2][3][5] = {MOE4_Q_TYPES(MOE_FMT_NVFP4), MOE4_Q_TYPES(MOE_FMT_MXFP4)};
#undef MOE4_Q_TYPES
#undef MOE4_Q
  const int per = kWarps / a.W;
  const dim3 grid(a.T / per + (a.T % per != 0));
  const cudaError_t err = launch_pdl(kernels[f.fmt][type][p], grid, dim3(kWarps * 32), 0, stream, a);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t launch_fp4_dequantize(const moe_fp4_t &f, void *out, int type, int64_t ld, cudaStream_t stream,
                                   int *launches) {
  const DequantArgs a = {f.q, f.scales, f.row_scale, out, ld, f.rows, f.K, f.K / 16, fp4_tiles_k(f.fmt, f.K),
                         f.row_scale_stride};
  using Kernel = void (*)(DequantArgs);
#define MOE4_D(F) {fp4_dequantize_kernel<F, MOE_BF16>, fp4_dequantize_kernel<F, MOE_FP16>, fp4_dequantize_kernel<F, MOE_FP32>}
  static const Kernel kernels[2][3] = {MOE4_D(MOE_FMT_NVFP4), MOE4_D(MOE_FMT_MXFP4)};
#undef MOE4_D
  const int64_t n = (int64_t)a.T * a.units, grid = (n + 255) / 256;
  if (grid >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  const cudaError_t err = launch_pdl(kernels[f.fmt][type], dim3((unsigned)grid), dim3(256), 0, stream, a);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t launch_fp4_pack_scales(const uint8_t *plain, int fmt, int rows, int K, uint8_t *out, cudaStream_t stream,
                                    int *launches) {
  const int tiles_k = fp4_tiles_k(fmt, K);
  const int64_t grid = ((int64_t)rows * tiles_k + 255) / 256;
  if (grid >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  const cudaError_t err = launch_pdl(fp4_pack_scales_kernel, dim3((unsigned)grid), dim3(256), 0, stream, plain, rows,
                                     K / fp4_block(fmt), tiles_k, out);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe4
