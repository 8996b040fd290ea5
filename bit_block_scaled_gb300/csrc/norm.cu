// The seam between two blocks: u = alpha * gate * post(z), h = residual + u,
// y = pre(h), each row in one pass.
//
// A row is read once and held in registers, NV chunks of 8 columns a thread;
// both norms sum it there, so z, residual and gate are read once and h and y
// written once, which is all the memory traffic there is, and what bounds it.
// RMS needs one sum over the row; LAYER takes the mean first and then the
// squares of the differences, which loses nothing when the mean is large.
//
// 8192 x 2880, bf16, RMS before and after with a gate a row: 33.5 us, 83% of the
// copy bandwidth. What counted were instructions: 33 an element with a CTA a row
// that looks up the weights' type (96 us, 44 at the best split), 9 needed. In fp32
// with a gate of every element and layer norms, 8192 x 2880: 90 us, 77%.
#include "common.cuh"
#include "device.cuh"
#include "kernels.h"
#include "types.cuh"

namespace moe4 {

namespace {

// Sum over the CTA; every thread gets it. buf: used in turn, so that one
// barrier a sum is enough.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float (*buf)[32], int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  constexpr int kWarps = THREADS / 32;
  float *b = buf[turn];
  turn ^= 1;
  const int lane = threadIdx.x & 31;
  if (lane == 0) b[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < kWarps ? b[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < kWarps) v += __shfl_xor_sync(0xffffffffu, v, o);
  return kWarps > 16 ? v : __shfl_sync(0xffffffffu, v, 0);  // the lanes past the warps hold none of it
}

struct NormArgs {
  const void *z, *res, *gate;
  void *h, *y;
  int64_t zs, rs, gst, gsh, hs, ys;
  int T, H;
  int shift;  // every row tensor's stride modulo 8, or -1
  float alpha;
  moe_norm_t post, pre;
  int has_post, has_pre;
};

// Column of a thread's value i of chunk j: VEC, eight neighbours (whole and
// aligned chunks); else a warp's lanes next to each other, value by value.
template <int THREADS, bool VEC>
__device__ __forceinline__ int column(int j, int i) {
  return VEC ? (threadIdx.x + j * THREADS) * 8 + i : threadIdx.x + (j * 8 + i) * THREADS;
}

// A thread's chunk j of a row, or of a norm's parameter; 0 past the row.
template <int THREADS, bool VEC>
__device__ __forceinline__ Raw8 take8(const void *p, int64_t at, int j, int H, int type) {
  if (VEC) return load_raw8(p, at + column<THREADS, VEC>(j, 0), type);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = column<THREADS, VEC>(j, i);
    v[i] = c < H ? load_as_f32(p, at + c, type) : 0.f;
  }
  return f32_to_raw8(v, type);
}

template <int THREADS, bool VEC>
__device__ __forceinline__ void store8(void *p, int64_t at, int j, int H, int type, const float (&v)[8]) {
  if (VEC) {
    store_raw8(p, at + column<THREADS, VEC>(j, 0), type, f32_to_raw8(v, type));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<THREADS, VEC>(j, i);
      if (c < H) store_from_f32(p, at + c, type, v[i]);
    }
  }
}

// x becomes (x - mean) * weight; returned is the factor 1 / sqrt(. + eps) that
// it has to be multiplied by, for the caller to fold in. With a bias the factor
// is put in here and 1 returned. weight(j, v) and bias(j, v) give the
// parameters of chunk j; columns that do not exist (exists(j, i)) hold 0.
template <int NV, int THREADS, typename E, typename W, typename B>
__device__ __forceinline__ float normalise(float (&x)[NV][8], const moe_norm_t &n, int H, float (*buf)[32], int &turn,
                                           E exists, W weight, B bias) {
  const float inv_h = 1.0f / (float)H;
  if (n.kind == MOE_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[j][i];
    const float mean = block_sum<THREADS>(s, buf, turn) * inv_h;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (exists(j, i)) x[j][i] -= mean;
  }
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) q += x[j][i] * x[j][i];
  // the weights go in while the sum (of the values before them) is on its way
#pragma unroll
  for (int j = 0; j < NV; ++j) weight(j, x[j]);
  const float r = rsqrtf(block_sum<THREADS>(q, buf, turn) * inv_h + n.eps);
  if (!n.bias) return r;
#pragma unroll
  for (int j = 0; j < NV; ++j) bias(j, r, x[j]);
  return 1.f;
}

// Few rows, long or unaligned ones: a CTA a row, as many threads as there are
// chunks.
template <int TA, int TR, int NV, int THREADS, bool VEC>
__global__ void __launch_bounds__(THREADS) norm_row_kernel(const NormArgs a) {
  __shared__ float buf[2][32];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const bool each_gate = a.gate && a.gsh != 0;
  auto live = [&](int j) { return column<THREADS, VEC>(j, 0) < a.H; };  // some of the chunk exists
  float x[NV][8], f = a.alpha;  // f: factor of all of the row
  if (a.gate && !each_gate) f *= load_as_f32(a.gate, row * a.gst, TA);
  Raw8 res[NV], gate[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[j][i] = 0.f;
    if (!live(j)) continue;
    if (a.z) raw8_to_f32(take8<THREADS, VEC>(a.z, row * a.zs, j, a.H, TA), TA, x[j]);
    if (a.res) res[j] = take8<THREADS, VEC>(a.res, row * a.rs, j, a.H, TR);
    if (each_gate) gate[j] = take8<THREADS, VEC>(a.gate, row * a.gst, j, a.H, TA);
  }
  auto norm = [&](const moe_norm_t &n) {
    return normalise<NV, THREADS>(
        x, n, a.H, buf, turn, [&](int j, int i) { return column<THREADS, VEC>(j, VEC ? 0 : i) < a.H; },
        [&](int j, float(&v)[8]) {
          if (!n.weight || !live(j)) return;
          float w[8];
          raw8_to_f32(take8<THREADS, VEC>(n.weight, 0, j, a.H, n.type), n.type, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= w[i] + n.offset;
        },
        [&](int j, float r, float(&v)[8]) {
          if (!live(j)) return;
          float b[8];
          raw8_to_f32(take8<THREADS, VEC>(n.bias, 0, j, a.H, n.type), n.type, b);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = v[i] * r + b[i];
        });
  };
  if (a.has_post) f *= norm(a.post);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!live(j)) continue;
    if (each_gate) {
      float gt[8];
      raw8_to_f32(gate[j], TA, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] *= gt[i];
    }
    float rv[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rv[i] = 0.f;
    if (a.res) raw8_to_f32(res[j], TR, rv);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[j][i] = a.z ? rv[i] + f * x[j][i] : rv[i];
    if (a.h) store8<THREADS, VEC>(a.h, row * a.hs, j, a.H, TR, x[j]);
  }
  if (!a.has_pre) return;
  const float r = norm(a.pre);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!live(j)) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[j][i] *= r;
    store8<THREADS, VEC>(a.y, row * a.ys, j, a.H, TA, x[j]);
  }
}

// Many rows: a CTA walks over them, holds the norms' weights in registers, and
// has its next row's loads under way while it works on the present one. Chunks
// past the row are zeros that are neither loaded nor stored.
// kRest: a gate of every element and norms with a bias, which cost registers.
// kShifted: rows that start off the 16-byte grid, where every
// row tensor's stride is the same modulo 8 (a width of 2881 in contiguous
// tensors). Chunks then lie on the grid of the memory, the row starting
// row * stride mod 8 elements into its first; the step over rows is a multiple
// of 8, so that a CTA meets one such shift only and its weights still stay in
// registers. A row's first and last chunk are stored value by value.
// 8192 x 2881, bf16: 104 us with every value by itself, 43 shifted, 33 for 2880.
enum { kPlain = 0, kRest = 1, kShifted = 2 };

template <int TA, int MODE>
constexpr int walkers(int threads) {  // CTAs an SM, by the registers that a thread needs (56, or up to 85)
  return (TA == MOE_FP32 || (MODE & kRest) ? 768 : 1152) / threads > 0
             ? (TA == MOE_FP32 || (MODE & kRest) ? 768 : 1152) / threads
             : 1;
}

// Values lo to hi of the chunk at element `at`, 0 in the others.
__device__ __forceinline__ Raw8 load_part(const void *p, int64_t at, int lo, int hi, int type) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i >= lo && i < hi ? load_as_f32(p, at + i, type) : 0.f;
  return f32_to_raw8(v, type);
}

template <int TA, int TR, int NV, int THREADS, int MODE>
__global__ void __launch_bounds__(THREADS, NV == 1 ? walkers<TA, MODE>(THREADS) : 1) norm_walk_kernel(const NormArgs a) {
  constexpr bool REST = MODE & kRest, SHIFTED = MODE & kShifted;
  const bool each = REST && a.gate && a.gsh != 0;
  __shared__ float buf[2][32];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  if (SHIFTED && blockIdx.x >= a.T) return;
  const int shift = SHIFTED ? (int)(blockIdx.x * (int64_t)a.shift & 7) : 0;
  const int c0 = threadIdx.x * 8 - shift;
  const bool one_gate = SHIFTED && each && a.gst == 0 && a.shift != 0;  // one row for all, not shifted with them
  bool live[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) live[j] = c0 + j * THREADS * 8 < a.H;
  // the part of chunk j that is in the row
  auto lo = [&](int j) { return c0 + j * THREADS * 8 < 0 ? shift : 0; };
  auto hi = [&](int j) { return min(8, a.H - (c0 + j * THREADS * 8)); };
  auto whole = [&](int j) { return !SHIFTED || (lo(j) == 0 && hi(j) == 8); };
  auto exists = [&](int j, int i) { return SHIFTED ? i >= lo(j) && i < hi(j) : live[j]; };
  // A chunk that is not whole is loaded whole all the same, so that nothing waits
  // for it here (74 -> 50 us); what lies next to the row in it, whoever may be
  // writing that, is masked after. Only where it would pass the tensor's end it
  // goes value by value.
  auto take = [&](const void *p, int64_t row, int64_t stride, int j, int type) {
    const int c = c0 + j * THREADS * 8;
    const bool inside = whole(j) || (a.T - 1 - row) * stride + a.H >= c + 8;
    return inside ? load_raw8(p, row * stride + c, type) : load_part(p, row * stride + c, lo(j), hi(j), type);
  };
  // chunk j of a parameter, which lies on the grid itself: the two chunks there that it is in, moved by the shift
  auto parameter = [&](const void *p, int j, int type, float(&v)[8]) {
    const int c = c0 + shift + j * THREADS * 8;
    if (!SHIFTED) {
      raw8_to_f32(load_raw8(p, c, type), type, v);
      return;
    }
    float t[16];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int from = c - 8 + 8 * k;
      if (from >= 0 && from + 8 <= a.H) {
        raw8_to_f32(load_raw8(p, from, type), type, v);
      } else {
        raw8_to_f32(load_part(p, from, from < 0 ? 8 : 0, a.H - from, type), type, v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) t[8 * k + i] = v[i];
    }
#pragma unroll
    for (int b = 4; b > 0; b >>= 1)
#pragma unroll
      for (int i = 15; i >= b; --i) t[i] = shift & b ? t[i - b] : t[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = t[8 + i];
  };
  auto mask = [&](int j, float(&v)[8]) {
    if (whole(j)) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!exists(j, i)) v[i] = 0.f;
  };
  auto store = [&](void *p, int64_t at, int j, int type, const float(&v)[8]) {
    const int64_t to = at + j * THREADS * 8;
    if (whole(j)) {
      store_raw8(p, to, type, f32_to_raw8(v, type));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (exists(j, i)) store_from_f32(p, to + i, type, v[i]);
    }
  };
  float wpost[NV][8], wpre[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    auto keep = [&](const moe_norm_t &n, bool has, float(&w)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = live[j] ? 1.f : 0.f;
      if (!has || !n.weight || !live[j]) return;
      parameter(n.weight, j, n.type, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] += n.offset;
    };
    keep(a.post, a.has_post, wpost[j]);
    keep(a.pre, a.has_pre, wpre[j]);
  }
  Raw8 z[NV], res[NV], gate[NV];
  const Raw8 zero = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  uint32_t gate_bits = 0;
  auto fetch = [&](int64_t row) {
    if (!each && a.gate)
      gate_bits = TA == MOE_FP32 ? static_cast<const uint32_t *>(a.gate)[row * a.gst]
                                 : static_cast<const uint16_t *>(a.gate)[row * a.gst];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      z[j] = a.z && live[j] ? take(a.z, row, a.zs, j, TA) : zero;
      res[j] = a.res && live[j] ? take(a.res, row, a.rs, j, TR) : zero;
      if (REST && each && !one_gate) gate[j] = live[j] ? take(a.gate, row, a.gst, j, TA) : zero;
    }
  };
  if (one_gate) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[8];
      gate[j] = zero;
      if (!live[j]) continue;
      parameter(a.gate, j, TA, v);
      gate[j] = f32_to_raw8(v, TA);
    }
  }
  fetch(blockIdx.x);
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    float x[NV][8], f = a.alpha;
    if (!each && a.gate) f *= load_as_f32(&gate_bits, 0, TA);
    Raw8 rs[NV], gt[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      raw8_to_f32(z[j], TA, x[j]);
      mask(j, x[j]);
      rs[j] = res[j];
      if (REST) gt[j] = gate[j];
    }
    if (row + gridDim.x < a.T) fetch(row + gridDim.x);
    auto norm = [&](const moe_norm_t &n, const float(&w)[NV][8]) {
      return normalise<NV, THREADS>(
          x, n, a.H, buf, turn, exists,
          [&](int j, float(&v)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= w[j][i];
          },
          [&](int j, float r, float(&v)[8]) {
            if (!REST || !live[j]) return;
            float b[8];
            parameter(n.bias, j, n.type, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * r + b[i];
          });
    };
    if (a.has_post) f *= norm(a.post, wpost);
    const int64_t hr = row * a.hs + c0, yr = row * a.ys + c0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[8];
      if (REST && each) {
        raw8_to_f32(gt[j], TA, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] *= v[i];
      }
      raw8_to_f32(rs[j], TR, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = v[i] + f * x[j][i];
      mask(j, x[j]);
      if (a.h && live[j]) store(a.h, hr, j, TR, x[j]);
    }
    if (!a.has_pre) continue;
    const float r = norm(a.pre, wpre);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] *= r;
      if (live[j]) store(a.y, yr, j, TA, x[j]);
    }
  }
}

template <int TA, int TR, int NV, int THREADS, bool VEC>
cudaError_t rows(const NormArgs &a, cudaStream_t stream) {
  return launch_pdl(norm_row_kernel<TA, TR, NV, THREADS, VEC>, dim3(a.T), dim3(THREADS), 0, stream, a);
}

template <int TA, int TR, int NV, int THREADS, int MODE>
cudaError_t walk(const NormArgs &a, int sms, cudaStream_t stream) {
  const int most = sms * (NV > 1 ? 1 : walkers<TA, MODE>(THREADS));
  // a multiple of 8 for kShifted, where CTAs past the last row end at once
  const int grid = a.T < most ? (MODE & kShifted ? (a.T + 7) & ~7 : a.T) : (MODE & kShifted ? most & ~7 : most);
  return launch_pdl(norm_walk_kernel<TA, TR, NV, THREADS, MODE>, dim3(grid), dim3(THREADS), 0, stream, a);
}

template <int TA, int TR, int MODE>
cudaError_t walk(const NormArgs &a, int chunks, int sms, cudaStream_t stream) {
  return chunks <= 128   ? walk<TA, TR, 1, 128, MODE>(a, sms, stream)
         : chunks <= 256 ? walk<TA, TR, 1, 256, MODE>(a, sms, stream)
         : chunks <= 384 ? walk<TA, TR, 1, 384, MODE>(a, sms, stream)
         : chunks <= 512 ? walk<TA, TR, 1, 512, MODE>(a, sms, stream)
                         : walk<TA, TR, 2, 512, MODE>(a, sms, stream);
}

// vec: whole chunks on the 16-byte grid; a.shift < 0: no common shift
template <int TA, int TR>
cudaError_t go(const NormArgs &a, bool vec, cudaStream_t stream) {
  const int sms = sm_count();
  const int chunks = (a.H + 7) / 8, shifted = (a.H + 7 + 7) / 8;
  const bool rest = (a.gate && a.gsh != 0) || (a.has_post && a.post.bias) || (a.has_pre && a.pre.bias);
  // from two rows an SM on walking pays (H 2880, bf16; a CTA a row / walking, us): 304 rows 4.2 / 4.1, 608 6.8 / 5.5,
  // 1216 9.6 / 7.5, 2432 19.9 / 13.0
  if (a.T > 2 * sms && vec && chunks <= 1024)
    return rest ? walk<TA, TR, kRest>(a, chunks, sms, stream) : walk<TA, TR, kPlain>(a, chunks, sms, stream);
  // off the grid from three on (H 2881, value by value / shifted): 330 rows 6.8 / 6.9, 608 8.9 / 8.1, 1216 15.7 / 10.6;
  // (H 1003) 330 4.8 / 5.5, 608 6.0 / 5.5
  if (a.T > 3 * sms && !vec && a.shift >= 0 && shifted <= 1024)
    return rest ? walk<TA, TR, kShifted | kRest>(a, shifted, sms, stream)
                : walk<TA, TR, kShifted>(a, shifted, sms, stream);
  if (!vec)
    return chunks <= 256    ? rows<TA, TR, 1, 256, false>(a, stream)
           : chunks <= 512  ? rows<TA, TR, 1, 512, false>(a, stream)
           : chunks <= 1024 ? rows<TA, TR, 2, 512, false>(a, stream)
                            : rows<TA, TR, 4, 512, false>(a, stream);
  return chunks <= 128    ? rows<TA, TR, 1, 128, true>(a, stream)
         : chunks <= 256  ? rows<TA, TR, 1, 256, true>(a, stream)
         : chunks <= 512  ? rows<TA, TR, 1, 512, true>(a, stream)
         : chunks <= 1024 ? rows<TA, TR, 2, 512, true>(a, stream)
                          : rows<TA, TR, 4, 512, true>(a, stream);
}

}  // namespace

moe_status_t launch_residual_norm(const void *z, int64_t zs, const void *res, int64_t rs, const void *gate,
                                  int64_t gst, int64_t gsh, int T, int H, int type, int res_type,
                                  const moe_norm_t *post, float alpha, void *h, int64_t hs, const moe_norm_t *pre,
                                  void *y, int64_t ys, cudaStream_t stream, int *launches) {
  if (T == 0) return MOE_OK;
  NormArgs a = {};
  a.z = z;
  a.res = res;
  a.gate = gate;
  a.h = h;
  a.y = y;
  a.zs = zs;
  a.rs = rs;
  a.gst = gst;
  a.gsh = gsh;
  a.hs = hs;
  a.ys = ys;
  a.T = T;
  a.H = H;
  a.alpha = alpha;
  if (post) a.post = *post;
  if (pre) a.pre = *pre;
  a.has_post = post != nullptr;
  a.has_pre = pre != nullptr;
  auto whole = [](const void *p, int64_t s) { return !p || s % 8 == 0; };
  const bool vec = H % 8 == 0 && whole(z, zs) && whole(res, rs) && whole(h, hs) && whole(y, ys) &&
                   whole(gsh ? gate : nullptr, gst);
  const struct {
    const void *p;
    int64_t stride;
  } rows_of[4] = {{z, zs}, {res, rs}, {h, hs}, {y, ys}};
  a.shift = (int)((h ? hs : ys) & 7);
  for (const auto &t : rows_of)
    if (t.p && (t.stride & 7) != a.shift) {
      a.shift = -1;
      break;
    }
  if (gate && gsh && gst != 0 && (gst & 7) != a.shift) a.shift = -1;
  cudaError_t err;
  if (type == MOE_BF16)
    err = res_type == MOE_FP32 ? go<MOE_BF16, MOE_FP32>(a, vec, stream) : go<MOE_BF16, MOE_BF16>(a, vec, stream);
  else if (type == MOE_FP16)
    err = res_type == MOE_FP32 ? go<MOE_FP16, MOE_FP32>(a, vec, stream) : go<MOE_FP16, MOE_FP16>(a, vec, stream);
  else
    err = go<MOE_FP32, MOE_FP32>(a, vec, stream);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe4
