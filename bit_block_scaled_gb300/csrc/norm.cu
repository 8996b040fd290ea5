// The seam between two blocks: u = alpha * gate * post(z), h = residual + u,
// y = pre(h), each row in one pass.
//
// A row is read once and held in registers as fp32, NV chunks of 8 columns a
// thread; both norms sum it there, so z, residual and gate are read once and
// h and y written once, which is all the memory traffic there is. RMS needs
// one sum over the row; LAYER takes the mean first and then the squares of
// the differences, which loses nothing when the mean is large.
#include "common.cuh"
#include "kernels.h"
#include "types.cuh"

namespace moe4 {

namespace {

constexpr int kMaxThreads = 512;

// Sum over the CTA; every thread gets it. buf: 2 x 32 floats used in turn, so
// that one barrier a sum is enough.
__device__ __forceinline__ float block_sum(float v, float (*buf)[32], int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) return v;
  float *b = buf[turn];
  turn ^= 1;
  if (lane == 0) b[warp] = v;
  __syncthreads();
  v = lane < warps ? b[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct NormArgs {
  const void *z, *res, *gate;
  void *h, *y;
  int64_t zs, rs, gst, gsh, hs, ys;
  int T, H;
  float alpha;
  moe_norm_t post, pre;
  int has_post, has_pre, vec;
};

// 8 values from column c; with vec whole and aligned, else one by one up to H
// (0 past it).
__device__ __forceinline__ void load8(const void *p, int64_t row, int c, const NormArgs &a, int type, float (&v)[8]) {
  if (a.vec) {
    raw8_to_f32(load_raw8(p, row + c, type), type, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < a.H ? load_as_f32(p, row + c + i, type) : 0.f;
  }
}

__device__ __forceinline__ void store8(void *p, int64_t row, int c, const NormArgs &a, int type, const float (&v)[8]) {
  if (a.vec) {
    store_raw8(p, row + c, type, f32_to_raw8(v, type));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < a.H) store_from_f32(p, row + c + i, type, v[i]);
  }
}

template <int NV>
__device__ __forceinline__ void normalise(float (&x)[NV][8], const moe_norm_t &n, const NormArgs &a, float (*buf)[32],
                                          int &turn) {
  const float inv_h = 1.0f / (float)a.H;
  float mean = 0.f;
  if (n.kind == MOE_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[j][i];
    mean = block_sum(s, buf, turn) * inv_h;
  }
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (threadIdx.x + j * blockDim.x) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < a.H) {
        x[j][i] -= mean;
        q += x[j][i] * x[j][i];
      }
  }
  const float r = rsqrtf(block_sum(q, buf, turn) * inv_h + n.eps);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (threadIdx.x + j * blockDim.x) * 8;
    if (c >= a.H) continue;
    float w[8], b[8];
    if (n.weight) load8(n.weight, 0, c, a, n.type, w);
    if (n.bias) load8(n.bias, 0, c, a, n.type, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[j][i] *= r;
      if (n.weight) x[j][i] *= w[i] + n.offset;
      if (n.bias) x[j][i] += b[i];
    }
  }
}

template <int TA, int TR, int NV>
__global__ void __launch_bounds__(kMaxThreads) residual_norm_kernel(const NormArgs a) {
  __shared__ float buf[2][32];
  int turn = 0;
  pdl_wait();
  pdl_trigger();
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    float x[NV][8], res[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (threadIdx.x + j * blockDim.x) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = res[j][i] = 0.f;
      if (c < a.H) {
        if (a.z) load8(a.z, t * a.zs, c, a, TA, x[j]);
        if (a.res) load8(a.res, t * a.rs, c, a, TR, res[j]);
      }
    }
    if (a.has_post) normalise<NV>(x, a.post, a, buf, turn);
    const float row_gate = a.gate && a.gsh == 0 ? load_as_f32(a.gate, t * a.gst, TA) : 1.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (threadIdx.x + j * blockDim.x) * 8;
      if (c >= a.H) continue;
      float gt[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) gt[i] = row_gate;
      if (a.gate && a.gsh != 0) load8(a.gate, t * a.gst, c, a, TA, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = a.z ? res[j][i] + a.alpha * gt[i] * x[j][i] : res[j][i];
      if (a.h) store8(a.h, t * a.hs, c, a, TR, x[j]);
    }
    if (a.has_pre) {
      normalise<NV>(x, a.pre, a, buf, turn);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (threadIdx.x + j * blockDim.x) * 8;
        if (c < a.H) store8(a.y, t * a.ys, c, a, TA, x[j]);
      }
    }
  }
}

template <int TA, int TR>
cudaError_t go(const NormArgs &a, cudaStream_t stream) {
  const int chunks = (a.H + 7) / 8;
  const int nv = chunks <= kMaxThreads ? 1 : chunks <= 2 * kMaxThreads ? 2 : 4;
  const int threads = ((chunks + nv - 1) / nv + 31) / 32 * 32;
  const dim3 grid(a.T), block(threads);
  if (nv == 1) return launch_pdl(residual_norm_kernel<TA, TR, 1>, grid, block, 0, stream, a);
  if (nv == 2) return launch_pdl(residual_norm_kernel<TA, TR, 2>, grid, block, 0, stream, a);
  return launch_pdl(residual_norm_kernel<TA, TR, 4>, grid, block, 0, stream, a);
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
  a.vec = H % 8 == 0 && whole(z, zs) && whole(res, rs) && whole(h, hs) && whole(y, ys) &&
          whole(gsh ? gate : nullptr, gst);
  cudaError_t err;
  if (type == MOE_BF16)
    err = res_type == MOE_FP32 ? go<MOE_BF16, MOE_FP32>(a, stream) : go<MOE_BF16, MOE_BF16>(a, stream);
  else if (type == MOE_FP16)
    err = res_type == MOE_FP32 ? go<MOE_FP16, MOE_FP32>(a, stream) : go<MOE_FP16, MOE_FP16>(a, stream);
  else
    err = go<MOE_FP32, MOE_FP32>(a, stream);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe4
