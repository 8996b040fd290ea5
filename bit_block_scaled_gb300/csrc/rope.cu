// Rotary positions: pairs (a, b) of a head become (a c - b s, b c + a s) with c, s
// the cosine and sine of position * frequency, times an amplitude; alone, or with
// the rotated keys and the values quantised into the paged cache in the same pass.
//
// Angles. A frequency is kept as a fraction of a turn a position, in 64-bit fixed
// point: position * fraction modulo 2^64 is the fraction of a turn that is left, with
// an error below |position| 2^-65 turns, whatever the position. Its two highest bits
// (rounded) are the quarter, the next 30 the angle within it, at most an eighth of a
// turn from its middle, whose sine and cosine are good to fp32's last bits. Negative
// positions turn back.
//
// Bound by memory: every value is read and written once. The sines of a CTA's tokens
// are made once, in shared memory, and used by all of its heads.
#include "checks.h"
#include "common.cuh"
#include "kernels.h"
#include "kvput.cuh"
#include "types.cuh"

namespace moe4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // of a head: at most 256 columns

// Tensors whose heads are rotated, [T][heads][D].
struct RopeTensor {
  const void *in;
  void *out;
  int64_t its, ith, ots, oth;
  int heads;
};

struct RopeArgs {
  RopeTensor x[2];
  const unsigned long long *turns;
  const int32_t *positions;
  float amplitude;
  int T, D, rot, tokens, head_blocks, heads_each;  // a CTA's tokens and heads
};

__device__ __forceinline__ float2 sine_of(unsigned long long turns, int position, float amplitude) {
  const uint32_t f = (uint32_t)((turns * (unsigned long long)(long long)position) >> 32);  // of 2^-32 turns
  const uint32_t quarter = (f + 0x20000000u) >> 30;
  const int rest = (int)(f - (quarter << 30));  // -2^29 .. 2^29
  float s, c;
  sincospif((float)rest * 0x1p-31f, &s, &c);  // half turns
  const float cc = (quarter & 1) ? -s : c, ss = (quarter & 1) ? c : s;
  return (quarter & 2) ? make_float2(-cc * amplitude, -ss * amplitude) : make_float2(cc * amplitude, ss * amplitude);
}

// Cosines and sines of the CTA's tokens: [tokens][pairs].
__device__ __forceinline__ void make_sines(float2 *sines, const RopeArgs &a, int t0, int tokens) {
  const int pairs = a.rot / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += blockDim.x) {
    const int t = i / pairs, p = i - t * pairs;
    if (t0 + t < a.T) sines[i] = sine_of(a.turns[p], a.positions[t0 + t], a.amplitude);
  }
}

// The rotated pair (a, b), w the cosine and sine: written out, so that every path rounds alike.
__device__ __forceinline__ float rotated_a(float a, float b, float2 w) { return fmaf(a, w.x, -__fmul_rn(b, w.y)); }
__device__ __forceinline__ float rotated_b(float a, float b, float2 w) { return fmaf(b, w.x, __fmul_rn(a, w.y)); }

// 8 pairs: a, b are their first and second halves.
__device__ __forceinline__ void rotate8(float (&a)[8], float (&b)[8], const float2 *cs) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 w = cs[i];
    const float x = a[i], y = b[i];
    a[i] = rotated_a(x, y, w);
    b[i] = rotated_b(x, y, w);
  }
}
// 8 values that hold 4 pairs side by side.
__device__ __forceinline__ void rotate4(float (&v)[8], const float2 *cs) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 w = cs[i];
    const float x = v[2 * i], y = v[2 * i + 1];
    v[2 * i] = rotated_a(x, y, w);
    v[2 * i + 1] = rotated_b(x, y, w);
  }
}

// Where the pairs fall on 16-byte pieces (rot a multiple of 16): a thread takes 16 columns of a head, 8 pairs or 16
// that are not rotated.
template <int TYPE, bool HALF>
__device__ __forceinline__ void rotate_piece(const RopeTensor &x, const float2 *cs, int64_t t, int h, int i, int rot) {
  const int c0 = i < rot / 16 ? (HALF ? 8 * i : 16 * i) : 16 * i, c1 = i < rot / 16 && HALF ? rot / 2 + 8 * i : c0 + 8;
  const int64_t in = t * x.its + h * x.ith, out = t * x.ots + h * x.oth;
  Raw8 ra = load_raw8(x.in, in + c0, TYPE), rb = load_raw8(x.in, in + c1, TYPE);
  if (i < rot / 16) {
    float a[8], b[8];
    raw8_to_f32(ra, TYPE, a);
    raw8_to_f32(rb, TYPE, b);
    if (HALF) {
      rotate8(a, b, cs + 8 * i);
    } else {
      rotate4(a, cs + 8 * i);
      rotate4(b, cs + 8 * i + 4);
    }
    ra = f32_to_raw8(a, TYPE);
    rb = f32_to_raw8(b, TYPE);
  }
  store_raw8(x.out, out + c0, TYPE, ra);
  store_raw8(x.out, out + c1, TYPE, rb);
}

// Any rot: a thread takes a pair, or one column that is not rotated.
template <int TYPE, bool HALF>
__device__ __forceinline__ void rotate_pair(const RopeTensor &x, const float2 *cs, int64_t t, int h, int i, int rot) {
  const int64_t in = t * x.its + h * x.ith, out = t * x.ots + h * x.oth;
  if (i >= rot / 2) {
    const int c = i + rot / 2;
    store_from_f32(x.out, out + c, TYPE, load_as_f32(x.in, in + c, TYPE));
    return;
  }
  const int c0 = HALF ? i : 2 * i, c1 = HALF ? i + rot / 2 : 2 * i + 1;
  const float a = load_as_f32(x.in, in + c0, TYPE), b = load_as_f32(x.in, in + c1, TYPE);
  const float2 w = cs[i];
  store_from_f32(x.out, out + c0, TYPE, rotated_a(a, b, w));
  store_from_f32(x.out, out + c1, TYPE, rotated_b(a, b, w));
}

// The heads [h0, h1) of tokens [t0, t0 + a.tokens), those of x[1] behind those of x[0].
template <int TYPE, bool HALF, bool PIECES>
__device__ __forceinline__ void rotate_block(const RopeArgs &a, const float2 *sines, int t0, int h0, int h1) {
  const int items = PIECES ? a.D / 16 : a.D - a.rot / 2, heads = h1 - h0;
  const int per_token = items * heads, n = min(a.tokens, a.T - t0) * per_token;
  for (int at = threadIdx.x; at < n; at += kThreads) {
    const int t = at / per_token, r = at - t * per_token, hh = r / items, i = r - hh * items, h = h0 + hh;
    const bool second = h >= a.x[0].heads;
    const RopeTensor &x = a.x[second];
    const float2 *cs = sines + t * (a.rot / 2);
    if (PIECES)
      rotate_piece<TYPE, HALF>(x, cs, t0 + t, second ? h - a.x[0].heads : h, i, a.rot);
    else
      rotate_pair<TYPE, HALF>(x, cs, t0 + t, second ? h - a.x[0].heads : h, i, a.rot);
  }
}

constexpr int kMaxTokens = 16;

template <int TYPE, bool HALF, bool PIECES>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  __shared__ float2 sines[kMaxTokens * kMaxPairs];
  pdl_wait();
  pdl_trigger();
  const int t0 = blockIdx.x / a.head_blocks * a.tokens, h0 = blockIdx.x % a.head_blocks * a.heads_each;
  make_sines(sines, a, t0, a.tokens);
  __syncthreads();
  rotate_block<TYPE, HALF, PIECES>(a, sines, t0, h0, min(h0 + a.heads_each, a.x[0].heads + a.x[1].heads));
}

// ------------------------------------------------------- with the cache write
struct WriteArgs {
  RopeArgs q;
  uint8_t *data;
  const void *k, *v;
  const int32_t *slots;
  unsigned int *status;
  int64_t kst, ksh, vst, vsh;
  uint32_t rows;  // T * kv heads
  int kv_heads, log_n, page, pages, q_ctas;
};

// A lane's 8 columns of a key, rotated.
template <int TYPE, bool HALF>
__device__ __forceinline__ void rotate_key(float (&x)[8], const void *k, int64_t row, int j, int rot, const float2 *cs) {
  const int c0 = 8 * j;
  if (c0 >= rot) return;
  if (!HALF) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c0 + 2 * i < rot) {
        const float2 w = cs[c0 / 2 + i];
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = rotated_a(a, b, w);
        x[2 * i + 1] = rotated_b(a, b, w);
      }
    return;
  }
  const int half = rot / 2;
  float y[8];  // the other ones of the pairs
  if (rot % 16 == 0) {
    raw8_to_f32(load_raw8(k, row + (c0 < half ? c0 + half : c0 - half), TYPE), TYPE, y);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + i;
      y[i] = c < rot ? load_as_f32(k, row + (c < half ? c + half : c - half), TYPE) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = c0 + i;
    if (c < rot) {
      const float2 w = cs[c < half ? c : c - half];
      x[i] = c < half ? rotated_a(x[i], y[i], w) : rotated_b(y[i], x[i], w);
    }
  }
}

// R rows (token, kv head) a lane; 1 << log_n lanes a row.
constexpr int kRows = 2;
static_assert(kThreads / 8 * kRows * 32 <= kMaxTokens * kMaxPairs, "sines of the keys' rows");

template <int FMT, int TYPE, bool HALF, bool PIECES>
__global__ void __launch_bounds__(kThreads) rope_write_kernel(const WriteArgs a) {
  __shared__ float2 sines[kMaxTokens * kMaxPairs];  // the keys' rows: 64, 32 or 16 tokens of 32, 64 or 128 pairs at most
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < a.q_ctas) {
    const int t0 = blockIdx.x / a.q.head_blocks * a.q.tokens, h0 = blockIdx.x % a.q.head_blocks * a.q.heads_each;
    make_sines(sines, a.q, t0, a.q.tokens);
    __syncthreads();
    rotate_block<TYPE, HALF, PIECES>(a.q, sines, t0, h0, min(h0 + a.q.heads_each, a.q.x[0].heads));
    return;
  }
  const int n = 1 << a.log_n, j = threadIdx.x & (n - 1), D = a.q.D;
  const uint32_t per = kThreads >> a.log_n, first = (blockIdx.x - a.q_ctas) * (per * kRows);
  const uint32_t last = min(first + per * kRows, a.rows) - 1;
  const int t0 = first / a.kv_heads;
  // tokens of these rows: at most their number
  make_sines(sines, a.q, t0, (int)(last / a.kv_heads) - t0 + 1);
  __syncthreads();
#pragma unroll
  for (int x = 0; x < kRows; ++x) {
    const uint32_t r = first + x * per + (threadIdx.x >> a.log_n);
    const bool live = r < a.rows;
    const int t = live ? r / (uint32_t)a.kv_heads : t0, head = live ? r - t * a.kv_heads : 0;
    int slot = a.slots[t];
    if (slot >= a.pages * a.page) {
      if (live && j == 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
      slot = -1;
    }
    const int64_t krow = (int64_t)t * a.kst + (int64_t)head * a.ksh;
    const Raw8 k = load_raw8(a.k, krow + 8 * j, TYPE);
    const Raw8 v = load_raw8(a.v, (int64_t)t * a.vst + (int64_t)head * a.vsh + 8 * j, TYPE);
    const bool held = live && slot >= 0;
    uint8_t *rec = nullptr;
    if (held) {
      const uint32_t block = (uint32_t)slot >> 4, page16 = (uint32_t)a.page >> 4, page = block / page16;
      rec = a.data + (((int64_t)page * a.kv_heads + head) * page16 + (block - page * page16)) * kv_record(FMT, D);
    }
    float f[8];
    raw8_to_f32(k, TYPE, f);
    rotate_key<TYPE, HALF>(f, a.k, krow, j, a.q.rot, sines + (t - t0) * (a.q.rot / 2));
    put8<FMT, MOE_FP32>(rec, slot & 15, 0, j, n, D, f32_to_raw8(f, MOE_FP32), held);
    put8<FMT, TYPE>(rec, slot & 15, 1, j, n, D, v, held);
  }
}

// How many tokens and heads a CTA takes: about four pieces a thread, all heads of its tokens where there are tokens
// enough for two CTAs an SM, else heads apart.
void share(RopeArgs &a, int heads, bool pieces) {
  const int items = pieces ? a.D / 16 : a.D - a.rot / 2, want = 4 * kThreads;
  a.tokens = 1;
  while (a.tokens < kMaxTokens && 2 * a.tokens * heads * items <= want && a.T / (2 * a.tokens) >= 304) a.tokens *= 2;
  a.head_blocks = 1;
  while (a.head_blocks < heads && a.tokens * (heads / a.head_blocks) * items > kThreads && (int64_t)a.T * a.head_blocks < 304)
    ++a.head_blocks;
  a.heads_each = (heads + a.head_blocks - 1) / a.head_blocks;
  a.head_blocks = (heads + a.heads_each - 1) / a.heads_each;
}

}  // namespace

moe_status_t launch_rope(const moe_rope_t &r, const int32_t *positions, int T, int D, const void *q, int64_t qst, int64_t qsh,
                         int q_heads, void *qo, int64_t qost, int64_t qosh, const void *k, int64_t kst, int64_t ksh,
                         int k_heads, void *ko, int64_t kost, int64_t kosh, int type, cudaStream_t stream, int *launches) {
  RopeArgs a = {{{q, qo, qst, qsh, qost, qosh, q_heads}, {k, ko, kst, ksh, kost, kosh, k_heads}},
                reinterpret_cast<const unsigned long long *>(r.turns), positions, r.amplitude, T, D, r.rot_dim, 1, 1, 1};
  // pairs on 16-byte pieces, or one by one
  bool pieces = a.rot % 16 == 0 && D % 16 == 0;
  for (const RopeTensor &x : a.x)
    if (x.heads)
      pieces &= strides8(x.its, x.ith) && strides8(x.ots, x.oth) && aligned16(x.in) && aligned16(x.out);
  share(a, q_heads + k_heads, pieces);
  using Kernel = void (*)(RopeArgs);
#define MOE4_R(T) {{rope_kernel<T, true, false>, rope_kernel<T, true, true>}, {rope_kernel<T, false, false>, rope_kernel<T, false, true>}}
  static const Kernel kernels[3][2][2] = {MOE4_R(MOE_BF16), MOE4_R(MOE_FP16), MOE4_R(MOE_FP32)};
#undef MOE4_R
  const int64_t ctas = (int64_t)((T + a.tokens - 1) / a.tokens) * a.head_blocks;
  if (ctas >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  const cudaError_t err = launch_pdl(kernels[type][r.layout == MOE_ROPE_INTERLEAVED][pieces],
                                     dim3((unsigned)ctas), dim3(kThreads), 0, stream, a);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status_t launch_rope_kv_write(const moe_rope_t &r, const int32_t *positions, int T, const void *q, int64_t qst,
                                  int64_t qsh, int q_heads, void *qo, int64_t qost, int64_t qosh, const void *k, int64_t kst,
                                  int64_t ksh, const void *v, int64_t vst, int64_t vsh, int type, const int32_t *slots,
                                  const moe_kv_cache_t &c, unsigned int *status, cudaStream_t stream, int *launches) {
  if ((int64_t)T * c.kv_heads >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  WriteArgs a = {};
  a.q = {{{q, qo, qst, qsh, qost, qosh, q ? q_heads : 0}, {}}, reinterpret_cast<const unsigned long long *>(r.turns), positions,
         r.amplitude, T, c.head_dim, r.rot_dim, 1, 1, 1};
  a.data = static_cast<uint8_t *>(c.data);
  a.k = k;
  a.v = v;
  a.slots = slots;
  a.status = status;
  a.kst = kst, a.ksh = ksh, a.vst = vst, a.vsh = vsh;
  a.rows = (uint32_t)((int64_t)T * c.kv_heads);
  a.kv_heads = c.kv_heads;
  a.log_n = c.head_dim == 64 ? 3 : c.head_dim == 128 ? 4 : 5;
  a.page = c.page_size;
  a.pages = c.num_pages;
  int64_t q_ctas = 0;
  if (q) {
    share(a.q, q_heads, a.q.rot % 16 == 0);
    q_ctas = (int64_t)((T + a.q.tokens - 1) / a.q.tokens) * a.q.head_blocks;
  }
  const uint32_t step = (kThreads >> a.log_n) * kRows;
  const int64_t ctas = q_ctas + a.rows / step + (a.rows % step != 0);
  if (ctas >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  a.q_ctas = (int)q_ctas;
  using Kernel = void (*)(WriteArgs);
#define MOE4_W(F, T) {{rope_write_kernel<F, T, true, false>, rope_write_kernel<F, T, true, true>}, {rope_write_kernel<F, T, false, false>, rope_write_kernel<F, T, false, true>}}
#define MOE4_W_TYPES(F) {MOE4_W(F, MOE_BF16), MOE4_W(F, MOE_FP16), MOE4_W(F, MOE_FP32)}
  static const Kernel kernels[4][3][2][2] = {MOE4_W_TYPES(MOE_KV_BF16), MOE4_W_TYPES(MOE_KV_FP16), MOE4_W_TYPES(MOE_KV_FP8),
                                             MOE4_W_TYPES(MOE_KV_NVFP4)};
#undef MOE4_W_TYPES
#undef MOE4_W
  const cudaError_t err = launch_pdl(kernels[c.fmt][type][r.layout == MOE_ROPE_INTERLEAVED][a.q.rot % 16 == 0],
                                     dim3((unsigned)ctas), dim3(kThreads), 0, stream, a);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe4
