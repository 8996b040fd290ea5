// Rotary positions: pairs (a, b) of a head become (a c - b s, b c + a s) with c, s
// the cosine and sine of position * frequency, times an amplitude; alone, or with
// the rotated keys and the values quantised into the paged cache in the same pass.
//
// Angles. A frequency is kept as a fraction of a turn a position, in 64-bit fixed
// point, rounded: position * fraction modulo 2^64 is the fraction of a turn that is
// left, with an error of at most |position| 2^-65 turns, whatever the position. Its two
// highest bits (rounded) are the quarter, the next 48 the angle within it, at most an
// eighth of a turn from its middle, whose sine and cosine are good to fp32's last bits.
// Negative positions turn back.
//
// Bound by memory: every value is read and written once. The sines of a CTA's tokens
// are made once, in shared memory, and used by all of its heads. 8192 tokens with 40
// heads of 128 take 27.5 us, 90% of the copy bandwidth, one token 1.7.
#include "checks.h"
#include "common.cuh"
#include "kernels.h"
#include "kvput.cuh"
#include "types.cuh"

namespace moe4 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;  // of a head: at most 256 columns

// Division of small numbers: x * d < 2^32 for every x that is divided.
struct Divisor {
  uint32_t d, m;
  Divisor() = default;
  explicit Divisor(uint32_t by) : d(by), m(by > 1 ? (uint32_t)((((uint64_t)1 << 32) - 1) / by + 1) : 0) {}
  __device__ __forceinline__ int div(int x) const { return m ? (int)__umulhi((uint32_t)x, m) : x; }
};

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
  float2 amplitude;  // its nearest float and the rest
  int T, D, rot, tokens, head_blocks, heads_each;  // a CTA's tokens and heads
  Divisor by_pairs, by_items, by_heads;  // pairs of a head; threads that share one; heads_each
};

// Cosine and sine of position * frequency, times the amplitude (in two parts). Root mean square errors, of the larger of the
// two and of the smaller: 1.94e-8 and 1.15e-8 at amplitude 1 (a correct rounding's 1.72e-8 and 1.13e-8), 2.67e-8 and 1.00e-8 of
// YaRN's for a factor of 32 (2.49e-8 and 0.98e-8). Of 50.6 million keys in FP8, 64 got another code than real
// arithmetic's, with correctly rounded ones 62: what is left is the products' rounding.
__device__ __forceinline__ float2 sine_of(unsigned long long turns, int position, float2 amplitude) {
  const unsigned long long p = turns * (unsigned long long)(long long)position;  // of 2^-64 turns
  const uint32_t f = (uint32_t)(p >> 32);
  const uint32_t quarter = (f + 0x20000000u) >> 30;
  const int rest = (int)(f - (quarter << 30));  // at most 2^29: 24 bits of it, and the 24 below them as a small angle
  const float x = (float)(rest & ~63) * 0x1p-31f;  // half turns
  const float dx = (float)((uint32_t)(p >> 14) & 0xffffffu) * (3.1415927f * 0x1p-49f);  // radians
  const float z = x * x, dz = fmaf(x, x, -z);
  // Taylor's series of sin(pi x) and of cos(pi x) - 1: the first terms left out are 2e-9 and 5e-10; pi in two parts
  float s = fmaf(z, 8.2145887e-2f, -5.9926453e-1f), c = fmaf(z, -2.5806891e-2f, 2.3533063e-1f);
  s = fmaf(z, s, 2.5501640f);
  s = fmaf(z, s, -5.1677128f);
  c = fmaf(z, c, -1.3352628f);
  c = fmaf(z, c, 4.0587121f);
  c = fmaf(z, c, -4.9348022f);
  const float sh = x * 3.1415927f;
  c = fmaf(z, c, dz * c);
  const float sl = fmaf(x, fmaf(z, s, -8.7422777e-8f), fmaf(x, 3.1415927f, -sh)) + fmaf(c, dx, dx);
  c = fmaf(-sh, dx, c);
  const float cosine = amplitude.x + fmaf(amplitude.x, c, amplitude.y);
  const float sine = fmaf(amplitude.x, sh, fmaf(amplitude.x, sl, amplitude.y * sh));
  const float cc = (quarter & 1) ? -sine : cosine, ss = (quarter & 1) ? cosine : sine;
  return (quarter & 2) ? make_float2(-cc, -ss) : make_float2(cc, ss);
}

// Cosines and sines of the CTA's tokens: [tokens][pairs rounded up to 8], in the order in which lanes with 8 pairs or 4 each
// read neighbouring 16 bytes, without bank conflicts: two pairs of each 8, then the next two.
__host__ __device__ __forceinline__ int sine_places(int rot) { return (rot + 15) / 16 * 8; }
__device__ __forceinline__ int sine_at(int p, int rot) {
  return ((p >> 1) & 3) * (sine_places(rot) / 4) + (p >> 3) * 2 + (p & 1);
}
// Pairs 2 m and 2 m + 1 of the 8 pairs number i.
__device__ __forceinline__ float4 two_sines(const float2 *cs, int i, int m, int rot) {
  return *reinterpret_cast<const float4 *>(cs + m * (sine_places(rot) / 4) + 2 * i);
}
__device__ __forceinline__ void make_sines(float2 *sines, const RopeArgs &a, int t0, int tokens) {
  const int pairs = a.rot / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += blockDim.x) {
    const int t = a.by_pairs.div(i), p = i - t * pairs;
    if (t0 + t < a.T) sines[t * sine_places(a.rot) + sine_at(p, a.rot)] = sine_of(a.turns[p], a.positions[t0 + t], a.amplitude);
  }
}

// The rotated pair (a, b), w the cosine and sine: written out, so that every path rounds alike.
__device__ __forceinline__ float rotated_a(float a, float b, float2 w) { return fmaf(a, w.x, -__fmul_rn(b, w.y)); }
__device__ __forceinline__ float rotated_b(float a, float b, float2 w) { return fmaf(b, w.x, __fmul_rn(a, w.y)); }

// 8 pairs, number i: a, b are their first and second halves.
__device__ __forceinline__ void rotate8(float (&a)[8], float (&b)[8], const float2 *cs, int i, int rot) {
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const float4 w = two_sines(cs, i, m, rot);
    const float x = a[2 * m], y = b[2 * m], u = a[2 * m + 1], v = b[2 * m + 1];
    a[2 * m] = rotated_a(x, y, make_float2(w.x, w.y));
    b[2 * m] = rotated_b(x, y, make_float2(w.x, w.y));
    a[2 * m + 1] = rotated_a(u, v, make_float2(w.z, w.w));
    b[2 * m + 1] = rotated_b(u, v, make_float2(w.z, w.w));
  }
}
// 8 values that hold 4 pairs side by side, half `part` of the 8 pairs number i.
__device__ __forceinline__ void rotate4(float (&v)[8], const float2 *cs, int i, int part, int rot) {
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const float4 w = two_sines(cs, i, 2 * part + m, rot);
    const float x = v[4 * m], y = v[4 * m + 1], z = v[4 * m + 2], u = v[4 * m + 3];
    v[4 * m] = rotated_a(x, y, make_float2(w.x, w.y));
    v[4 * m + 1] = rotated_b(x, y, make_float2(w.x, w.y));
    v[4 * m + 2] = rotated_a(z, u, make_float2(w.z, w.w));
    v[4 * m + 3] = rotated_b(z, u, make_float2(w.z, w.w));
  }
}

// Columns [p, p + 8) of a row that lies on the 16-byte grid, from the two pieces around them; those outside [0, D) are not
// read. Their values are moved by words, and 16-bit ones by half a word.
template <int TYPE>
__device__ __forceinline__ Raw8 load_window(const void *x, int64_t row, int p, int D) {
  constexpr int W = TYPE == MOE_FP32 ? 8 : 4;  // words of 8 values
  const int m = p & 7, c = p - m;
  Raw8 lo = {}, hi = {};
  if (c >= 0) lo = load_raw8(x, row + c, TYPE);
  if (m && c + 8 < D) hi = load_raw8(x, row + c + 8, TYPE);
  uint32_t w[16] = {lo.a.x, lo.a.y, lo.a.z, lo.a.w, lo.b.x, lo.b.y, lo.b.z, lo.b.w};
  const uint32_t v[8] = {hi.a.x, hi.a.y, hi.a.z, hi.a.w, hi.b.x, hi.b.y, hi.b.z, hi.b.w};
#pragma unroll
  for (int i = 0; i < W; ++i) w[W + i] = v[i];
#pragma unroll
  for (int s = W / 2; s >= 1; s /= 2) {
    const bool move = (TYPE == MOE_FP32 ? m : m >> 1) & s;
#pragma unroll
    for (int i = 0; i + s < 2 * W; ++i) w[i] = move ? w[i + s] : w[i];
  }
  if (TYPE != MOE_FP32) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16 * (m & 1));
  }
  Raw8 r;
  r.a = make_uint4(w[0], w[1], w[2], w[3]);
  r.b = TYPE == MOE_FP32 ? make_uint4(w[4], w[5], w[6], w[7]) : make_uint4(0, 0, 0, 0);
  return r;
}

// The other 8 values of a lane's pairs where they are half a rotation away. PIECES: rot is a multiple of 16, here and below;
// known to the compiler, because the registers that the other case needs cost this one a third of its rate.
template <int TYPE, bool PIECES>
__device__ __forceinline__ Raw8 load_partners(const void *x, int64_t row, int c0, int rot, int D) {
  const int half = rot / 2;
  if (PIECES) return load_raw8(x, row + (c0 >= rot ? c0 : c0 < half ? c0 + half : c0 - half), TYPE);
  if (c0 >= rot) return Raw8{};
  const Raw8 r = load_window<TYPE>(x, row, c0 < half ? c0 + half : c0 - half, D);
  if (c0 >= half || c0 + 8 <= half) return r;
  // the first halves end within these columns: the others' partners are the first of the row
  float u[8], v[8];
  raw8_to_f32(r, TYPE, u);
  raw8_to_f32(load_window<TYPE>(x, row, c0 - half, D), TYPE, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = c0 + i < half ? u[i] : v[i];
  return f32_to_raw8(u, TYPE);  // exact
}

// A lane's 8 columns of a head, rotated.
template <int TYPE, bool HALF, bool PIECES>
__device__ __forceinline__ void rotate_columns(float (&x)[8], const Raw8 &partners, int c0, int rot, const float2 *cs) {
  if (c0 >= rot) return;
  if (!HALF) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = x[i];
    rotate4(v, cs, c0 / 16, (c0 >> 3) & 1, rot);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = PIECES || c0 + i < rot ? v[i] : x[i];
    return;
  }
  const int half = rot / 2;
  float y[8];
  raw8_to_f32(partners, TYPE, y);
  if (PIECES) {
    // rotated_a(x, y) or rotated_b(y, x), which differ in a sign
    const uint32_t sign = c0 < half ? 0x80000000u : 0u;
    auto signed_sine = [&](float s) { return __uint_as_float(__float_as_uint(s) ^ sign); };
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float4 w = two_sines(cs, (c0 < half ? c0 : c0 - half) / 8, m, rot);
      x[2 * m] = fmaf(x[2 * m], w.x, __fmul_rn(y[2 * m], signed_sine(w.y)));
      x[2 * m + 1] = fmaf(x[2 * m + 1], w.z, __fmul_rn(y[2 * m + 1], signed_sine(w.w)));
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = c0 + i;
    const float2 w = cs[sine_at(c >= rot ? 0 : c < half ? c : c - half, rot)];
    const float sine = __uint_as_float(__float_as_uint(w.y) ^ (c < half ? 0x80000000u : 0u));
    const float turned = fmaf(x[i], w.x, __fmul_rn(y[i], sine));  // as above, without a branch
    x[i] = c < rot ? turned : x[i];
  }
}

// A thread's share of a head. kPieces: 16 columns, 8 pairs or 16 columns that are not rotated, where the pairs fall on
// 16-byte pieces (rot a multiple of 16). kColumns: 8 columns, and in halves the other ones of their pairs moved into place;
// a power of two of lanes of one warp have a head. kPairs, for heads off the 16-byte grid: a pair, or one column that is
// not rotated. 8192 tokens with 40 heads of 128, rot 96 by pieces: 27.7 us; rot 100 by columns 34 interleaved and 78 in
// halves (62 M instructions: moving costs more than reading; value by value 92), by pairs 107 and 117.
enum { kPairs = 0, kPieces = 1, kColumns = 2 };

template <int TYPE, bool HALF, int MODE>
struct Item {
  Raw8 a, b;
  float x, y;
  __device__ __forceinline__ void load(const RopeTensor &s, int64_t t, int h, int i, int D, int rot) {
    const int64_t in = t * s.its + h * s.ith;
    if (MODE == kPieces) {
      const bool turned = i < rot / 16;
      const int c0 = turned && HALF ? 8 * i : 16 * i, c1 = turned && HALF ? rot / 2 + 8 * i : c0 + 8;
      a = load_raw8(s.in, in + c0, TYPE);
      b = load_raw8(s.in, in + c1, TYPE);
    } else if (MODE == kColumns) {
      if (8 * i < D) {
        a = load_raw8(s.in, in + 8 * i, TYPE);
        if (HALF && 8 * i < rot) b = load_partners<TYPE, false>(s.in, in, 8 * i, rot, D);
      }
    } else if (i < rot / 2) {
      x = load_as_f32(s.in, in + (HALF ? i : 2 * i), TYPE);
      y = load_as_f32(s.in, in + (HALF ? i + rot / 2 : 2 * i + 1), TYPE);
    } else {
      x = load_as_f32(s.in, in + i + rot / 2, TYPE);
    }
  }
  __device__ __forceinline__ void store(const RopeTensor &s, int64_t t, int h, int i, int D, int rot, const float2 *cs) {
    const int64_t out = t * s.ots + h * s.oth;
    if (MODE == kPieces) {
      const bool turned = i < rot / 16;
      const int c0 = turned && HALF ? 8 * i : 16 * i, c1 = turned && HALF ? rot / 2 + 8 * i : c0 + 8;
      if (turned) {
        float u[8], v[8];
        raw8_to_f32(a, TYPE, u);
        raw8_to_f32(b, TYPE, v);
        if (HALF) {
          rotate8(u, v, cs, i, rot);
        } else {
          rotate4(u, cs, i, 0, rot);
          rotate4(v, cs, i, 1, rot);
        }
        a = f32_to_raw8(u, TYPE);
        b = f32_to_raw8(v, TYPE);
      }
      store_raw8(s.out, out + c0, TYPE, a);
      store_raw8(s.out, out + c1, TYPE, b);
    } else if (MODE == kColumns) {
      if (8 * i < D) {
        float u[8];
        raw8_to_f32(a, TYPE, u);
        rotate_columns<TYPE, HALF, false>(u, b, 8 * i, rot, cs);
        store_raw8(s.out, out + 8 * i, TYPE, f32_to_raw8(u, TYPE));
      }
    } else if (i < rot / 2) {
      const float2 w = cs[sine_at(i, rot)];
      store_from_f32(s.out, out + (HALF ? i : 2 * i), TYPE, rotated_a(x, y, w));
      store_from_f32(s.out, out + (HALF ? i + rot / 2 : 2 * i + 1), TYPE, rotated_b(x, y, w));
    } else {
      store_from_f32(s.out, out + i + rot / 2, TYPE, x);
    }
  }
};

// The heads [h0, h1) of tokens [t0, t0 + a.tokens), those of x[1] behind those of x[0]. A thread keeps its place in a head
// and walks the heads, two at a time; the first ones are asked for before the sines are made.
template <int TYPE, bool HALF, int MODE>
__device__ __forceinline__ void rotate_block(const RopeArgs &a, float2 *sines, int t0, int h0, int h1) {
  // moved partners need the second head's registers: 78 us with one at a time, 92 with two
  constexpr int U = MODE == kColumns && HALF ? 1 : 2;
  const int items = a.by_items.d, heads = h1 - h0;
  const int first = a.by_items.div(threadIdx.x), i = threadIdx.x - first * items, step = a.by_items.div(kThreads);
  const int tokens = min(a.tokens, a.T - t0);
  const bool whole = heads == a.heads_each;  // the last heads may be fewer
  const int rows = (int)threadIdx.x < step * items ? tokens * heads : 0;
  Item<TYPE, HALF, MODE> it[U];
  bool made = false;
  for (int r0 = first; r0 < rows || !made; r0 += U * step) {
    int t[U], h[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * step;
      t[u] = whole ? a.by_heads.div(r) : r / heads;
      h[u] = h0 + r - t[u] * heads;
      if (r < rows) {
        const bool second = h[u] >= a.x[0].heads;
        it[u].load(a.x[second], t0 + t[u], second ? h[u] - a.x[0].heads : h[u], i, a.D, a.rot);
      }
    }
    if (!made) {
      make_sines(sines, a, t0, tokens);
      __syncthreads();
      made = true;
    }
    if (MODE == kColumns) {
      // the lanes of a head have read each other's columns before any is written where it was
      const unsigned lanes = items == 32 ? 0xffffffffu : ((1u << items) - 1) << (threadIdx.x & 31 & ~(items - 1));
      __syncwarp(lanes);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (r0 + u * step < rows) {
        const bool second = h[u] >= a.x[0].heads;
        it[u].store(a.x[second], t0 + t[u], second ? h[u] - a.x[0].heads : h[u], i, a.D, a.rot, sines + t[u] * sine_places(a.rot));
      }
  }
}

constexpr int kMaxTokens = 16;

template <int TYPE, bool HALF, int MODE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
  __shared__ __align__(16) float2 sines[kMaxTokens * kMaxPairs];
  pdl_wait();
  pdl_trigger();
  const int block = a.head_blocks == 1 ? blockIdx.x : blockIdx.x / a.head_blocks;
  const int t0 = block * a.tokens, h0 = (blockIdx.x - block * a.head_blocks) * a.heads_each;
  rotate_block<TYPE, HALF, MODE>(a, sines, t0, h0, min(h0 + a.heads_each, a.x[0].heads + a.x[1].heads));
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
  int kv_heads, log_n, page, pages, rows_each;
  uint32_t kv_ctas;
};

// First the CTAs that write a row (token, kv head) of keys and values for each 1 << log_n lanes, then those that rotate
// queries (dealing them out in turn made no difference). Bound by instructions next to memory: 12345 tokens, 32 heads on 8
// of 128, into FP8 take 49 us, 84% of the copy bandwidth; the queries alone
// take 32 (93%), the cache write without a rotation 16. Into NVFP4 60, the floor 39.5: the write alone is 29, a division a value.
template <int FMT, int TYPE, bool HALF, int MODE>
__global__ void __launch_bounds__(kThreads) rope_write_kernel(const WriteArgs a) {
  __shared__ __align__(16) float2 sines[kMaxTokens * kMaxPairs];
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= a.kv_ctas) {
    const int at = blockIdx.x - a.kv_ctas, block = a.q.head_blocks == 1 ? at : at / a.q.head_blocks;
    const int t0 = block * a.q.tokens, h0 = (at - block * a.q.head_blocks) * a.q.heads_each;
    rotate_block<TYPE, HALF, MODE>(a.q, sines, t0, h0, min(h0 + a.q.heads_each, a.q.x[0].heads));
    return;
  }
  // a lane 8 columns of a.rows_each rows, the next one's asked for while one is quantised
  const int n = 1 << a.log_n, j = threadIdx.x & (n - 1), D = a.q.D;
  const uint32_t per = kThreads >> a.log_n, first = blockIdx.x * (per * a.rows_each);
  const int t0 = first / a.kv_heads, t1 = (min(first + per * a.rows_each, a.rows) - 1) / a.kv_heads;
  uint32_t r = first + (threadIdx.x >> a.log_n);
  int t = r / (uint32_t)a.kv_heads, head = r - t * a.kv_heads;
  const int t_step = per / (uint32_t)a.kv_heads, head_step = per - t_step * a.kv_heads;
  Raw8 k, partners, v;
  int slot;
  auto load = [&]() {
    if (r >= a.rows) t = t0, head = 0;  // reads what is there, and writes nothing
    slot = a.slots[t];
    const int64_t krow = (int64_t)t * a.kst + (int64_t)head * a.ksh;
    k = load_raw8(a.k, krow + 8 * j, TYPE);
    if (HALF) partners = load_partners<TYPE, MODE == kPieces>(a.k, krow, 8 * j, a.q.rot, a.q.D);
    v = load_raw8(a.v, (int64_t)t * a.vst + (int64_t)head * a.vsh + 8 * j, TYPE);
  };
  load();
  make_sines(sines, a.q, t0, t1 - t0 + 1);
  __syncthreads();
  const uint32_t page16 = (uint32_t)a.page >> 4;
  for (int x = 0; x < a.rows_each; ++x) {
    const bool live = r < a.rows;
    if (slot >= a.pages * a.page) {
      if (live && j == 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
      slot = -1;
    }
    const bool held = live && slot >= 0;
    const int token = slot & 15;
    uint8_t *rec = nullptr;
    if (held) {
      const uint32_t block = (uint32_t)slot >> 4, page = block / page16;
      rec = a.data + (((int64_t)page * a.kv_heads + head) * page16 + (block - page * page16)) * kv_record(FMT, D);
    }
    float f[8];
    raw8_to_f32(k, TYPE, f);
    rotate_columns<TYPE, HALF, MODE == kPieces>(f, partners, 8 * j, a.q.rot, sines + (t - t0) * sine_places(a.q.rot));
    const Raw8 own = v;
    if (x + 1 < a.rows_each) {
      r += per;
      t += t_step;
      head += head_step;
      if (head >= a.kv_heads) head -= a.kv_heads, ++t;
      load();
    }
    put8<FMT, MOE_FP32>(rec, token, 0, j, n, D, f32_to_raw8(f, MOE_FP32), held);
    put8<FMT, TYPE>(rec, token, 1, j, n, D, own, held);
  }
}

float2 split(double v) {
  const float hi = (float)v;
  return make_float2(hi, (float)(v - hi));
}

// How many tokens and heads a CTA takes: about four items a thread, all heads of its tokens where there are tokens
// enough for two CTAs an SM, else heads apart.
void share(RopeArgs &a, int heads, int mode) {
  int items = mode == kPieces ? a.D / 16 : a.D - a.rot / 2;
  if (mode == kColumns)
    for (items = 1; 8 * items < a.D;) items *= 2;
  a.tokens = 1;
  while (a.tokens < kMaxTokens && 2 * a.tokens * heads * items <= 4 * kThreads && a.T / (2 * a.tokens) >= 304) a.tokens *= 2;
  a.head_blocks = 1;
  while (a.head_blocks < heads && (heads / a.head_blocks) * items > kThreads && (int64_t)a.T * a.head_blocks < 304) ++a.head_blocks;
  a.heads_each = (heads + a.head_blocks - 1) / a.head_blocks;
  a.head_blocks = (heads + a.heads_each - 1) / a.heads_each;
  a.by_pairs = Divisor(a.rot / 2);
  a.by_items = Divisor(items);
  a.by_heads = Divisor(a.heads_each);
}

}  // namespace

moe_status_t launch_rope(const moe_rope_t &r, const int32_t *positions, int T, int D, const void *q, int64_t qst, int64_t qsh,
                         int q_heads, void *qo, int64_t qost, int64_t qosh, const void *k, int64_t kst, int64_t ksh,
                         int k_heads, void *ko, int64_t kost, int64_t kosh, int type, cudaStream_t stream, int *launches) {
  RopeArgs a = {{{q, qo, qst, qsh, qost, qosh, q_heads}, {k, ko, kst, ksh, kost, kosh, k_heads}},
                reinterpret_cast<const unsigned long long *>(r.turns), positions, split(r.amplitude), T, D, r.rot_dim, 1, 1, 1};
  bool grid = D % 8 == 0;  // heads begin and end on 16 bytes
  for (const RopeTensor &x : a.x)
    if (x.heads) grid &= strides8(x.its, x.ith) && strides8(x.ots, x.oth) && aligned16(x.in) && aligned16(x.out);
  const int mode = !grid ? kPairs : a.rot % 16 == 0 && D % 16 == 0 ? kPieces : kColumns;
  share(a, q_heads + k_heads, mode);
  using Kernel = void (*)(RopeArgs);
#define MOE4_M(T, H) {rope_kernel<T, H, kPairs>, rope_kernel<T, H, kPieces>, rope_kernel<T, H, kColumns>}
#define MOE4_R(T) {MOE4_M(T, true), MOE4_M(T, false)}
  static const Kernel kernels[3][2][3] = {MOE4_R(MOE_BF16), MOE4_R(MOE_FP16), MOE4_R(MOE_FP32)};
#undef MOE4_R
#undef MOE4_M
  const int64_t ctas = ((int64_t)T + a.tokens - 1) / a.tokens * a.head_blocks;
  if (ctas >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  const cudaError_t err = launch_pdl(kernels[type][r.layout == MOE_ROPE_INTERLEAVED][mode],
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
         split(r.amplitude), T, c.head_dim, r.rot_dim, 1, 1, 1};
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
  const int mode = a.q.rot % 16 == 0 ? kPieces : kColumns;
  share(a.q, q ? q_heads : 1, mode);
  if (q) q_ctas = ((int64_t)T + a.q.tokens - 1) / a.q.tokens * a.q.head_blocks;
  // one row a lane until there are CTAs enough for every SM four times over, then four, as far as the sines of their
  // tokens fit
  const uint32_t per = kThreads >> a.log_n;
  static_assert(kThreads / 8 * 32 <= kMaxTokens * kMaxPairs, "sines of one row a lane: 32, 16 or 8 tokens of 32, 64 or 128 pairs");
  a.rows_each = 1;
  if (a.rows > 4 * per * 608 && ((4 * per - 1) / c.kv_heads + 2) * sine_places(r.rot_dim) <= kMaxTokens * kMaxPairs) a.rows_each = 4;
  const uint32_t step = per * a.rows_each;
  a.kv_ctas = a.rows / step + (a.rows % step != 0);
  const int64_t ctas = q_ctas + a.kv_ctas;
  if (ctas >= (int64_t)1 << 31) return MOE_ERR_UNSUPPORTED;
  using Kernel = void (*)(WriteArgs);
#define MOE4_M(F, T, H) {rope_write_kernel<F, T, H, kPieces>, rope_write_kernel<F, T, H, kColumns>}
#define MOE4_W(F, T) {MOE4_M(F, T, true), MOE4_M(F, T, false)}
#define MOE4_W_TYPES(F) {MOE4_W(F, MOE_BF16), MOE4_W(F, MOE_FP16), MOE4_W(F, MOE_FP32)}
  static const Kernel kernels[4][3][2][2] = {MOE4_W_TYPES(MOE_KV_BF16), MOE4_W_TYPES(MOE_KV_FP16), MOE4_W_TYPES(MOE_KV_FP8),
                                             MOE4_W_TYPES(MOE_KV_NVFP4)};
#undef MOE4_W_TYPES
#undef MOE4_W
#undef MOE4_M
  const cudaError_t err = launch_pdl(kernels[c.fmt][type][r.layout == MOE_ROPE_INTERLEAVED][mode == kColumns],
                                     dim3((unsigned)ctas), dim3(kThreads), 0, stream, a);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe4
