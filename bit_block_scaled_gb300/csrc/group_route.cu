// Routing with expert groups: scores s = softmax(l) or sigmoid(l), selection
// scores c = s + bias (or the logits, which order the experts alike), the best
// groups, the k best experts in them, weights from s alone.
//
// One warp a token. Group g owns L = 32 / (n_group rounded up to a power of
// two) lanes, which share its experts (E <= 256 leaves at most 16 a lane), so
// what a group needs is log2(L) shuffles. An expert's key is the upper 24
// ordered bits of c with the expert's index below them; each lane sorts its
// keys, and five merges of sorted lists of 4 or 8 leave the whole warp with the
// k best in order. 16-bit logits ordered by themselves fit the 24 bits, so
// their many ties are decided by the index in the key.
//
// Which experts are chosen is decided on the real numbers. Keys and fp32 scores
// carry errors (key_error2, score_error2). Where every gap that the selection
// rests on is wider than them, the keys are right. Otherwise the candidates'
// scores are computed as pairs of floats (pair_score, off by 1e-9 at most), one
// a lane, and where even those are close, in 64 bits: a 64-bit exponential
// takes a warp 3 us, a pair 0.2. What is left -- groups too close for pairs, a
// softmax over infinities, more than 32 candidates -- goes through select_exact,
// 16 us for a row, with its loops rolled up because its instructions come from
// memory each time. 8192 random rows of 256 experts in 8 groups with a bias:
// some 200 with close choices and one in two calls with close groups; 16.5 us for
// sigmoids, 21 for softmax (37 with its sum in 64 bits).
#include <type_traits>

#include "common.cuh"
#include "device.cuh"
#include "kernels.h"
#include "types.cuh"

namespace moe4 {

namespace {

constexpr int kWarps = 4;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kMaxFloat = 3.402823466e38f;

struct RouteArgs {
  const void *logits;
  const float *bias;
  int32_t *ids;
  float *weights;
  int64_t ld;
  int type, T, k, n_group, topk_group, gs, lanes;  // gs: experts a group; lanes: lanes a group
  int score, top2, renorm;
  float scale;
};

// One warp's working space for open rows.
struct Scratch {
  int id[32];
  double c[32];
  float order[256];  // what orders the experts, in fp32
};

// An unsigned key that orders as the float does (-0 made +0 before); 0 is free
// for "no candidate", below the key of -inf.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ float not_nan(float v) { return v == v ? v : -INFINITY; }

// Bound on twice the error of an fp32 selection score of size |v|. Sigmoid: E =
// exp(-l) is off by 2^-22 + |l| 2^-23 of itself, which 1 / (1 + E) turns into
// at most s (1 - s) of that (<= 0.6e-7 + 0.27e-7), sum, quotient and the bias
// add at most 2^-22 of s and 2^-24 of the result: below 5e-7 + 6e-8 |v|.
// Softmax: the exponential likewise (s |l - m| < 0.37), its sum of up to 256
// terms at most 21 * 2^-24 + 2^-22 of itself (16 in a lane, five shuffles):
// below 2e-6 + 6e-8 |v|.
__device__ __forceinline__ float score_error2(int score, float v) {
  return (score == MOE_SCORE_SOFTMAX ? 4e-6f : 1e-6f) + 1.3e-7f * fabsf(v);
}
// Bound on the error of a group's score of fp32 value v, whose best are x and y
// (y only where it takes two), for comparing v - error with another's v + error:
// the scores' errors are of their own size, which their sum may have lost, and
// the sum and the difference round by 2^-24 of it each. Infinities are exact.
__device__ __forceinline__ float group_error(int score, bool two, float x, float y, float v) {
  auto half = [&](float s) { return fabsf(s) <= kMaxFloat ? 0.5f * score_error2(score, s) : 0.f; };
  return half(x) + (two ? half(y) : 0.f) + (fabsf(v) <= kMaxFloat ? 1.3e-7f * fabsf(v) : 0.f);
}
// Twice the error of a score cut to the 24 bits of a key (2^-15 of it).
__device__ __forceinline__ float key_error2(int score, float v) { return score_error2(score, v) + 3.1e-5f * fabsf(v); }

__device__ __forceinline__ float warp_max(float v) { return value_of(__reduce_max_sync(kAll, key_of(v))); }
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// exp(l - m) with the limits at infinite m: logits equal to m count 1, others 0.
__device__ __forceinline__ float exp_rel(float l, float m) {
  if (fabsf(m) > kMaxFloat) return l == m ? 1.f : 0.f;
  return expf(l - m);
}
__device__ __forceinline__ double exp_rel64(float l, float m) {
  if (fabsf(m) > kMaxFloat) return l == m ? 1.0 : 0.0;
  return exp((double)l - (double)m);
}

// Batcher's odd-even merge sort of a lane's keys, largest first.
template <int PL>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[PL]) {
#pragma unroll
  for (int p = 1; p < PL; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < PL; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < PL && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t hi = max(key[i + j], key[i + j + k]), lo = min(key[i + j], key[i + j + k]);
            key[i + j] = hi;
            key[i + j + k] = lo;
          }
}

// Merges each lane's KL sorted keys with those of the lane o away, both keeping
// the KL best in order: the larger of key i and the other's key KL - 1 - i are
// the best, in a bitonic order that log2(KL) exchanges sort.
template <int KL>
__device__ __forceinline__ void merge_keys(uint32_t (&key)[KL], int o) {
  uint32_t other[KL];
#pragma unroll
  for (int i = 0; i < KL; ++i) other[i] = __shfl_xor_sync(kAll, key[KL - 1 - i], o);
#pragma unroll
  for (int i = 0; i < KL; ++i) key[i] = max(key[i], other[i]);
#pragma unroll
  for (int d = KL / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < KL; ++i)
      if ((i & d) == 0) {
        const uint32_t hi = max(key[i], key[i + d]), lo = min(key[i], key[i + d]);
        key[i] = hi;
        key[i + d] = lo;
      }
}

// This lane's logits (NaN as -inf, -inf where there is no expert), all loads
// under way together.
template <int PL>
__device__ __forceinline__ void load_logits(const RouteArgs &a, int64_t at, const int (&id)[PL], unsigned valid,
                                            float (&l)[PL]) {
  auto each = [&](auto get) {
#pragma unroll
    for (int i = 0; i < PL; ++i) l[i] = (valid >> i) & 1u ? get(id[i]) : -INFINITY;
  };
  if (a.type == MOE_FP32) {
    const float *p = static_cast<const float *>(a.logits) + at;
    each([&](int i) { return p[i]; });
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(a.logits) + at;
    if (a.type == MOE_BF16)
      each([&](int i) { return load_as_f32(p, i, MOE_BF16); });
    else
      each([&](int i) { return load_as_f32(p, i, MOE_FP16); });
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) l[i] = not_nan(l[i]);
}

// What orders expert e, in 64 bits.
__device__ double order64(const RouteArgs &a, int64_t at, float m, double sum, int e, bool scored) {
  const float l = not_nan(load_as_f32(a.logits, at + e, a.type));
  if (!scored) return l;
  double s = a.score == MOE_SCORE_SOFTMAX ? exp_rel64(l, m) / sum : 1.0 / (1.0 + exp(-(double)l));
  if (a.bias) s += (double)a.bias[e];
  return s == s ? s : -INFINITY;
}

// A number as a float and the part of it below that float's precision.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = a + b, v = s - a;
  return {s, (a - (s - v)) + (b - v)};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair s = two_sum(a.hi, b.hi);
  s.lo += a.lo + b.lo;
  return two_sum(s.hi, s.lo);
}
__device__ __forceinline__ Pair square(Pair a) {
  const float h = a.hi * a.hi;
  return two_sum(h, fmaf(a.hi, a.hi, -h) + 2.f * a.hi * a.lo);
}
__device__ __forceinline__ float difference(Pair a, Pair b) { return (a.hi - b.hi) + (a.lo - b.lo); }

__device__ __forceinline__ Pair quotient(Pair n, Pair d) {
  const float q = n.hi / d.hi;
  return {q, (fmaf(-d.hi, q, n.hi) + (n.lo - d.lo * q)) / d.hi};  // a Newton step with the remainder
}

// exp(x), x.hi in -80..80, as 2^n exp(r / 64)^64 with r within ln 2 / 2: the
// part of the series beyond 1 + r / 64 is below 1.5e-5 there, so its fp32 error
// is 1e-12, which six squarings make 6e-11 of the exponential.
__device__ __noinline__ Pair pair_exp(Pair x) {
  const float n = rintf(x.hi * 1.44269504f);
  // r = x - n ln 2, a two-part reduction after Cody and Waite: ln 2 as 0.693145751953125 (16 bits, so that n times it
  // is exact) + 1.42860682030941723e-6
  Pair r = two_sum(fmaf(n, -0.693145751953125f, x.hi), n * -1.42860682030941723e-6f);
  r.hi *= 0.015625f;
  r.lo = (r.lo + x.lo) * 0.015625f;
  const float q = r.hi * r.hi * (0.5f + r.hi * (0.166666667f + r.hi * 0.0416666667f));
  Pair e = two_sum(1.f, r.hi);
  e.lo += r.lo + q;
  e = two_sum(e.hi, e.lo);
#pragma unroll
  for (int i = 0; i < 6; ++i) e = square(e);
  const float two_n = __uint_as_float((uint32_t)((int)n + 127) << 23);
  return {e.hi * two_n, e.lo * two_n};
}

// exp(l - m), m finite and at least l; beyond -80 it is below any tolerance.
__device__ __forceinline__ Pair pair_exp_rel(float l, float m) {
  Pair x = two_sum(l, -m);
  if (!(x.hi > -80.f)) x = {-80.f, 0.f};
  return pair_exp(x);
}

// The score of a logit, plus b. sum: of a softmax's exponentials.
__device__ __forceinline__ Pair pair_score(const RouteArgs &a, float l, float b, float m, Pair sum) {
  if (a.score == MOE_SCORE_SOFTMAX) return add(quotient(pair_exp_rel(l, m), sum), {b, 0.f});
  const Pair e = pair_exp({-fminf(fmaxf(l, -80.f), 80.f), 0.f});
  return add(quotient({1.f, 0.f}, add({1.f, 0.f}, e)), {b, 0.f});
}

// Sum of the softmax's exponentials over the warp, off by 7e-11 of it: their
// own error and 13 additions' (8 in a lane, five shuffles).
__device__ __noinline__ Pair pair_sum(const RouteArgs &a, int64_t at, float m) {
  Pair sum = {0.f, 0.f};
#pragma unroll 1
  for (int e = threadIdx.x & 31; e < a.n_group * a.gs; e += 32)
    sum = add(sum, pair_exp_rel(not_nan(load_as_f32(a.logits, at + e, a.type)), m));
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) sum = add(sum, {__shfl_xor_sync(kAll, sum.hi, o), __shfl_xor_sync(kAll, sum.lo, o)});
  return sum;
}

// Bound on twice the error of a pair of size |v|: a softmax score is off by 1.4e-10 at most, a sigmoid by less; what
// is added to it rounds by 2^-47 of its size.
__device__ __forceinline__ float pair_error2(float v) { return 1e-9f + 1e-12f * fabsf(v); }

// Sum of the softmax's exponentials in 64 bits, over the warp.
__device__ double sum64(const RouteArgs &a, int64_t at, float m, int experts) {
  double sum = 0.0;
#pragma unroll 1
  for (int e = threadIdx.x & 31; e < experts; e += 32) sum += exp_rel64(not_nan(load_as_f32(a.logits, at + e, a.type)), m);
  return warp_sum(sum);
}

// n <= 32 candidates, one a lane, into the order of their 64-bit scores.
__device__ __noinline__ int rank64(const RouteArgs &a, int64_t at, float m, int experts, int n, int mine, Scratch &w) {
  const int lane = threadIdx.x & 31;
  const double sum = a.bias && a.score == MOE_SCORE_SOFTMAX ? sum64(a, at, m, experts) : 1.0;
  const double v = lane < n ? order64(a, at, m, sum, mine, a.bias) : 0.0;
  int place = 0;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const double ov = __shfl_sync(kAll, v, j);
    const int oid = __shfl_sync(kAll, mine, j);
    place += ov > v || (ov == v && oid < mine);
  }
  if (lane < n) w.id[place] = mine;
  __syncwarp();
  mine = lane < a.k ? w.id[lane] : 0;
  __syncwarp();
  return mine;
}

// Of this lane's group, whose score lies in low..high: whether it is surely
// among the best, and whether it may be all the same.
__device__ __forceinline__ void place_groups(const RouteArgs &a, int g, float low, float high, bool &sure, bool &maybe) {
  int may = 0, are = 0;  // groups that may be ahead of it, and that are
#pragma unroll 1
  for (int h = 0; h < a.n_group; ++h) {
    const float ol = __shfl_sync(kAll, low, h * a.lanes), oh = __shfl_sync(kAll, high, h * a.lanes);
    may += h != g && !(oh < low);
    are += h != g && ol > high;
  }
  sure = g < a.n_group && may < a.topk_group;
  maybe = g < a.n_group && !sure && are < a.topk_group;
}

// The choice for an open row, the j-th id in lane j, from the logits on.
__device__ __noinline__ int select_exact(const RouteArgs &a, int64_t at, float m, float fsum, Scratch &w) {
  const int lane = threadIdx.x & 31, g = lane / a.lanes, sub = lane & (a.lanes - 1), e0 = g * a.gs + sub;
  const int experts = a.n_group * a.gs;
  const int mine_n = g < a.n_group && sub < a.gs ? (a.gs - sub + a.lanes - 1) / a.lanes : 0;  // experts of this lane
  const bool grouped = a.topk_group < a.n_group, scored = a.bias || (grouped && a.top2);
  const double sum = scored && a.score == MOE_SCORE_SOFTMAX ? sum64(a, at, m, experts) : 1.0;
  auto score32 = [&](int e) {
    const float l = not_nan(load_as_f32(a.logits, at + e, a.type));
    if (!scored) return l;
    float v = a.score == MOE_SCORE_SOFTMAX ? exp_rel(l, m) / fsum : 1.0f / (1.0f + expf(-l));
    if (a.bias) v += a.bias[e];
    return not_nan(v);
  };
  float b1 = -INFINITY, b2 = -INFINITY;  // the two best of the group
#pragma unroll 1
  for (int i = 0; i < mine_n; ++i) {
    const int e = e0 + i * a.lanes;
    const float v = score32(e);
    w.order[e] = v;
    b2 = fmaxf(b2, fminf(b1, v));
    b1 = fmaxf(b1, v);
  }
  bool kept = g < a.n_group;
  if (grouped) {
#pragma unroll 1
    for (int o = 1; o < a.lanes; o <<= 1) {
      const float o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
      b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
      b1 = fmaxf(b1, o1);
    }
    const float gv = g < a.n_group ? (a.top2 ? not_nan(b1 + b2) : b1) : -INFINITY;
    int ahead = 0;
#pragma unroll 1
    for (int h = 0; h < a.n_group; ++h) {
      const float ov = __shfl_sync(kAll, gv, h * a.lanes);
      ahead += ov > gv || (ov == gv && h < g);
    }
    if (!scored) {
      kept = kept && ahead < a.topk_group;
    } else {
      // those that are surely kept as fp32 has it, and those that are within the error of the other side
      const float ge = group_error(a.score, a.top2, b1, b2, gv), low = gv - ge, high = gv + ge;
      bool sure, maybe;
      place_groups(a, g, low, high, sure, maybe);
      // 64-bit scores of those of an undecided group that can be its best, or its two best
      const float edge = a.top2 ? b2 : b1, least = edge - score_error2(a.score, edge);
      double d1 = -INFINITY, d2 = -INFINITY;
      int i = 0;
#pragma unroll 1
      while (true) {  // one candidate of each lane at a time
        while (maybe && i < mine_n && w.order[e0 + i * a.lanes] < least) ++i;
        const bool need = maybe && i < mine_n;
        const unsigned who = __ballot_sync(kAll, need);
        if (!who) break;
        const int to = __popc(who & ((1u << lane) - 1u)), cnt = __popc(who);
        if (need) w.id[to] = e0 + i * a.lanes;
        ++i;
        __syncwarp();
        if (lane < cnt) w.c[lane] = order64(a, at, m, sum, w.id[lane], true);
        __syncwarp();
#pragma unroll 1
        for (int j = 0; j < cnt; ++j)
          if (w.id[j] / a.gs == g) {
            const double v = w.c[j];
            d2 = fmax(d2, fmin(d1, v));
            d1 = fmax(d1, v);
          }
        __syncwarp();
      }
      double gd = a.top2 ? d1 + d2 : d1;
      if (!(gd == gd)) gd = -INFINITY;
      int place = 0;
#pragma unroll 1
      for (int h = 0; h < a.n_group; ++h) {
        const double od = __shfl_sync(kAll, gd, h * a.lanes);
        const bool om = __shfl_sync(kAll, (int)maybe, h * a.lanes), os = __shfl_sync(kAll, (int)sure, h * a.lanes);
        place += os || (om && (od > gd || (od == gd && h < g)));
      }
      kept = sure || (maybe && place < a.topk_group);
    }
  }
  if (scored && !a.bias) {  // the logits order the experts of the kept groups
#pragma unroll 1
    for (int i = 0; i < mine_n; ++i)
      w.order[e0 + i * a.lanes] = not_nan(load_as_f32(a.logits, at + e0 + i * a.lanes, a.type));
  }
  // candidates in fp32 order, by index among equals: k, and with computed scores those within the error of the k-th
  const unsigned all = kept ? (1u << mine_n) - 1u : 0u;
  unsigned left = all;
  int mine = 0, n = 0;
  float kth = 0.f;
#pragma unroll 1
  while (n < 32) {
    float best = -INFINITY;
    int bid = 0x7fffffff;
#pragma unroll 1
    for (unsigned l = left; l; l &= l - 1) {
      const int e = e0 + (__ffs(l) - 1) * a.lanes;
      if (bid == 0x7fffffff || w.order[e] > best) {
        best = w.order[e];
        bid = e;
      }
    }
    const uint32_t key = bid != 0x7fffffff ? key_of(best) : 0u, top = __reduce_max_sync(kAll, key);
    if (top == 0u) break;
    const int id = __reduce_min_sync(kAll, key == top ? bid : 0x7fffffff);
    const float v = value_of(top);
    if (n >= a.k && (!a.bias || v < kth - score_error2(a.score, kth))) break;
    if (n < a.k) kth = v;
    if (bid == id) left &= ~(1u << ((id - e0) / a.lanes));
    if (lane == n) mine = id;
    ++n;
  }
  if (!a.bias) return mine;
  if (n < 32) return rank64(a, at, m, experts, n, mine, w);
  // more candidates than lanes: every expert in 64 bits, k times over
  left = all;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    double best = -INFINITY;
    int bid = 0x7fffffff;
#pragma unroll 1
    for (unsigned l = left; l; l &= l - 1) {
      const int e = e0 + (__ffs(l) - 1) * a.lanes;
      const double v = order64(a, at, m, sum, e, true);
      if (bid == 0x7fffffff || v > best) {
        best = v;
        bid = e;
      }
    }
    const int own = bid;
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(kAll, best, o);
      const int oid = __shfl_xor_sync(kAll, bid, o);
      if (oid != 0x7fffffff && (bid == 0x7fffffff || ov > best || (ov == best && oid < bid))) {
        best = ov;
        bid = oid;
      }
    }
    if (own == bid) left &= ~(1u << ((bid - e0) / a.lanes));
    if (lane == j) mine = bid;
  }
  return mine;
}

// PL: experts a lane, rounded up to a power of two; KL: choices held, 4 or 8;
// FULL: every lane has PL experts
template <int PL, int KL, bool FULL>
__global__ void __launch_bounds__(kWarps * 32, PL <= 8 ? 7 : 5) group_route_kernel(const RouteArgs a) {
  __shared__ Scratch scratch[kWarps];
  pdl_wait();
  pdl_trigger();
  const bool grouped = a.topk_group < a.n_group;
  const bool by_score = a.bias || (grouped && a.top2);    // some order rests on computed scores
  const bool exact_keys = !a.bias && a.type != MOE_FP32;  // 24 bits hold the logits
  const int lane = threadIdx.x & 31, g = lane / a.lanes, sub = lane & (a.lanes - 1);
  Scratch &own = scratch[threadIdx.x >> 5];
  unsigned valid = 0;
  int id[PL];
  float bias[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    id[i] = g * a.gs + sub + i * a.lanes;
    if (FULL || (g < a.n_group && sub + i * a.lanes < a.gs)) valid |= 1u << i;
    bias[i] = a.bias && ((valid >> i) & 1u) ? a.bias[id[i]] : 0.f;
  }
  if (FULL) valid = (1u << PL) - 1u;
  for (int t = blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.T; t += gridDim.x * kWarps) {
    const int64_t at = (int64_t)t * a.ld;
    float l[PL], m = 0.f, sum = 1.f;
    load_logits<PL>(a, at, id, valid, l);
    if (a.score == MOE_SCORE_SOFTMAX && (by_score || !a.renorm)) {
      m = l[0];
#pragma unroll
      for (int i = 1; i < PL; ++i) m = fmaxf(m, l[i]);
      m = warp_max(m);
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if ((valid >> i) & 1u) sum += exp_rel(l[i], m);
      sum = warp_sum(sum);
    }
    auto score = [&](float x) {
      return a.score == MOE_SCORE_SOFTMAX ? __fdividef(exp_rel(x, m), sum) : __fdividef(1.0f, 1.0f + __expf(-x));
    };
    uint32_t full[PL];  // keys of what orders the experts, whole; 0: no expert
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < PL; ++i) full[i] = (valid >> i) & 1u ? key_of(not_nan(score(l[i]) + bias[i])) : 0u;
    } else {
#pragma unroll
      for (int i = 0; i < PL; ++i) full[i] = (valid >> i) & 1u ? key_of(l[i]) : 0u;
    }
    // pairs decide close choices, but for a softmax over infinities; its sum is taken where a row needs it first
    const bool pairs = a.score == MOE_SCORE_SIGMOID || fabsf(m) <= kMaxFloat;
    Pair psum = {0.f, 0.f};
    auto need_sum = [&] {
      if (a.score == MOE_SCORE_SOFTMAX && psum.hi == 0.f) psum = pair_sum(a, at, m);
    };
    bool open = false;  // the groups are undecided, or there are too many candidates
    if (grouped) {
      uint32_t b1 = 0u, b2 = 0u;
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        b2 = max(b2, min(b1, full[i]));
        b1 = max(b1, full[i]);
      }
      for (int o = 1; o < a.lanes; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
        b2 = max(max(b2, o2), min(b1, o1));
        b1 = max(b1, o1);
      }
      uint32_t gk = 0;
      float x = 0.f, y = 0.f;  // the group's best two
      if (g < a.n_group) {
        x = value_of(b1);
        y = value_of(b2);
        if (a.top2 && !a.bias) {
          x = score(x);
          y = score(y);
        }
        gk = !a.top2 ? b1 : key_of(not_nan(x + y));
      }
      int ahead = 0;  // groups before this one; equal ones by index
      for (int h = 0; h < a.n_group; ++h) {
        const uint32_t ok = __shfl_sync(kAll, gk, h * a.lanes);
        ahead += ok > gk || (ok == gk && h < g);
      }
      bool kept = g < a.n_group && ahead < a.topk_group;
      if (by_score) {
        // the least that a kept group's score can be, and the most that a dropped one's can
        const float gv = value_of(gk), ge = g < a.n_group ? group_error(a.score, a.top2, x, y, gv) : 0.f;
        const float low = gv - ge, high = gv + ge;
        const float lv = value_of(__reduce_min_sync(kAll, kept ? key_of(low) : kAll)),
                    nv = value_of(__reduce_max_sync(kAll, kept || g >= a.n_group ? 0u : key_of(high)));
        open = !(lv > nv);
        if (open && pairs) {
          need_sum();
          // pairs for the groups within the error of the other side, of those experts that can be their best (two)
          const float edge = value_of(a.top2 ? b2 : b1);
          bool sure, maybe;
          place_groups(a, g, low, high, sure, maybe);
          const uint32_t least = !a.bias ? (a.top2 ? b2 : b1) : key_of(edge - score_error2(a.score, edge));
          Pair d1 = {-INFINITY, 0.f}, d2 = d1;
          unsigned need = 0;
#pragma unroll
          for (int i = 0; i < PL; ++i)
            if (maybe && full[i] && full[i] >= least) need |= 1u << i;
          auto put = [&](Pair v) {
            if (difference(v, d1) > 0.f || d1.hi == -INFINITY) {
              d2 = d1;
              d1 = v;
            } else if (difference(v, d2) > 0.f || d2.hi == -INFINITY) {
              d2 = v;
            }
          };
#pragma unroll 1
          for (; need; need &= need - 1) {
            const int e = g * a.gs + sub + (__ffs(need) - 1) * a.lanes;
            put(pair_score(a, not_nan(load_as_f32(a.logits, at + e, a.type)), a.bias ? a.bias[e] : 0.f, m, psum));
          }
          __syncwarp();
#pragma unroll 1
          for (int o = 1; o < a.lanes; o <<= 1) {
            const Pair o1 = {__shfl_xor_sync(kAll, d1.hi, o), __shfl_xor_sync(kAll, d1.lo, o)},
                       o2 = {__shfl_xor_sync(kAll, d2.hi, o), __shfl_xor_sync(kAll, d2.lo, o)};
            if (o1.hi != -INFINITY) put(o1);
            if (o2.hi != -INFINITY) put(o2);
          }
          const Pair gd = a.top2 ? add(d1, d2) : d1;
          const float gde = pair_error2(d1.hi) + (a.top2 ? pair_error2(d2.hi) : 0.f);  // of the scores' sizes
          bool near = false;
          int place = 0;
#pragma unroll 1
          for (int h = 0; h < a.n_group; ++h) {
            const Pair od = {__shfl_sync(kAll, gd.hi, h * a.lanes), __shfl_sync(kAll, gd.lo, h * a.lanes)};
            const bool om = __shfl_sync(kAll, (int)maybe, h * a.lanes), os = __shfl_sync(kAll, (int)sure, h * a.lanes);
            const float d = difference(od, gd), ode = __shfl_sync(kAll, gde, h * a.lanes);
            place += os || (om && d > 0.f);
            near = near || (maybe && om && h != g && !(fabsf(d) > 0.5f * (gde + ode)));
          }
          open = __any_sync(kAll, near);
          kept = sure || (maybe && place < a.topk_group);
        }
      }
      if (!kept) {
#pragma unroll
        for (int i = 0; i < PL; ++i) full[i] = 0u;
      }
    }
    uint32_t sorted[PL], best[KL];
#pragma unroll
    for (int i = 0; i < PL; ++i) sorted[i] = full[i] ? (full[i] & ~255u) | (uint32_t)(255 - id[i]) : 0u;
    sort_keys<PL>(sorted);
#pragma unroll
    for (int i = 0; i < KL; ++i) best[i] = i < PL ? sorted[i < PL ? i : 0] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) merge_keys<KL>(best, o);
    // lane j takes the j-th choice
    uint32_t key = best[0], last = best[0];
#pragma unroll
    for (int i = 1; i < KL; ++i) {
      if (lane == i) key = best[i];
      if (i == a.k - 1) last = best[i];
    }
    const bool has = lane < a.k;
    int mine = has ? 255 - (int)(key & 255u) : 0;
    float lv = has ? not_nan(load_as_f32(a.logits, at + mine, a.type)) : -INFINITY;
    if (!exact_keys) {
      // others within the error of the last choice
      const float lastv = value_of(last & ~255u);
      const uint32_t edge = a.bias ? key_of(lastv - key_error2(a.score, lastv)) & ~255u : last & ~255u;
      unsigned within = 0, extra = 0;
#pragma unroll
      for (int i = 0; i < PL; ++i) within += full[i] >= edge ? 1u : 0u;
      const bool extras = __reduce_add_sync(kAll, within) != (unsigned)a.k;
      if (extras)
#pragma unroll
        for (int i = 0; i < PL; ++i)
          if (full[i] >= edge && ((full[i] & ~255u) | (uint32_t)(255 - id[i])) < last) extra |= 1u << i;
      const uint32_t next = __shfl_down_sync(kAll, key, 1);
      const float p = value_of(key & ~255u), v = value_of(next & ~255u);
      const bool close = lane + 1 < a.k && (a.bias ? !(p - v > key_error2(a.score, fmaxf(fabsf(p), fabsf(v))))
                                                   : (key >> 8) == (next >> 8));
      bool rank = false;  // by 64-bit scores
      int n = a.k;        // candidates
      if (!open && (extras || __any_sync(kAll, close))) {
        while (const unsigned who = __ballot_sync(kAll, extra != 0)) {  // those beyond the k: behind them, lane by lane
          const int to = n + __popc(who & ((1u << lane) - 1u));
          if (extra) {
            if (to < 32) own.id[to] = g * a.gs + sub + (__ffs(extra) - 1) * a.lanes;
            extra &= extra - 1;
          }
          n += __popc(who);
        }
        __syncwarp();
        if (lane >= a.k && lane < min(n, 32)) mine = own.id[lane];
        __syncwarp();
        open = n > 32;
        rank = a.bias && !pairs;
        if (!open && !rank) {
          if (a.bias) need_sum();
          const bool in = lane < n;
          const float x = in ? not_nan(load_as_f32(a.logits, at + mine, a.type)) : 0.f;
          const Pair c = in && a.bias ? pair_score(a, x, a.bias[mine], m, psum) : Pair{x, 0.f};
          int place = 0;
          bool near = false;
#pragma unroll 1
          for (int j = 0; j < n; ++j) {
            const Pair o = {__shfl_sync(kAll, c.hi, j), __shfl_sync(kAll, c.lo, j)};
            const int oid = __shfl_sync(kAll, mine, j);
            const float d = a.bias ? difference(o, c) : o.hi == c.hi ? 0.f : o.hi > c.hi ? 1.f : -1.f;
            place += d > 0.f || (d == 0.f && oid < mine);
            near = near || (in && j != lane && a.bias && !(fabsf(d) > pair_error2(c.hi)));
          }
          rank = __any_sync(kAll, near);
          if (!rank) {
            if (in) own.id[place] = mine;
            __syncwarp();
            if (has) mine = own.id[lane];
            __syncwarp();
          }
        }
      }
      if (open)
        mine = select_exact(a, at, m, sum, own);
      else if (rank)
        mine = rank64(a, at, m, a.n_group * a.gs, n, mine, own);
      if (has) lv = not_nan(load_as_f32(a.logits, at + mine, a.type));
    } else if (open) {
      mine = select_exact(a, at, m, sum, own);
      if (has) lv = not_nan(load_as_f32(a.logits, at + mine, a.type));
    }
    // weights
    const float mx = warp_max(lv);
    float w = 0.f;
    if (a.score == MOE_SCORE_SOFTMAX) {
      if (has) w = a.renorm ? exp_rel(lv, mx) : exp_rel(lv, m) / sum;
    } else if (has) {
      // renormalised ones are taken relative to exp(the largest logit) where that is below 0, or those far under it
      // would be subnormal, or all 0, before they are divided by their sum
      const float x = expf(-fabsf(lv));
      w = (lv >= 0.f ? 1.0f : exp_rel(lv, a.renorm ? fminf(mx, 0.f) : 0.f)) / (1.0f + x);
    }
    if (a.renorm) {
      float total = w;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);  // k <= 8
      w /= total;
    }
    if (has) {
      a.ids[(int64_t)t * a.k + lane] = mine;
      a.weights[(int64_t)t * a.k + lane] = w * a.scale;
    }
  }
}

template <int PL, int KL, bool FULL>
cudaError_t go(const RouteArgs &a, cudaStream_t stream) {
  auto kern = group_route_kernel<PL, KL, FULL>;
  static PerDevice fits;  // CTAs that are resident on the device
  const int fit = fits.get([&] {
    int n = 0;
    const bool ok = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kWarps * 32, 0) == cudaSuccess;
    return ok ? n * sm_count() : 0;
  });
  if (fit < 1) return cudaErrorUnknown;
  const int need = (a.T + kWarps - 1) / kWarps;
  return launch_pdl(kern, dim3(need < fit ? need : fit), dim3(kWarps * 32), 0, stream, a);
}

}  // namespace

moe_status_t launch_group_route(const void *logits, int type, int64_t ld, const float *bias, int T, int E, int k,
                                const moe_router_t &r, int32_t *ids, float *weights, cudaStream_t stream,
                                int *launches) {
  if (T == 0) return MOE_OK;
  RouteArgs a;
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.ld = ld;
  a.type = type;
  a.T = T;
  a.k = k;
  // without a limit the groups do not matter
  a.n_group = r.topk_group < r.n_group ? r.n_group : 1;
  a.topk_group = r.topk_group < r.n_group ? r.topk_group : 1;
  a.gs = E / a.n_group;
  int p2 = 1;
  while (p2 < a.n_group) p2 <<= 1;
  a.lanes = 32 / p2;
  a.score = r.score;
  a.top2 = r.group_score == MOE_GROUP_TOP2;
  a.renorm = r.renormalize != 0;
  a.scale = r.scale;
  const int per = (a.gs + a.lanes - 1) / a.lanes;
  const bool four = k <= 4;
  const bool full = a.n_group * a.lanes == 32 && a.gs % a.lanes == 0;
  auto sized = [&](auto pl) {
    constexpr int kPl = decltype(pl)::value;
    if (full && per == kPl) return four ? go<kPl, 4, true>(a, stream) : go<kPl, 8, true>(a, stream);
    return four ? go<kPl, 4, false>(a, stream) : go<kPl, 8, false>(a, stream);
  };
  const cudaError_t err = per <= 1   ? sized(std::integral_constant<int, 1>())
                          : per <= 2 ? sized(std::integral_constant<int, 2>())
                          : per <= 4 ? sized(std::integral_constant<int, 4>())
                          : per <= 8 ? sized(std::integral_constant<int, 8>())
                                     : sized(std::integral_constant<int, 16>());
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe4
