// Routing with expert groups: scores s = softmax(l) or sigmoid(l), selection
// scores c = s + bias (or the logits, which order the experts alike), the best
// groups, the k best experts in them, weights from s alone.
//
// One warp a token. Group g owns L = 32 / (n_group rounded up to a power of
// two) lanes, which share its experts (E <= 256 leaves at most 16 a lane), so
// what a group needs is log2(L) shuffles. A lane sorts its experts once by a
// 32-bit key, the ordered bits of c with the low bits replaced by the expert's
// place in the lane; after that a choice is one warp-wide maximum over the
// lanes' heads, and the winning lane moves on to its next. 16-bit logits
// ordered by themselves leave room for the whole expert index, so their many
// ties are decided in the key.
//
// Which experts are chosen is decided on the real numbers. The keys carry an
// error: the truncation, and that of fp32 scores (score_error2). Where every
// gap that the selection rests on -- last kept group to first dropped one,
// each choice to the next -- is wider, the order is right. Other rows are
// `open`. Where it is the order of the k + 1 first that is, they are ranked by
// 64-bit scores, one a lane (64-bit exponentials run at a 64th of the fp32
// rate); that is about one row in 400 with random fp32 logits and a bias.
// Undecided groups, and more candidates, go through select_exact, which has
// its loops rolled up: run by a warp in ten thousand, its instructions come
// from memory each time.
#include "common.cuh"
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
// The same for a score cut to the 28 bits of a key (2^-19 of it).
__device__ __forceinline__ float key_error2(int score, float v) { return score_error2(score, v) + 2e-6f * fabsf(v); }

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

// What a warp knows of its token.
template <int PL>
struct Row {
  float l[PL];  // logits of this lane's experts (NaN as -inf)
  float m, sum; // softmax: maximum and sum of exp(l - m) over all, where needed
  int64_t at;   // of the logits in memory
  int lane, g, sub, e0;
  unsigned valid;  // which of l are experts
};

// Which experts are this lane's.
template <int PL>
__device__ __forceinline__ void enter_row(const RouteArgs &a, Row<PL> &r) {
  r.lane = threadIdx.x & 31;
  r.g = r.lane / a.lanes;
  r.sub = r.lane & (a.lanes - 1);
  r.e0 = r.g * a.gs + r.sub;
  r.valid = 0;
#pragma unroll
  for (int i = 0; i < PL; ++i)
    if (r.g < a.n_group && r.sub + i * a.lanes < a.gs) r.valid |= 1u << i;
}

// This lane's logits, all loads under way together.
template <int PL>
__device__ __forceinline__ void load_logits(const RouteArgs &a, Row<PL> &r) {
  auto each = [&](auto get) {
#pragma unroll
    for (int i = 0; i < PL; ++i) r.l[i] = (r.valid >> i) & 1u ? get(r.at + r.e0 + i * a.lanes) : -INFINITY;
  };
  if (a.type == MOE_FP32)
    each([&](int64_t i) { return load_as_f32(a.logits, i, MOE_FP32); });
  else if (a.type == MOE_BF16)
    each([&](int64_t i) { return load_as_f32(a.logits, i, MOE_BF16); });
  else
    each([&](int64_t i) { return load_as_f32(a.logits, i, MOE_FP16); });
#pragma unroll
  for (int i = 0; i < PL; ++i) r.l[i] = not_nan(r.l[i]);
}

// What orders expert e, in 64 bits.
__device__ double order64(const RouteArgs &a, int64_t at, float m, double sum, int e, bool scored) {
  const float l = not_nan(load_as_f32(a.logits, at + e, a.type));
  if (!scored) return l;
  double s = a.score == MOE_SCORE_SOFTMAX ? exp_rel64(l, m) / sum : 1.0 / (1.0 + exp(-(double)l));
  if (a.bias) s += (double)a.bias[e];
  return s == s ? s : -INFINITY;
}

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
      // the last kept and the first dropped as fp32 has it; those that are within the error of the other side
      const unsigned in = __ballot_sync(kAll, kept && ahead == a.topk_group - 1),
                     out = __ballot_sync(kAll, kept && ahead == a.topk_group);
      const float lv = __shfl_sync(kAll, gv, __ffs(in) - 1), nv = __shfl_sync(kAll, gv, __ffs(out) - 1);
      const float tol = 2.f * score_error2(a.score, fmaxf(fabsf(lv), fabsf(nv)));
      const bool sure = kept && gv > lv + tol;
      const bool maybe = kept && !sure && !(gv < nv - tol);
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

// PL: experts a lane, rounded up to a power of two
template <int PL>
__global__ void __launch_bounds__(kWarps * 32, PL <= 8 ? 7 : 5) group_route_kernel(const RouteArgs a) {
  __shared__ Scratch scratch[kWarps];
  pdl_wait();
  pdl_trigger();
  const bool grouped = a.topk_group < a.n_group;
  const bool by_score = a.bias || (grouped && a.top2);  // some order rests on computed scores
  const bool short_keys = !a.bias && a.type != MOE_FP32;  // 19 bits of order hold any, 13 of index
  Row<PL> r;
  enter_row<PL>(a, r);
  float bias[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) bias[i] = a.bias && ((r.valid >> i) & 1u) ? a.bias[r.e0 + i * a.lanes] : 0.f;
  for (int t = blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.T; t += gridDim.x * kWarps) {
    r.at = (int64_t)t * a.ld;
    load_logits<PL>(a, r);
    r.m = 0.f;
    r.sum = 1.f;
    if (a.score == MOE_SCORE_SOFTMAX && (by_score || !a.renorm)) {
      float m = r.l[0];
#pragma unroll
      for (int i = 1; i < PL; ++i) m = fmaxf(m, r.l[i]);
      r.m = warp_max(m);
      r.sum = 0.f;
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if ((r.valid >> i) & 1u) r.sum += exp_rel(r.l[i], r.m);
      r.sum = warp_sum(r.sum);
    }
    auto score = [&](float l) {
      return a.score == MOE_SCORE_SOFTMAX ? __fdividef(exp_rel(l, r.m), r.sum) : __fdividef(1.0f, 1.0f + __expf(-l));
    };
    uint32_t key[PL], full[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      full[i] = (r.valid >> i) & 1u ? key_of(a.bias ? not_nan(score(r.l[i]) + bias[i]) : r.l[i]) : 0u;
      const uint32_t cut = short_keys ? (full[i] & ~0x1FFFu) | (0x1FFFu - (uint32_t)(r.e0 + i * a.lanes))
                                      : (full[i] & ~15u) | (uint32_t)(15 - i);
      key[i] = full[i] ? cut : 0u;
    }
    sort_keys<PL>(key);
    bool open = false;         // the groups, or too many candidates, are undecided
    bool open_order = false;   // so is the order of the first k + 1
    if (grouped) {
      uint32_t b1 = key[0], b2 = PL > 1 ? key[PL > 1] : 0u;
      if (by_score) {  // whole, not as the keys have them: the scores, or the logits whose scores are wanted
        b1 = b2 = 0u;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
          b2 = max(b2, min(b1, full[i]));
          b1 = max(b1, full[i]);
        }
      }
      for (int o = 1; o < a.lanes; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
        b2 = max(max(b2, o2), min(b1, o1));
        b1 = max(b1, o1);
      }
      uint32_t gk = 0;
      if (r.g < a.n_group) {
        const float x = value_of(b1), y = value_of(b2);
        gk = !a.top2 ? b1 : key_of(not_nan(a.bias ? x + y : score(x) + score(y)));
      }
      int ahead = 0;  // groups before this one; equal ones by index
      for (int h = 0; h < a.n_group; ++h) {
        const uint32_t ok = __shfl_sync(kAll, gk, h * a.lanes);
        ahead += ok > gk || (ok == gk && h < r.g);
      }
      const bool kept = r.g < a.n_group && ahead < a.topk_group;
      const uint32_t last = __reduce_min_sync(kAll, kept ? gk : kAll), next = __reduce_max_sync(kAll, kept ? 0u : gk);
      if (by_score) {
        const float lv = value_of(last), nv = value_of(next);
        open = !(lv - nv > (a.top2 ? 2.f : 1.f) * score_error2(a.score, fmaxf(fabsf(lv), fabsf(nv))));
      } else if (!short_keys) {
        open = (last >> 4) == (next >> 4);
      }
      if (!kept) {
#pragma unroll
        for (int i = 0; i < PL; ++i) key[i] = 0u;
      }
    }
    int mine = 0;
    uint32_t prev = kAll, kth = 0;
    int candidates = 0;
    // the two after the last choice decide whether that one is sure, and whether the first k + 1 are all that matter
    const int rounds = a.k + (short_keys ? 0 : 2);
    for (int j = 0; j < rounds; ++j) {
      const uint32_t top = __reduce_max_sync(kAll, key[0]);
      const unsigned who = __ballot_sync(kAll, key[0] == top);
      if (top == 0u) break;  // fewer candidates than k + 2
      candidates = j + 1;
      const int from = __ffs(who) - 1;
      if (!short_keys) {
        auto close = [&](uint32_t hi, uint32_t lo) {
          if (!a.bias) return (hi >> 4) == (lo >> 4);
          const float p = value_of(hi & ~15u), v = value_of(lo & ~15u);
          return !(p - v > key_error2(a.score, fmaxf(fabsf(p), fabsf(v))));
        };
        if (j == a.k + 1)
          open = open || close(kth, top);
        else if (j > 0)
          open_order = open_order || close(prev, top);
        if (j == a.k - 1) kth = top;
      }
      prev = top;
      const int id = short_keys ? (int)(0x1FFFu - (top & 0x1FFFu))
                                : __shfl_sync(kAll, r.e0, from) + (int)(15u - (top & 15u)) * a.lanes;
      if (r.lane == j) mine = id;
      if (r.lane == from) {
#pragma unroll
        for (int i = 0; i + 1 < PL; ++i) key[i] = key[i + 1];
        key[PL - 1] = 0u;
      }
    }
    if (open)
      mine = select_exact(a, r.at, r.m, r.sum, scratch[threadIdx.x >> 5]);
    else if (open_order)
      mine = rank64(a, r.at, r.m, a.n_group * a.gs, min(a.k + 1, candidates), mine, scratch[threadIdx.x >> 5]);
    // weights: lane j has the j-th choice
    const bool has = r.lane < a.k;
    const float lv = has ? not_nan(load_as_f32(a.logits, r.at + mine, a.type)) : -INFINITY;
    const float mx = warp_max(lv);
    float w = 0.f;
    if (a.score == MOE_SCORE_SOFTMAX) {
      if (has) w = a.renorm ? exp_rel(lv, mx) : exp_rel(lv, r.m) / r.sum;
    } else if (has) {
      // far below 0 every sigmoid is exp(l), which only its ratios keep in range
      if (a.renorm && mx < -30.f) {
        w = exp_rel(lv, mx);
      } else {
        const float x = expf(-fabsf(lv));
        w = lv >= 0.f ? 1.0f / (1.0f + x) : x / (1.0f + x);
      }
    }
    if (a.renorm) {
      float sum = w;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);  // k <= 8
      w /= sum;
    }
    if (has) {
      a.ids[(int64_t)t * a.k + r.lane] = mine;
      a.weights[(int64_t)t * a.k + r.lane] = w * a.scale;
    }
  }
}

template <int PL>
cudaError_t go(const RouteArgs &a, cudaStream_t stream) {
  static int fit = 0;  // CTAs that are resident on the device
  if (fit == 0) {
    int dev = 0, sms = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, group_route_kernel<PL>, kWarps * 32, 0);
    if (e != cudaSuccess) return e;
    fit = sms * n;
  }
  const int need = (a.T + kWarps - 1) / kWarps;
  return launch_pdl(group_route_kernel<PL>, dim3(need < fit ? need : fit), dim3(kWarps * 32), 0, stream, a);
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
  cudaError_t err;
  if (per <= 1)
    err = go<1>(a, stream);
  else if (per <= 2)
    err = go<2>(a, stream);
  else if (per <= 4)
    err = go<4>(a, stream);
  else if (per <= 8)
    err = go<8>(a, stream);
  else
    err = go<16>(a, stream);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe4
