// Routing with expert groups: scores s = softmax(l) or sigmoid(l), selection
// scores c = s + bias (or the logits, which order the experts alike), the best
// groups, the k best experts in them, weights from s alone.
//
// One warp a token. Group g owns L = 32 / (n_group rounded up to a power of
// two) lanes, which share its experts, so a group's largest and second-largest
// scores are log2(L) shuffles; E <= 256 leaves at most 16 experts a lane.
//
// Which experts are chosen is decided on the real numbers. fp32 scores carry
// an error of up to `err` (derived at score_error below); where every gap that
// the selection rests on -- last kept group to first dropped one, each chosen
// expert to the next -- is wider than the two errors together, fp32 has the
// right order. The other rows are done again with scores in 64 bits, which
// exact ties also take (fp32 cannot tell them from near ties). Ordering by the
// logits themselves is exact, and needs no check.
#include "common.cuh"
#include "kernels.h"
#include "types.cuh"

namespace moe4 {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxK = 8;
constexpr unsigned kAll = 0xffffffffu;

struct RouteArgs {
  const void *logits;
  const float *bias;
  int32_t *ids;
  float *weights;
  int64_t ld;
  int type, T, E, k, n_group, topk_group, gs, lanes;  // gs: experts a group; lanes: lanes a group
  int score, top2, renorm;
  float scale;
};

// An unsigned key that orders as the float does (-0 made +0 before); 0 is free
// for "no candidate", below the key of -inf.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// Bound on twice the error of an fp32 selection score of size |v|.
// Sigmoid: E = ex2(-l log2 e) is off by 2^-22 + |l| 2^-23 of itself, which
// 1 / (1 + E) turns into at most s (1 - s) of that (<= 0.6e-7 + 0.27e-7), the
// sum, the reciprocal and the bias add at most 2^-24 + 2^-22 of s and 2^-24 of
// the result: below 5e-7 + 6e-8 |v|. Softmax: the exponential likewise (s
// |l - m| < 0.37), its sum of up to 256 terms at most 21 * 2^-24 + 2^-22 of
// itself (8 or 16 in a lane, five shuffles): below 2e-6 + 6e-8 |v|.
__device__ __forceinline__ float score_error2(int score, float v) {
  return (score == MOE_SCORE_SOFTMAX ? 4e-6f : 1e-6f) + 1.3e-7f * fabsf(v);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// exp(l - m) with the limits at infinite m: logits equal to m count 1, others 0.
template <typename F>
__device__ __forceinline__ F exp_rel(float l, float m) {
  if (fabsf(m) > 3.402823466e38f) return l == m ? F(1) : F(0);
  return sizeof(F) == 8 ? F(exp((double)l - (double)m)) : F(expf(l - m));
}

// The same selection with 64-bit scores, for the rows that fp32 leaves open.
// sc: scores of this lane's experts for the group stage (top2) and the expert
// stage; returns the j-th id in lane j.
template <int PL>
__device__ __noinline__ int select64(const RouteArgs &a, const float (&l)[PL], float m, int lane, int sub, int g) {
  const double none = -INFINITY;
  double s[PL];
  double sum = 0.0;
  if (a.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int x = sub + i * a.lanes;
      s[i] = (g < a.n_group && x < a.gs) ? exp_rel<double>(l[i], m) : 0.0;
      sum += s[i];
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] /= sum;
  } else {
#pragma unroll
    for (int i = 0; i < PL; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
  }
  unsigned valid = 0;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const int x = sub + i * a.lanes;
    if (g < a.n_group && x < a.gs) {
      valid |= 1u << i;
      if (a.bias) s[i] += (double)a.bias[g * a.gs + x];
      if (s[i] != s[i]) s[i] = none;
    }
  }
  if (a.topk_group < a.n_group) {
    double b1 = none, b2 = none;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if ((valid >> i) & 1u) {
        if (a.top2) {
          if (s[i] > b1) {
            b2 = b1;
            b1 = s[i];
          } else if (s[i] > b2) {
            b2 = s[i];
          }
        } else {
          b1 = fmax(b1, a.bias ? s[i] : (double)l[i]);
        }
      }
    for (int o = 1; o < a.lanes; o <<= 1) {
      const double o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
      b2 = fmax(fmin(b1, o1), fmax(b2, o2));
      b1 = fmax(b1, o1);
    }
    double gv = a.top2 ? b1 + b2 : b1;
    gv = gv == gv ? gv : none;
    int rank = 0;  // groups ahead of this lane's
    for (int h = 0; h < a.n_group; ++h) {
      const double ov = __shfl_sync(kAll, gv, h * a.lanes);
      rank += (ov > gv || (ov == gv && h < g)) ? 1 : 0;
    }
    if (rank >= a.topk_group) valid = 0;
  }
  int mine = 0;
  for (int j = 0; j < a.k; ++j) {
    double best = none;
    int bid = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int e = g * a.gs + sub + i * a.lanes;
      const double v = a.bias ? s[i] : (double)l[i];
      if (((valid >> i) & 1u) && (v > best || (v == best && e < bid))) {
        best = v;
        bid = e;
      }
    }
    const int own = bid;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(kAll, best, o);
      const int oid = __shfl_xor_sync(kAll, bid, o);
      if (ov > best || (ov == best && oid < bid)) {
        best = ov;
        bid = oid;
      }
    }
    if (own == bid) valid &= ~(1u << ((bid - g * a.gs - sub) / a.lanes));
    if (lane == j) mine = bid;
  }
  return mine;
}

template <int PL>
__global__ void __launch_bounds__(kWarps * 32) group_route_kernel(const RouteArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int g = lane / a.lanes, sub = lane & (a.lanes - 1);
  const int e0 = g * a.gs + sub;
  const int64_t row = (int64_t)t * a.ld;
  float l[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    l[i] = -INFINITY;
    if (g < a.n_group && sub + i * a.lanes < a.gs) {
      const float v = load_as_f32(a.logits, row + e0 + i * a.lanes, a.type);
      l[i] = v == v ? v : -INFINITY;
    }
  }
  const bool grouped = a.topk_group < a.n_group;
  const bool scored = a.bias || (grouped && a.top2);  // some order rests on computed scores
  float m = 0.f, sum = 1.f;
  if (a.score == MOE_SCORE_SOFTMAX && (scored || !a.renorm)) {
    m = l[0];
#pragma unroll
    for (int i = 1; i < PL; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (g < a.n_group && sub + i * a.lanes < a.gs) sum += exp_rel<float>(l[i], m);
    sum = warp_sum(sum);
  }
  uint32_t key[PL];  // order of the experts
  float sc[PL];      // computed scores
  bool open = false; // fp32 leaves the selection open
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    const bool valid = g < a.n_group && sub + i * a.lanes < a.gs;
    float v = l[i];
    if (scored && valid) {
      v = a.score == MOE_SCORE_SOFTMAX ? exp_rel<float>(l[i], m) / sum : 1.0f / (1.0f + __expf(-l[i]));
      if (a.bias) v += a.bias[e0 + i * a.lanes];
      v = v == v ? v : -INFINITY;
    }
    sc[i] = v;
    key[i] = valid ? key_of(a.bias ? v : l[i]) : 0u;
  }
  if (grouped) {
    uint32_t b1 = 0, b2 = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const uint32_t v = key[i] == 0u ? 0u : key_of(a.top2 ? sc[i] : (a.bias ? sc[i] : l[i]));
      b2 = max(b2, min(b1, v));
      b1 = max(b1, v);
    }
    for (int o = 1; o < a.lanes; o <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(kAll, b1, o), o2 = __shfl_xor_sync(kAll, b2, o);
      b2 = max(max(b2, o2), min(b1, o1));
      b1 = max(b1, o1);
    }
    uint32_t gk = 0;
    if (g < a.n_group) {
      const float v = value_of(b1) + value_of(b2);
      gk = a.top2 ? key_of(v == v ? v : -INFINITY) : b1;
    }
    // the topk_group best groups, one after another; then the best one left
    bool kept = false;
    uint32_t last = 0;
    for (int j = 0; j < a.topk_group; ++j) {
      last = __reduce_max_sync(kAll, kept ? 0u : gk);
      const int winner = __reduce_min_sync(kAll, !kept && gk == last ? g : 32);
      kept = kept || g == winner;
    }
    if (scored) {
      const uint32_t next = __reduce_max_sync(kAll, kept ? 0u : gk);
      const float lv = value_of(last), nv = value_of(next);
      open = !(lv - nv > (a.top2 ? 2.f : 1.f) * score_error2(a.score, fmaxf(fabsf(lv), fabsf(nv))));
    }
    if (!kept) {
#pragma unroll
      for (int i = 0; i < PL; ++i) key[i] = 0u;
    }
  }
  int mine = 0;
  float prev = INFINITY;
  const int rounds = a.k + (a.bias ? 1 : 0);
  for (int j = 0; j < rounds; ++j) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const uint32_t top = __reduce_max_sync(kAll, best);
    const float v = value_of(top);
    if (a.bias) {  // top 0: fewer candidates than k + 1
      if (j > 0 && top != 0u && !(prev - v > score_error2(a.score, fmaxf(fabsf(prev), fabsf(v))))) open = true;
      prev = v;
    }
    const int bid = best == top && top != 0u ? e0 + at * a.lanes : 0x7fffffff;
    const int id = __reduce_min_sync(kAll, bid);
    if (bid == id && j < a.k) {
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (i == at) key[i] = 0u;
    }
    if (lane == j) mine = id;
  }
  if (open) {
    if (a.score == MOE_SCORE_SOFTMAX) {
      m = l[0];
#pragma unroll
      for (int i = 1; i < PL; ++i) m = fmaxf(m, l[i]);
      m = warp_max(m);
    }
    mine = select64<PL>(a, l, m, lane, sub, g);
  }
  // weights: lane j has the j-th choice
  const bool has = lane < a.k;
  float lv = -INFINITY;
  if (has) {
    lv = load_as_f32(a.logits, row + mine, a.type);
    lv = lv == lv ? lv : -INFINITY;
  }
  const float mx = warp_max(lv);
  float w = 0.f;
  if (a.score == MOE_SCORE_SOFTMAX) {
    if (has) w = a.renorm ? exp_rel<float>(lv, mx) : exp_rel<float>(lv, m) / sum;
  } else if (has) {
    // far below 0 every sigmoid is exp(l), which only its ratios keep in range
    if (a.renorm && mx < -30.f) {
      w = exp_rel<float>(lv, mx);
    } else {
      const float x = expf(-fabsf(lv));
      w = lv >= 0.f ? 1.0f / (1.0f + x) : x / (1.0f + x);
    }
  }
  if (a.renorm) w /= warp_sum(w);
  if (has) {
    a.ids[(int64_t)t * a.k + lane] = mine;
    a.weights[(int64_t)t * a.k + lane] = w * a.scale;
  }
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
  a.E = E;
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
  const dim3 grid((T + kWarps - 1) / kWarps), block(kWarps * 32);
  auto go = [&](auto kern) { return launch_pdl(kern, grid, block, 0, stream, a); };
  cudaError_t err;
  if (per <= 1)
    err = go(group_route_kernel<1>);
  else if (per <= 2)
    err = go(group_route_kernel<2>);
  else if (per <= 4)
    err = go(group_route_kernel<4>);
  else if (per <= 8)
    err = go(group_route_kernel<8>);
  else
    err = go(group_route_kernel<16>);
  if (launches) ++*launches;
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe4
