// Attention of one new token a sequence over the paged key-value cache.
//
//   out = sum_i p_i v_i / (sum_i p_i + sink),  p_i = exp(scale q.k_i - m)
//
// with the running maximum m and sum held per query head in fp32, in one pass
// over the cache; log2 units throughout (p = exp2).
//
// What bounds it is the reading of the cache: G query heads share a key, so a
// byte read carries only G (16-bit) to 4 G (4-bit) multiply-adds. The design
// is around keeping bulk copies in flight:
//  - A record (16 tokens of one head: keys, values and their scales) is one
//    contiguous piece of memory. Each warp has its own ring of STAGES records
//    in shared memory, filled by one bulk copy each (one lane issues, an
//    mbarrier counts the bytes), so warps run free of each other.
//  - The matrix products are transposed, S^T[key][head] = K Q^T and
//    O^T[d][head] = V^T P^T, so that the 16 rows of an mma.sync are 16 keys or
//    16 columns and its 8 columns are heads: up to 8 heads of a group cost no
//    padding. tcgen05 would want 128 keys a tile for the same 8 columns and a
//    round trip of P through shared memory; at these intensities the tensor
//    pipe is nowhere near its limit either way.
//  - FP8 and NVFP4 codes are expanded in registers to f16, exactly (E2M1 times
//    its E4M3 block scale has 6 significant bits); the power-of-two row scales
//    never touch them: the key's multiplies its scores, the value's is added
//    to the exponent of its probabilities. The query is scaled by a power of
//    two into f16 range.
//  - The maximum is lazy: it moves only when a score passes it by 4 (in log2),
//    so the accumulators are seldom rescaled. Where p is multiplied as f16 it
//    is lifted by 2^11, to at most 2^15: what falls under f16's normal range
//    (relative precision is lost there) is 2^-25 of the largest.
//  - P is rounded to the type that it is multiplied in, bf16 for BF16 caches
//    (2^-8 of it at most) and f16 otherwise (2^-11); its sum is taken before.
//    The outputs' error against 64 bits is then 0.0020 for BF16 caches of long
//    contexts and 0.0017 otherwise, as with fp32 probabilities, whose 0.0017 is
//    the rounding of the output. P as two bf16 terms gives BF16 caches 0.0017 too
//    and takes 4% longer at 64 columns, 11% at 256.
//
// Work is split evenly over all records of all sequences and heads, whatever
// their lengths. Lay the records out one (sequence, head) after another, each
// preceded by kLead empty units, which stand for the time that beginning and
// ending one takes; CTA c takes units [c * per, (c + 1) * per) and each of its
// warps a quarter of them. A (sequence, head) that falls to one warp is written
// from its registers; what is shared by warps of a CTA is joined in shared
// memory, once at the end; what is shared by CTAs goes to the workspace as a
// partial output with its log-sum, and a second kernel joins those. All orders
// are fixed, so results do not vary from run to run.
// The second kernel is not needed in two cases. Where no (sequence, head) can be
// long, CTAs take whole ones, even shares of the units moved to the nearest
// beginning of one. Where there are few and none is very long, a cluster of 2, 4
// or 8 CTAs takes one and joins it through distributed shared memory.
//
// 16 sequences of 65536 tokens in BF16, 32 heads on 8 of 128: 610 us, 104% of the
// copy bandwidth. 32 of 32768, 64 heads on 8 of 64: FP8 199 us, 81%; NVFP4 196 us,
// 47%: 283 instructions a record at 63% of the issue slots with 3.7 warps a
// scheduler. Of 5.9 cycles between two instructions of a warp 1.6 are the latency
// of the one before, 1.0 other warps' turns, 0.7 a busy pipe (the ALU's, which the
// conversions of codes share, is 50% busy, the others less).
#include <algorithm>

#include "common.cuh"
#include "device.cuh"
#include "kernels.h"
#include "kvcache.cuh"
#include "types.cuh"

namespace moe4 {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kW = 4;              // warps of a CTA
constexpr int kMaxCtas = 640;      // partial outputs the workspace holds: two a CTA
constexpr int kMaxB = 4096;
constexpr int kJoinThreads = 256;
constexpr int kCluster = 8;        // CTAs of a cluster, at most
// How CTAs share the work: even shares of all units, whole (sequence, head)s, one of them, or a cluster one of them.
enum { kStream = 0, kWhole = 1, kSingle = 2, kClustered = 3 };
constexpr int kLead = 5;           // empty units before each (sequence, head)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 4.f;      // lazy maximum, log2

struct AttnArgs {
  const void *q;
  const uint8_t *data;
  const int32_t *table, *lens;
  const float *sinks;
  void *out;
  float *lse;
  unsigned int *status;
  int64_t *per;      // units a CTA
  int *starts;       // [B + 1] first record of each sequence, as if of one head
  float *part_o;     // [2 kMaxCtas][NH][D]
  float *part_lse;   // [2 kMaxCtas][NH], log2
  int64_t qsb, qsh, osb, osh, ts;
  int q_type, B, heads, kv_heads, G, GB, window, page, pages, max_pages, ctas, mode, cluster;
  float scale;       // scale * log2 e
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// low half from x, high half from y
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  uint32_t r;
  if (BF)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
  return h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// 8 E2M1 codes to 4 pairs
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t *h) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Tokens of sequence b that are read: [first, len), in records [lo, lo + n), n >= 1.
struct Span {
  int len, first, lo, n;
};

__device__ __forceinline__ Span span_of(const AttnArgs &a, int b) {
  Span s;
  const int cap = a.max_pages * a.page;
  s.len = min(max(a.lens[b], 0), cap);
  s.first = a.window > 0 ? max(0, s.len - a.window) : 0;
  s.lo = s.first >> 4;
  s.n = max(1, ((s.len + 15) >> 4) - s.lo);
  return s;
}

// Compile-time shape: NT column tiles of 8 heads a CTA.
template <int FMT, int D, int NT>
struct Shape {
  static constexpr bool kBf = FMT == MOE_KV_BF16;
  static constexpr bool kQuant = FMT >= MOE_KV_FP8;
  static constexpr float kLift = kBf ? 0.f : 11.f;  // log2, of the p that are multiplied
  static constexpr int kRow = kv_row(FMT, D);
  static constexpr int kRec = kv_record(FMT, D);
  static constexpr int kStage = (kRec + 127) / 128 * 128;
  // records in flight a warp, and how many of them are asked for at a time
  static constexpr int kStages = kRec >= 8192 ? 2 : kRec >= 4096 ? 3 : kRec >= 2048 ? 4 : 8;
  static constexpr int kGroup = kStages / 2;
  // records that a warp works on at a time: two of FP8 and NVFP4, whose time is instructions (what is done once a tile,
  // waiting, voting, branching, is a third of them); 16-bit caches wait for memory
  static constexpr int kTile = kQuant && NT == 1 && kStages >= 4 ? 2 : 1;
  static constexpr int kHeads = 8 * NT;
  // FP8, NVFP4: codes of a lane's load of a key (16 bytes, 8 of a 32-byte row), and of a value
  static constexpr int kKeyCodes = (kRow >= 64 ? 16 : 8) * (FMT == MOE_KV_NVFP4 ? 2 : 1);
  static constexpr int kValCodes = D / 8 < 16 * (FMT == MOE_KV_NVFP4 ? 2 : 1) ? D / 8 : 16 * (FMT == MOE_KV_NVFP4 ? 2 : 1);
  static constexpr int kKeyLoads = D / 4 / kKeyCodes, kValLoads = D / 8 / kValCodes;
  // column of code e of a key's lane c (of 4), and of a value's lane r (of 8): loads lie next to each other by lane
  __host__ __device__ static constexpr int key_col(int c, int e) {
    return e / kKeyCodes * 4 * kKeyCodes + c * kKeyCodes + e % kKeyCodes;
  }
  __host__ __device__ static constexpr int val_col(int r, int e) {
    return e / kValCodes * 8 * kValCodes + r * kValCodes + e % kValCodes;
  }
  static constexpr int kLdo = D + 4;  // row of the joining buffer, padded against bank conflicts
  static constexpr int kJoin = kW * kHeads * kLdo * 4;
  static constexpr int kMl = 2 * kW * kHeads * 3 * 4;
  static_assert(kStages * kStage >= kHeads * kLdo * 4, "a partial output fits the ring");
  static constexpr int kRing = kW * kStages * kStage;
  static constexpr int kFixed = kRing + kJoin + kMl + kW * kStages * 8;
};

// One (sequence, head) of a warp's range.
struct Seg {
  int64_t at;         // its first unit
  int b, hb;          // sequence; kv head * GB + block of heads
  int rec, end;       // this warp's records of it, relative to the span
  Span s;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Shared memory at this CTA's address `addr` in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// log2-sum `lse2` with the sink's logit, and the factor that the output takes.
__device__ __forceinline__ float with_sink(const AttnArgs &a, int head, float lse2, float &g) {
  if (!a.sinks) return lse2;
  const float sk = a.sinks[head] * kLog2e;
  const float top = fmaxf(lse2, sk);
  if (top == -INFINITY) return lse2;
  const float all = top + log2f(ex2(lse2 - top) + ex2(sk - top));
  if (lse2 != -INFINITY) g *= ex2(lse2 - all);
  return all;
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(kW * 32) attn_kernel(const AttnArgs a) {
  using S = Shape<FMT, D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;  // row and column of mma fragments
  // Tokens that rows r and r + 8 of S^T stand for: r and r + 8, or for FP8 and NVFP4 two neighbours, in an order in
  // which the lanes of every load of keys and of values fall into different banks.
  const int key0 = !S::kQuant ? r : r & 1 ? 8 + 2 * ((r >> 1) ^ 2) : r;
  // ring of records; once it is drained, the warp's last partial output
  uint8_t *ring = smem + warp * S::kStages * S::kStage;
  const uint32_t ring32 = smem_u32(ring);
  float *join_o = reinterpret_cast<float *>(smem + S::kRing);                // [kW] first partial outputs
  float *join_ml = reinterpret_cast<float *>(smem + S::kRing + S::kJoin);    // [2 kW][heads][3]
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kRing + S::kJoin + S::kMl);
  int *start = reinterpret_cast<int *>(smem + S::kFixed);  // [B + 1] first record of each sequence
  __shared__ int warp_sum[kW];
  __shared__ float share_lse[S::kHeads];     // what this CTA has for its cluster, with the outputs over the rings
  __shared__ int seg_of[kW][2], ends0[kW];  // (sequence, head) of each warp's first and last partial, or -1

  // Places of this lane's loads in a record, FP8 and NVFP4. Held in registers (the compiler would rather work them out
  // again at every use, six instructions each).
  [[maybe_unused]] int k_at[S::kKeyLoads][2], v_at[S::kValLoads][4], ks_at = 0, vs_at[2] = {0, 0}, ex_at = 0;
  if constexpr (S::kQuant) {
    constexpr int kPacked = FMT == MOE_KV_NVFP4 ? 2 : 1;  // codes a byte
    auto hold = [](int v) {
      asm volatile("" : "+r"(v));
      return v;
    };
#pragma unroll
    for (int p = 0; p < S::kKeyLoads; ++p)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        k_at[p][x] = hold(kv_place(S::kRow, key0 + x, S::key_col(c, p * S::kKeyCodes) / kPacked));
#pragma unroll
    for (int p = 0; p < S::kValLoads; ++p)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        v_at[p][x] = hold(16 * S::kRow + kv_place(S::kRow, 2 * c + (x >> 1) + (x & 1 ? 8 + 2 * (c ^ 2) - 2 * c : 0),
                                                  S::val_col(r, p * S::kValCodes) / kPacked));
    ks_at = hold(kv_scales_at(FMT, D) + S::key_col(c, 0) + key0);
    vs_at[0] = hold(kv_scales_at(FMT, D) + D + (S::val_col(r, 0) & ~15) + 2 * c);
    vs_at[1] = hold(kv_scales_at(FMT, D) + D + (S::val_col(r, 0) & ~15) + 8 + 2 * (c ^ 2));
    ex_at = hold(kv_exps_at(FMT, D) + key0);
  }
  const uint32_t bar0 = smem_u32(bars + warp * S::kStages);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) mbar_init(bar0 + 8 * i, 1);
    fence_mbar_init();
    seg_of[warp][0] = seg_of[warp][1] = -1;
  }
  pdl_wait();
  pdl_trigger();

  const int HB = a.kv_heads * a.GB;
  auto bad_length = [&](int b) { return a.lens[b] < 0 || a.lens[b] > a.max_pages * a.page; };
  auto seg_at = [&](int64_t u) {  // the (sequence, head) that unit u falls in
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (((int64_t)start[mid] + (int64_t)mid * kLead) * HB <= u)
        lo = mid;
      else
        hi = mid;
    }
    const int64_t at = ((int64_t)start[lo] + (int64_t)lo * kLead) * HB;
    const int units = start[lo + 1] - start[lo] + kLead;
    Seg s = {};
    s.b = lo;
    s.hb = (int)((u - at) / units);
    s.at = at + (int64_t)s.hb * units;
    return s;
  };
  Seg cu;
  int64_t cta0, cta1;  // this CTA's units
  if (a.mode >= kSingle) {  // which (sequence, head) is known; its records are units 0 .. n
    const int ranks = a.cluster, seg = blockIdx.x / ranks, rank = blockIdx.x % ranks;
    cu.b = seg / HB;
    cu.hb = seg % HB;
    cu.at = -kLead;
    const int64_t n = span_of(a, cu.b).n;
    cta0 = n * rank / ranks;
    cta1 = n * (rank + 1) / ranks;
    if (rank == 0 && cu.hb == 0 && tid == 0 && bad_length(cu.b)) raise_status(a.status, MOE_ERR_BAD_INDEX);
    __syncwarp();  // the barriers are set up
  } else {
    // first record of every sequence: running sum of their record counts
    int base = 0;
    for (int b0 = 0; b0 < a.B; b0 += kW * 32) {
      const int b = b0 + tid;
      int n = 0;
      if (b < a.B) {
        n = span_of(a, b).n;
        if (blockIdx.x == 0 && bad_length(b)) raise_status(a.status, MOE_ERR_BAD_INDEX);
      }
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) warp_sum[warp] = x;
      __syncthreads();
      int before = base;
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        if (w < warp) before += warp_sum[w];
        base += warp_sum[w];
      }
      if (b < a.B) start[b] = before + x - n;
      __syncthreads();
    }
    if (tid == 0) start[a.B] = base;
    __syncthreads();
    const int64_t total = ((int64_t)base + (int64_t)a.B * kLead) * HB;
    if (a.mode == kWhole) {
      // even shares, moved to the nearest beginning of a (sequence, head)
      auto whole = [&](int c) {
        const int64_t u = total * c / a.ctas;
        if (u >= total) return total;
        const Seg s = seg_at(u);
        const int units = start[s.b + 1] - start[s.b] + kLead;
        return 2 * (u - s.at) < units ? s.at : s.at + units;
      };
      const int64_t edge = whole(blockIdx.x + (lane & 1));  // both searches at once
      cta0 = __shfl_sync(kAll, edge, 0);
      cta1 = __shfl_sync(kAll, edge, 1);
    } else {
      const int64_t per = (total + a.ctas - 1) / a.ctas;
      if (blockIdx.x == 0) {  // what the joining kernel needs of this
        if (tid == 0) *a.per = per;
        for (int b = tid; b <= a.B; b += kW * 32) a.starts[b] = start[b];
      }
      cta0 = (int64_t)blockIdx.x * per;
      cta1 = min(cta0 + per, total);
    }
    if (cta0 >= cta1) return;
  }
  const int64_t share = (cta1 - cta0 + kW - 1) / kW;
  const int64_t u0 = min(cta0 + warp * share, cta1), u1 = min(u0 + share, cta1);
  if (a.mode < kSingle && u0 < u1) cu = seg_at(u0);

  // the records of the (sequence, head) k.b, k.hb that begins at unit k.at
  auto fill = [&](Seg &k) {
    k.s = span_of(a, k.b);
    const int64_t r0 = k.at + kLead;  // unit of record 0
    k.rec = (int)max((int64_t)0, u0 - r0);
    k.end = (int)min((int64_t)k.s.n, u1 - r0);
  };
  // on to the next one; false at the end of the range
  auto next = [&](Seg &k) {
    k.at += k.s.n + kLead;
    if (k.at >= u1) return false;
    if (++k.hb == HB) {
      k.hb = 0;
      ++k.b;
    }
    fill(k);
    return true;
  };
  bool more = u0 < u1;
  if (more) fill(cu);

  // ------------------------------------------------ copies, issued ahead of their use
  Seg is = cu;
  bool is_more = more;
  int issued = 0;  // copies issued by this warp
  int ids = -1, ids_next = -1;  // pages of records batch .. batch + 31 of the issuing segment, and of the 32 after
  int batch = 0;
  bool fresh = true;
  unsigned missing = 0;    // ring slots whose record lies in no page (bit a stage)
  const int page16 = a.page >> 4;
  auto page_of = [&](int rec) {
    return rec < is.end && is.s.len > 0 ? a.table[is.b * a.ts + (is.s.lo + rec) / page16] : -1;
  };
  // asks for up to kGroup records of one segment, lane i for the i-th; the ring has room for them
  auto issue = [&]() {
    while (is_more && is.rec >= is.end) {
      is_more = next(is);
      fresh = true;
    }
    if (!is_more) return;
    if (fresh || is.rec == batch + 32) {
      ids = fresh ? page_of(is.rec + lane) : ids_next;
      batch = is.rec;
      fresh = false;
      ids_next = page_of(batch + 32 + lane);
    }
    const int n = min(min(S::kGroup, is.end - is.rec), batch + 32 - is.rec);
    const int pg = __shfl_sync(kAll, ids, (is.rec - batch + lane) & 31);
    const int slot = (issued + lane) % S::kStages;
    const bool mine = lane < n, ok = pg >= 0 && pg < a.pages;
    if (mine) {
      if (ok) {
        const int off = (is.s.lo + is.rec + lane) % page16;
        const int64_t rec = ((int64_t)pg * a.kv_heads + is.hb / a.GB) * page16 + off;
        mbar_arrive_expect_tx(bar0 + 8 * slot, S::kRec);
        bulk_load(ring32 + slot * S::kStage, a.data + rec * S::kRec, S::kRec, bar0 + 8 * slot);
      } else {
        if (is.s.len > 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
        mbar_arrive(bar0 + 8 * slot);
      }
    }
    const unsigned lost = __ballot_sync(kAll, mine && !ok);
    if (lost | missing)
      for (int i = 0; i < n; ++i) {
        const unsigned bit = 1u << ((issued + i) % S::kStages);
        missing = (lost >> i) & 1u ? missing | bit : missing & ~bit;
      }
    issued += n;
    is.rec += n;
  };
#pragma unroll 1
  for (int i = 0; i < S::kStages / S::kGroup; ++i) issue();

  bool dead = false;  // a copy did not arrive in time: issue no more
  int done = 0;       // records consumed
  int dead_at = 0;    // the first that did not arrive
  for (; more; more = next(cu)) {
    if (cu.rec >= cu.end) continue;  // only empty units of it
    const bool begins = cu.rec == 0 && a.mode != kClustered, ends = cu.end == cu.s.n;
    const int kvh = cu.hb / a.GB, h0 = kvh * a.G + (cu.hb % a.GB) * S::kHeads;
    const int nh = min(S::kHeads, a.G - (cu.hb % a.GB) * S::kHeads);
    // ---- the query of this (sequence, heads): B fragments, head r of each tile
    uint32_t qf[NT][D / 16][2];
    float qs[NT][2];  // factor of the scores of heads 2c, 2c + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = 8 * nt + r;
      const uint16_t *qp = static_cast<const uint16_t *>(a.q) + cu.b * a.qsb + (int64_t)(h0 + h) * a.qsh;
      uint32_t raw[D / 8];
#pragma unroll
      for (int e = 0; e < D / 8; ++e) {  // pairs 2e, 2e + 1 of this lane's D / 4 columns
        int d;
        if (!S::kQuant)
          d = (e >> 1) * 16 + (e & 1) * 8 + 2 * c;
        else
          d = S::key_col(c, 2 * e);
        raw[e] = h < nh ? *reinterpret_cast<const uint32_t *>(qp + d) : 0u;
      }
      qs[nt][0] = qs[nt][1] = a.scale;
      if (S::kQuant) {  // f16 times a power of two that brings the largest to [2^14, 2^15)
        float2 f[D / 8];
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
          if (a.q_type == MOE_BF16)
            f[e] = make_float2(__uint_as_float(raw[e] << 16), __uint_as_float(raw[e] & 0xFFFF0000u));
          else
            f[e] = __half22float2(*reinterpret_cast<const __half2 *>(&raw[e]));
          amax = fmaxf(amax, fmaxf(fabsf(f[e].x), fabsf(f[e].y)));
        }
        amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 2));
        // exponent of amax, kept to where 2^e and 2^-e are normal fp32
        const int e14 = min(max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -112), 112);
        const float up = __uint_as_float((uint32_t)(127 - e14) << 23);
#pragma unroll
        for (int e = 0; e < D / 8; ++e) raw[e] = pack2<false>(f[e].x * up, f[e].y * up);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int ex = __shfl_sync(kAll, e14, (2 * c + x) * 4);
          qs[nt][x] = a.scale * __uint_as_float((uint32_t)(127 + ex) << 23);
        }
      }
#pragma unroll
      for (int e = 0; e < D / 8; ++e) qf[nt][e >> 1][e & 1] = raw[e];
    }

    // lazy maxima, of the scores (ref, thr) and of the scores with the value's row scale (refw, thrw): exponentials
    // are taken against ref, a score above thr moves it
    float ref[NT][2], thr[NT][2], refw[NT][2], thrw[NT][2], l[NT][2];
    float o[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        ref[nt][x] = refw[nt][x] = l[nt][x] = 0.f;
        thr[nt][x] = thrw[nt][x] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[nt][i][x] = 0.f;
    }

#pragma unroll 1
    for (; cu.rec < cu.end; cu.rec += S::kTile) {
      // kTile records at a time; of one that is not there (past the range, in no page) no token is read
      const int pos = (cu.s.lo + cu.rec) * 16;
      bool there[S::kTile], here = true;
      bool edge = pos < cu.s.first || pos + 16 * S::kTile > cu.s.len;  // not all of the tokens are read
#pragma unroll
      for (int n = 0; n < S::kTile; ++n) {
        const int slot = (done + n) % S::kStages;
        there[n] = n == 0 || cu.rec + n < cu.end;
        here = here && (!there[n] || mbar_try_wait(bar0 + 8 * slot, ((done + n) / S::kStages) & 1));
        there[n] = there[n] && !((missing >> slot) & 1u);
        edge = edge || !there[n];
      }
      if (!dead && !__all_sync(kAll, here)) {  // not all there yet
        const int n = min(S::kTile, cu.end - cu.rec);
        for (int i = 0; i < n && !dead; ++i) {
          const bool late = !mbar_wait(bar0 + 8 * ((done + i) % S::kStages), ((done + i) / S::kStages) & 1);
          if (__any_sync(kAll, late)) {
            if (late) raise_status(a.status, MOE_ERR_TIMEOUT);
            dead = true;
            dead_at = done + i;
          }
        }
      }
      if (!dead) {
        auto read = [&](int n, int key) {
          return there[n] && pos + 16 * n + key >= cu.s.first && pos + 16 * n + key < cu.s.len;
        };
        const uint8_t *st[S::kTile];
        uint32_t st32[S::kTile];
#pragma unroll
        for (int n = 0; n < S::kTile; ++n) {
          st[n] = ring + (done + n) % S::kStages * S::kStage;
          st32[n] = ring32 + (done + n) % S::kStages * S::kStage;
        }
        // ---- S^T = K Q^T
        float sc[S::kTile][NT][4];
#pragma unroll
        for (int n = 0; n < S::kTile; ++n) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[n][nt][x] = 0.f;
        if constexpr (!S::kQuant) {
          const int key = (lane & 7) + (lane & 8);
          const int half = lane >> 4;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t af[4];
            ldsm4(af, st32[n] + kv_place(S::kRow, key, 32 * ks + 16 * half));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma<S::kBf>(sc[n][nt], af, qf[nt][ks][0], qf[nt][ks][1]);
          }
        } else {
#pragma unroll
          for (int p = 0; p < S::kKeyLoads; ++p) {  // one load of each of the two keys
            if constexpr (FMT == MOE_KV_FP8) {
              const uint4 x = *reinterpret_cast<const uint4 *>(st[n] + k_at[p][0]);
              const uint4 y = *reinterpret_cast<const uint4 *>(st[n] + k_at[p][1]);
              const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t af[4] = {e4m3x2_f16x2(xs[k] & 0xFFFFu), e4m3x2_f16x2(ys[k] & 0xFFFFu),
                                        e4m3x2_f16x2(xs[k] >> 16), e4m3x2_f16x2(ys[k] >> 16)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma<false>(sc[n][nt], af, qf[nt][4 * p + k][0], qf[nt][4 * p + k][1]);
              }
            } else {
              uint32_t xs[4], ys[4];
              if constexpr (S::kKeyCodes == 32) {
                *reinterpret_cast<uint4 *>(xs) = *reinterpret_cast<const uint4 *>(st[n] + k_at[p][0]);
                *reinterpret_cast<uint4 *>(ys) = *reinterpret_cast<const uint4 *>(st[n] + k_at[p][1]);
              } else {
                *reinterpret_cast<uint2 *>(xs) = *reinterpret_cast<const uint2 *>(st[n] + k_at[p][0]);
                *reinterpret_cast<uint2 *>(ys) = *reinterpret_cast<const uint2 *>(st[n] + k_at[p][1]);
              }
#pragma unroll
              for (int b = 0; b < S::kKeyCodes / 16; ++b) {  // a block of 16
                const uint32_t s2 = e4m3x2_f16x2(*reinterpret_cast<const uint16_t *>(
                    st[n] + ks_at + 4 * S::kKeyCodes * p + 16 * b));  // scales of both keys
                const uint32_t fx = __byte_perm(s2, 0, 0x1010), fy = __byte_perm(s2, 0, 0x3232);
                uint32_t hx[8], hy[8];
                e2m1x8_f16(xs[2 * b], hx);
                e2m1x8_f16(xs[2 * b + 1], hx + 4);
                e2m1x8_f16(ys[2 * b], hy);
                e2m1x8_f16(ys[2 * b + 1], hy + 4);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t af[4] = {hmul2(hx[2 * k], fx), hmul2(hy[2 * k], fy), hmul2(hx[2 * k + 1], fx),
                                          hmul2(hy[2 * k + 1], fy)};
                  const int ks = (p * (S::kKeyCodes / 16) + b) * 4 + k;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) mma<false>(sc[n][nt], af, qf[nt][ks][0], qf[nt][ks][1]);
                }
              }
            }
          }
        }
        }
        // ---- scores in log2; tw = score + log2 of the value's row scale
        float tw[S::kTile][NT][4];
#pragma unroll
        for (int n = 0; n < S::kTile; ++n) {
        float kx[2] = {1.f, 1.f}, vx[2] = {0.f, 0.f};
        if constexpr (S::kQuant) {
          const uint8_t *ex = st[n] + ex_at;
          const uint32_t k2 = *reinterpret_cast<const uint16_t *>(ex), v2 = *reinterpret_cast<const uint16_t *>(ex + 16);
          // 255 marks a row with a NaN, its codes are 0: 0 * 2^128 makes the key's score NaN by itself
          kx[0] = __uint_as_float((k2 & 255u) << 23);
          kx[1] = __uint_as_float((k2 >> 8) << 23);
          const float nan = __int_as_float(0x7fc00000);
          const uint32_t v0 = v2 & 255u, v1 = v2 >> 8;
          vx[0] = v0 == 255u ? nan : __uint_as_float(0x4B000000u | v0) - 8388735.f;  // v0 - 127
          vx[1] = v1 == 255u ? nan : __uint_as_float(0x4B000000u | v1) - 8388735.f;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            sc[n][nt][x] *= S::kQuant ? qs[nt][x & 1] * kx[x >> 1] : qs[nt][x & 1];
            if (S::kQuant) tw[n][nt][x] = sc[n][nt][x] + vx[x >> 1];
          }
        if (edge) {
          const bool in[2] = {read(n, key0), read(n, S::kQuant ? key0 + 1 : key0 + 8)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (!in[x >> 1]) sc[n][nt][x] = tw[n][nt][x] = -INFINITY;
        }
        }
        // the largest of the lane's tokens
        float top[NT][2], topw[NT][2];
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            top[nt][x] = fmaxf(sc[0][nt][x], sc[0][nt][x + 2]);
            if (S::kTile > 1) top[nt][x] = fmaxf(top[nt][x], fmaxf(sc[S::kTile - 1][nt][x], sc[S::kTile - 1][nt][x + 2]));
            grow |= top[nt][x] > thr[nt][x];
            if (S::kQuant) {
              topw[nt][x] = fmaxf(tw[0][nt][x], tw[0][nt][x + 2]);
              if (S::kTile > 1)
                topw[nt][x] = fmaxf(topw[nt][x], fmaxf(tw[S::kTile - 1][nt][x], tw[S::kTile - 1][nt][x + 2]));
              grow |= topw[nt][x] > thrw[nt][x];
            }
          }
        if (__any_sync(kAll, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              // the maximum over the tokens, lifted where the exponentials are multiplied as f16
              auto move = [&](float t, float lift, float &rf, float &th) {
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) t = fmaxf(t, __shfl_xor_sync(kAll, t, sh));
                const float old = th == -INFINITY ? -INFINITY : rf + lift;
                if (!(t > old)) return 1.f;
                rf = t - lift;
                th = t + kSlack;
                return ex2(old - t);
              };
              float f = move(top[nt][x], S::kQuant ? 0.f : S::kLift, ref[nt][x], thr[nt][x]);
              l[nt][x] *= f;
              if (S::kQuant) f = move(topw[nt][x], S::kLift, refw[nt][x], thrw[nt][x]);
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[nt][i][x] *= f;
                o[nt][i][x + 2] *= f;
              }
            }
        }
        // ---- p, its sum, and P^T as B fragments: lane (r, c) gets head r, rows 2c, 2c + 1 (pf[0]) and + 8 (pf[1])
        uint32_t pf[S::kTile][NT][2];
#pragma unroll
        for (int n = 0; n < S::kTile; ++n)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float p = ex2(sc[n][nt][x] - ref[nt][x & 1]);
            l[nt][x & 1] += p;
            w[x] = S::kQuant ? ex2(tw[n][nt][x] - refw[nt][x & 1]) : p;
          }
          pf[n][nt][0] = transpose8(pack2<S::kBf>(w[0], w[1]));
          pf[n][nt][1] = transpose8(pack2<S::kBf>(w[2], w[3]));
        }
        // ---- O^T += V^T P^T; values of tokens that are not read may be anything (0 * NaN must not come in)
#pragma unroll
        for (int n = 0; n < S::kTile; ++n) {
        if constexpr (!S::kQuant) {
          const int key = (lane & 7) + ((lane >> 4) << 3);
          const int half = (lane >> 3) & 1;
          uint32_t keep[2] = {kAll, kAll};
          if (edge)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              keep[x] = (read(n, 2 * c + 8 * x) ? 0xFFFFu : 0u) | (read(n, 2 * c + 1 + 8 * x) ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t af[4];
            ldsm4t(af, st32[n] + 16 * S::kRow + kv_place(S::kRow, key, 32 * i + 16 * half));
            if (edge) {
              af[0] &= keep[0];
              af[1] &= keep[0];
              af[2] &= keep[1];
              af[3] &= keep[1];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma<S::kBf>(o[nt][i], af, pf[n][nt][0], pf[n][nt][1]);
          }
        } else {
          // A register of two neighbouring columns of one value is used as it is expanded: the k index of the product
          // is (token, column parity), with P in the even places for the even columns (o[..][2t]) and in the odd ones
          // for the odd columns (o[..][2t + 1]). That doubles the mma count, of a pipe that is a fifth busy, and
          // saves a byte permutation for every two values of the busiest pipe.
          const int tok[4] = {2 * c, 8 + 2 * (c ^ 2), 2 * c + 1, 9 + 2 * (c ^ 2)};  // in pf[0], pf[0], pf[1], pf[1]
          uint32_t pe[NT][4], po[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              pe[nt][2 * k] = pf[n][nt][k] & 0xFFFFu;
              pe[nt][2 * k + 1] = pf[n][nt][k] >> 16;
              po[nt][2 * k] = pf[n][nt][k] << 16;
              po[nt][2 * k + 1] = pf[n][nt][k] & 0xFFFF0000u;
            }
#pragma unroll
          for (int p = 0; p < S::kValLoads; ++p) {  // one load of each of the four tokens
            uint32_t h[4][S::kValCodes / 2];
            if constexpr (FMT == MOE_KV_FP8) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t w[S::kValCodes / 4];
                if constexpr (S::kValCodes == 16)
                  *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(st[n] + v_at[p][k]);
                else
                  *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(st[n] + v_at[p][k]);
                if (edge && !read(n, tok[k]))
#pragma unroll
                  for (int y = 0; y < S::kValCodes / 4; ++y) w[y] = 0u;
#pragma unroll
                for (int y = 0; y < S::kValCodes / 4; ++y) {
                  h[k][2 * y] = e4m3x2_f16x2(w[y] & 0xFFFFu);
                  h[k][2 * y + 1] = e4m3x2_f16x2(w[y] >> 16);
                }
              }
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t w[S::kValCodes / 8];
                const uint8_t *src = st[n] + v_at[p][k];
                if constexpr (S::kValCodes == 32)
                  *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(src);
                else if constexpr (S::kValCodes == 16)
                  *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(src);
                else
                  w[0] = *reinterpret_cast<const uint32_t *>(src);
#pragma unroll
                for (int y = 0; y < S::kValCodes / 8; ++y) e2m1x8_f16(w[y], h[k] + 4 * y);
              }
#pragma unroll
              for (int b = 0; b < (S::kValCodes + 15) / 16; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k) {  // tokens tok[k] and tok[k + 2] are neighbours
                  uint32_t s2 = *reinterpret_cast<const uint16_t *>(st[n] + vs_at[k] + 8 * S::kValCodes * p + 16 * b);
                  if (edge) s2 &= (read(n, tok[k]) ? 0xFFu : 0u) | (read(n, tok[k + 2]) ? 0xFF00u : 0u);
                  s2 = e4m3x2_f16x2(s2);
                  const uint32_t f0 = __byte_perm(s2, 0, 0x1010), f1 = __byte_perm(s2, 0, 0x3232);
#pragma unroll
                  for (int y = 0; y < (S::kValCodes < 16 ? 4 : 8); ++y) {
                    h[k][8 * b + y] = hmul2(h[k][8 * b + y], f0);
                    h[k + 2][8 * b + y] = hmul2(h[k + 2][8 * b + y], f1);
                  }
                }
            }
#pragma unroll
            for (int t = 0; t < S::kValCodes / 4; ++t)  // rows r and r + 8: pairs 2t and 2t + 1
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t af[4] = {h[2 * k][2 * t], h[2 * k][2 * t + 1], h[2 * k + 1][2 * t],
                                        h[2 * k + 1][2 * t + 1]};
                const int at = 2 * (p * (S::kValCodes / 4) + t);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma<false>(o[nt][at], af, pe[nt][2 * k], pe[nt][2 * k + 1]);
                  mma<false>(o[nt][at + 1], af, po[nt][2 * k], po[nt][2 * k + 1]);
                }
              }
          }
        }
        }
      }
      __syncwarp();
      done += min(S::kTile, cu.end - cu.rec);
      while (!dead && is_more && issued - done <= S::kStages - S::kGroup) issue();
    }

    // ---- the maxima as they are, and the sum of p over the lanes that share a head
    float m[NT][2], mw[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[nt][x] += __shfl_xor_sync(kAll, l[nt][x], sh);
        m[nt][x] = thr[nt][x] == -INFINITY && l[nt][x] == 0.f ? -INFINITY : ref[nt][x];
        mw[nt][x] = !S::kQuant ? m[nt][x] : thrw[nt][x] == -INFINITY && l[nt][x] == 0.f ? -INFINITY : refw[nt][x];
      }
    if (begins && ends) {  // all of it: written from here
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int h = 8 * nt + 2 * c + x;
          if (h >= nh) continue;
          const bool none = l[nt][x] == 0.f;  // l is at least 2^-kSlack otherwise
          float g = none ? 0.f : ex2(mw[nt][x] - m[nt][x]) / l[nt][x];
          const float lse2 = with_sink(a, h0 + h, none ? -INFINITY : m[nt][x] + log2f(l[nt][x]), g);
          uint16_t *po = static_cast<uint16_t *>(a.out) + cu.b * a.osb + (int64_t)(h0 + h) * a.osh;
          auto pack = [&](float v0, float v1) {
            return a.q_type == MOE_BF16 ? pack2<true>(v0 * g, v1 * g) : pack2<false>(v0 * g, v1 * g);
          };
#pragma unroll
          for (int i = 0; i < D / 16; i += 2) {
            const float(&e)[4] = o[nt][i];
            const float(&f)[4] = o[nt][i + 1];
            if (S::kQuant) {
              *reinterpret_cast<uint2 *>(po + S::val_col(r, 2 * i)) =
                  make_uint2(pack(e[x], f[x]), pack(e[x + 2], f[x + 2]));
            } else {
              const uint32_t u = pack(e[x], e[x + 2]), v = pack(f[x], f[x + 2]);
              po[16 * i + r] = (uint16_t)u;
              po[16 * i + 8 + r] = (uint16_t)(u >> 16);
              po[16 * i + 16 + r] = (uint16_t)v;
              po[16 * i + 24 + r] = (uint16_t)(v >> 16);
            }
          }
          if (a.lse && r == 0) a.lse[(int64_t)cu.b * a.heads + h0 + h] = lse2 / kLog2e;
        }
    } else {
      // partial: one that began before this warp's range in the first place, else (the range's last) in the ring
      const int second = begins ? 1 : 0;
      float *po = second ? reinterpret_cast<float *>(ring) : join_o + warp * S::kHeads * S::kLdo;
      float *ml = join_ml + (2 * warp + second) * S::kHeads * 3;
      if (lane == 0) {
        seg_of[warp][second] = cu.b * HB + cu.hb;
        if (!second) ends0[warp] = ends;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int h = 8 * nt + 2 * c + x;
          if (r == 0) {
            ml[3 * h] = m[nt][x];
            ml[3 * h + 1] = l[nt][x];
            ml[3 * h + 2] = mw[nt][x];
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int d = S::kQuant ? S::val_col(r, 2 * (i & ~1)) + (i & 1) : 16 * i + r;
            po[h * S::kLdo + d] = o[nt][i][x];
            po[h * S::kLdo + d + (S::kQuant ? 2 : 8)] = o[nt][i][x + 2];
          }
        }
    }
  }
  // a wait that ran out leaves copies in flight: wait for them, with the same limit
  if (dead)
    for (int i = dead_at; i < issued; ++i) mbar_wait(bar0 + 8 * (i % S::kStages), (i / S::kStages) & 1);

  // ---------------- what the warps share: chains of a partial and the first partials of the warps after it
  __syncthreads();
  for (int lead = -1; lead < kW; ++lead) {
    const int w0 = max(lead, 0), second = lead >= 0;
    const int seg = seg_of[w0][second];
    if (seg < 0) continue;
    int last = w0;  // warp of the chain's last part
    bool ended = !second && ends0[0];
    while (!ended && last + 1 < kW && seg_of[last + 1][0] == seg) {
      ++last;
      ended = ends0[last];
    }
    const int b = seg / HB, hb = seg % HB;
    const int h0 = hb / a.GB * a.G + hb % a.GB * S::kHeads, nh = min(S::kHeads, a.G - hb % a.GB * S::kHeads);
    const bool all = second && ended;
    const int pslot = 2 * blockIdx.x + second;
    for (int at = tid; at < nh * (D / 4); at += kW * 32) {
      const int h = at / (D / 4), d = at % (D / 4) * 4;
      float M = -INFINITY, MW = -INFINITY;
      for (int w = w0; w <= last; ++w) {
        const float *ml = join_ml + ((2 * w + (w == w0 ? second : 0)) * S::kHeads + h) * 3;
        M = fmaxf(M, ml[0]);
        MW = fmaxf(MW, ml[2]);
      }
      float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
      const float Mr = M == -INFINITY ? 0.f : M, MWr = MW == -INFINITY ? 0.f : MW;
      for (int w = w0; w <= last; ++w) {
        const bool in_ring = w == w0 && second;
        const float *ml = join_ml + ((2 * w + in_ring) * S::kHeads + h) * 3;
        const float *po = in_ring ? reinterpret_cast<const float *>(smem + w * S::kStages * S::kStage)
                                  : join_o + w * S::kHeads * S::kLdo;
        L += ml[1] * ex2(ml[0] - Mr);
        const float f = ex2(ml[2] - MWr);
        const float4 v = *reinterpret_cast<const float4 *>(po + h * S::kLdo + d);
        acc[0] += v.x * f;
        acc[1] += v.y * f;
        acc[2] += v.z * f;
        acc[3] += v.w * f;
      }
      float lse2 = L == 0.f ? -INFINITY : Mr + log2f(L);
      float g = L == 0.f ? 0.f : ex2(MWr - Mr) / L;
      if (all) {
        lse2 = with_sink(a, h0 + h, lse2, g);
        uint2 pk;
        if (a.q_type == MOE_BF16)
          pk = make_uint2(pack2<true>(acc[0] * g, acc[1] * g), pack2<true>(acc[2] * g, acc[3] * g));
        else
          pk = make_uint2(pack2<false>(acc[0] * g, acc[1] * g), pack2<false>(acc[2] * g, acc[3] * g));
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + b * a.osb + (int64_t)(h0 + h) * a.osh + d) = pk;
        if (a.lse && d == 0) a.lse[(int64_t)b * a.heads + h0 + h] = lse2 / kLog2e;
      } else if (a.mode == kClustered) {  // over the rings, which are drained
        *reinterpret_cast<float4 *>(smem + (h * D + d) * 4) =
            make_float4(acc[0] * g, acc[1] * g, acc[2] * g, acc[3] * g);
        if (d == 0) share_lse[h] = lse2;
      } else {
        *reinterpret_cast<float4 *>(a.part_o + ((int64_t)pslot * S::kHeads + h) * D + d) =
            make_float4(acc[0] * g, acc[1] * g, acc[2] * g, acc[3] * g);
        if (d == 0) a.part_lse[pslot * S::kHeads + h] = lse2;
      }
    }
  }
  if (a.mode != kClustered) return;

  // ---------------- the cluster's CTAs joined, 4 columns of a head a thread
  if (cta0 >= cta1 && tid < S::kHeads) share_lse[tid] = -INFINITY;
  cluster_sync();
  const int seg = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster, b = seg / HB, hb = seg % HB;
  const int h0 = hb / a.GB * a.G + hb % a.GB * S::kHeads, nh = min(S::kHeads, a.G - hb % a.GB * S::kHeads);
  const uint32_t o32 = smem_u32(smem), lse32 = smem_u32(share_lse);
  for (int at = rank * (kW * 32) + tid; at < nh * (D / 4); at += a.cluster * kW * 32) {
    const int h = at / (D / 4), d = at % (D / 4) * 4;
    float w[kCluster], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < kCluster; ++k) {
      w[k] = k < a.cluster ? ld_cluster(at_rank(lse32 + 4 * h, k)) : -INFINITY;
      top = fmaxf(top, w[k]);
    }
    const float ref = top == -INFINITY ? 0.f : top;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kCluster; ++k) {
      if (w[k] == -INFINITY) continue;  // it has nothing
      w[k] = ex2(w[k] - ref);
      sum += w[k];
      const float4 v = ld_cluster4(at_rank(o32 + (h * D + d) * 4, k));
      acc[0] += w[k] * v.x;
      acc[1] += w[k] * v.y;
      acc[2] += w[k] * v.z;
      acc[3] += w[k] * v.w;
    }
    float g = sum == 0.f ? 0.f : 1.f / sum;
    const float lse2 = with_sink(a, h0 + h, sum == 0.f ? -INFINITY : ref + log2f(sum), g);
    const uint2 pk = a.q_type == MOE_BF16
                         ? make_uint2(pack2<true>(acc[0] * g, acc[1] * g), pack2<true>(acc[2] * g, acc[3] * g))
                         : make_uint2(pack2<false>(acc[0] * g, acc[1] * g), pack2<false>(acc[2] * g, acc[3] * g));
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + b * a.osb + (int64_t)(h0 + h) * a.osh + d) = pk;
    if (a.lse && d == 0) a.lse[(int64_t)b * a.heads + h0 + h] = lse2 / kLog2e;
  }
  cluster_sync();  // the others may still be reading here
}

// Joins the partial outputs of one (sequence, kv head, block of heads), if
// there are several: grid (B * HB, slices of the heads). A warp a head turns
// the partials' log-sums into weights; then a thread takes 4 columns of a head,
// and where there are fewer of those than threads, every so many-th partial.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs a) {
  constexpr int kHeads = 8 * NT, kWarps = kJoinThreads / 32, kCols = D / 4;
  extern __shared__ float wts[];  // [heads of this slice][parts]
  __shared__ float4 acc_s[kJoinThreads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int HB = a.kv_heads * a.GB;
  const int b = blockIdx.x / HB, hb = blockIdx.x % HB;
  const int nh = min(kHeads, a.G - hb % a.GB * kHeads), h0 = hb / a.GB * a.G + hb % a.GB * kHeads;
  // heads of this slice
  const int each = (nh + gridDim.y - 1) / gridDim.y, from = blockIdx.y * each, heads = min(each, nh - from);
  pdl_wait();
  pdl_trigger();
  const int64_t per = *a.per;
  const int s0 = a.starts[b], n = a.starts[b + 1] - s0;
  const int64_t first = ((int64_t)s0 + (int64_t)b * kLead) * HB + (int64_t)hb * (n + kLead) + kLead, last = first + n - 1;
  const int c0 = (int)(first / per), c1 = (int)(last / per);
  if (c0 == c1 || heads <= 0) return;
  const int parts = c1 - c0 + 1;
  // it begins in CTA c0, and in the others it began before
  auto slot = [&](int i) { return i == 0 ? 2 * c0 + 1 : 2 * (c0 + i); };
  const int items = heads * kCols, groups = max(1, kJoinThreads / items);
  // the first partials of the first round are on their way while the weights are made
  constexpr int kAhead = 8;
  float4 ahead[kAhead];
  const int at0 = groups > 1 ? tid % items : tid, grp = groups > 1 ? tid / items : 0;
  const bool live0 = at0 < items && grp < groups;
  const float *src0 = a.part_o + (int64_t)(from + at0 / kCols) * D + at0 % kCols * 4;
#pragma unroll
  for (int x = 0; x < kAhead; ++x) {
    const int i = grp + x * groups;
    ahead[x] = live0 && i < parts ? *reinterpret_cast<const float4 *>(src0 + (int64_t)slot(i) * (kHeads * D))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int k = warp; k < heads; k += kWarps) {
    const int h = from + k;
    float top = -INFINITY;
    bool bad = false;
    for (int i = lane; i < parts; i += 32) {
      const float v = a.part_lse[slot(i) * kHeads + h];
      wts[k * parts + i] = v;
      top = fmaxf(top, v);
      bad = bad || v != v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int i = lane; i < parts; i += 32) sum += ex2(wts[k * parts + i] - ref);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    float lse2 = sum == 0.f ? -INFINITY : ref + log2f(sum);
    float g = sum == 0.f ? 0.f : 1.f / sum;
    if (__any_sync(kAll, bad)) g = lse2 = __int_as_float(0x7fc00000);
    lse2 = with_sink(a, h0 + h, lse2, g);
    for (int i = lane; i < parts; i += 32) wts[k * parts + i] = g * ex2(wts[k * parts + i] - ref);
    if (a.lse && lane == 0) a.lse[(int64_t)b * a.heads + h0 + h] = lse2 / kLog2e;
  }
  __syncthreads();
  for (int base = 0; base < items; base += kJoinThreads) {
    const int at = at0 + base;
    const bool live = at < items && grp < groups;
    const int k = at / kCols, d = at % kCols * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto put = [&](int i, float4 v) {
      const float w = wts[k * parts + i];
      acc.x += w * v.x;
      acc.y += w * v.y;
      acc.z += w * v.z;
      acc.w += w * v.w;
    };
    if (live) {
      const float *src = a.part_o + (int64_t)(from + k) * D + d;
      int i = grp;
      if (base == 0) {
#pragma unroll
        for (int x = 0; x < kAhead; ++x, i += groups)
          if (i < parts) put(i, ahead[x]);
      }
#pragma unroll 4
      for (; i < parts; i += groups) put(i, *reinterpret_cast<const float4 *>(src + (int64_t)slot(i) * (kHeads * D)));
    }
    if (groups > 1) {
      acc_s[tid] = acc;
      __syncthreads();
      if (live && grp == 0)
        for (int i = 1; i < groups; ++i) {
          const float4 v = acc_s[i * items + at];
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
        }
    }
    if (live && grp == 0) {
      const uint2 pk = a.q_type == MOE_BF16 ? make_uint2(pack2<true>(acc.x, acc.y), pack2<true>(acc.z, acc.w))
                                            : make_uint2(pack2<false>(acc.x, acc.y), pack2<false>(acc.z, acc.w));
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + b * a.osb + (int64_t)(h0 + from + k) * a.osh + d) = pk;
    }
  }
}

// column tiles of 8 heads a CTA takes: the accumulators of 16 heads at D = 256 would not fit registers
int tiles_of(int G, int D) { return G > 8 && D <= 128 ? 2 : 1; }

template <int FMT, int D, int NT>
moe_status_t go(AttnArgs &a, cudaStream_t stream, int *launches) {
  using S = Shape<FMT, D, NT>;
  // shared memory in steps of 1 KB of sequence starts, so that few sizes occur
  const int step = a.B / 256, smem = S::kFixed + (step + 1) * 1024 + 4;
  static PerDevice occs[kMaxB / 256 + 1];  // resident CTAs an SM by step
  auto kern = attn_kernel<FMT, D, NT>;
  const int sms = sm_count();
  const int occ = occs[step].get([&] {
    int n = 0;
    const bool ok = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         S::kFixed + (kMaxB / 256 + 1) * 1024 + 4) == cudaSuccess &&
                    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kW * 32, smem) == cudaSuccess;
    return ok ? n : 0;
  });
  if (occ < 1) return MOE_ERR_CUDA;
  // the most records that a (sequence, head) can have
  const int64_t tokens = (int64_t)a.max_pages * a.page, groups = (int64_t)a.B * a.kv_heads * a.GB;
  const int64_t most = a.window > 0 && a.window < tokens ? (a.window + 14) / 16 + 1 : std::max<int64_t>(tokens / 16, 1);
  // A CTA or a cluster for each (sequence, head), the largest whose CTAs fit two an SM and have a record for every warp,
  // as long as no warp gets more than 8 records: so much may be lost to unequal lengths. us, this way / by even shares and
  // the second kernel:
  //   clusters of 8: 777 tokens in FP8 on 8 heads of 128 8.2 / 10.9; NVFP4 of 64 on 8 heads, 2048 tokens 8.9 / 11.0, 4096
  //     11.0 / 11.6 (8192, 16 records a warp, 15.0 / 13.0)
  //   of 4 and 2: 8 x 2048 tokens in BF16 of 128 17.9 / 21.3; unequal lengths: 16 of up to 1024 in BF16 12.3 / 11.0, 8 of
  //     up to 2048 in FP8 11.3 / 12.3
  //   single CTAs: 48 sequences with a window of 128 on 4 heads 6.8 / 11.6
  //   whole ones: 256 sequences of 64 tokens on 8 heads 11.6 / 21.9
  const int64_t fit = std::min(sms * occ, kMaxCtas);
  int c = kCluster;
  while (c > 1 && (groups * c > 2 * sms || most < c * kW)) c >>= 1;
  a.mode = most > 8 * kW * c ? kStream : c > 1 ? kClustered : groups <= fit ? kSingle : kWhole;
  a.cluster = c;
  a.ctas = a.mode >= kSingle  ? (int)groups * c
           : a.mode == kWhole ? (int)fit
                              : (int)std::min<int64_t>(fit, (groups * (most + kLead) + 2 * kW - 1) / (2 * kW));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(kW * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.mode == kClustered ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return MOE_ERR_CUDA;
  if (launches) ++*launches;
  if (a.ctas > 1 && a.mode == kStream) {
    // few groups: their heads apart, so that more SMs share the work
    const int heads = std::min(a.G, S::kHeads);
    const int slices = (int)std::min<int64_t>(heads, std::max<int64_t>(1, 2 * sms / groups));
    const int each = (heads + slices - 1) / slices;
    const int wts = each * a.ctas * 4;  // at most 16 heads of all CTAs: 40 KB
    if (launch_pdl(attn_join_kernel<D, NT>, dim3((unsigned)groups, slices), dim3(kJoinThreads), wts, stream, a) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    if (launches) ++*launches;
  }
  return MOE_OK;
}

template <int FMT>
moe_status_t by_dim(AttnArgs &a, int D, cudaStream_t stream, int *launches) {
  const int nt = tiles_of(a.G, D);
  if (D == 64) return nt == 1 ? go<FMT, 64, 1>(a, stream, launches) : go<FMT, 64, 2>(a, stream, launches);
  if (D == 128) return nt == 1 ? go<FMT, 128, 1>(a, stream, launches) : go<FMT, 128, 2>(a, stream, launches);
  return go<FMT, 256, 1>(a, stream, launches);
}

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t attn_workspace(int G, int D) {
  const size_t heads = 8 * (size_t)tiles_of(G, D);
  return up256(MOE_STATUS_BYTES) + up256((kMaxB + 3) * 4) + up256(2 * kMaxCtas * heads * 4) +
         up256(2 * kMaxCtas * heads * D * 4);
}

moe_status_t launch_attn_decode(const void *q, int q_type, int64_t qsb, int64_t qsh, const moe_kv_cache_t &c,
                                const int32_t *table, int64_t ts, int max_pages, const int32_t *lens, int B,
                                int heads, float scale, int window, const float *sinks, void *out, int64_t osb,
                                int64_t osh, float *lse, void *ws, cudaStream_t stream, int *launches) {
  if (B == 0) return MOE_OK;
  if (B > kMaxB) return MOE_ERR_UNSUPPORTED;
  AttnArgs a = {};
  a.q = q;
  a.data = static_cast<const uint8_t *>(c.data);
  a.table = table;
  a.lens = lens;
  a.sinks = sinks;
  a.out = out;
  a.lse = lse;
  a.qsb = qsb;
  a.qsh = qsh;
  a.osb = osb;
  a.osh = osh;
  a.ts = ts;
  a.q_type = q_type;
  a.B = B;
  a.heads = heads;
  a.kv_heads = c.kv_heads;
  a.G = heads / c.kv_heads;
  const int H = 8 * tiles_of(a.G, c.head_dim);
  a.GB = (a.G + H - 1) / H;
  a.window = window;
  a.page = c.page_size;
  a.pages = c.num_pages;
  a.max_pages = max_pages;
  a.scale = scale * kLog2e;
  uint8_t *w = static_cast<uint8_t *>(ws);
  a.status = reinterpret_cast<unsigned int *>(w);
  w += up256(MOE_STATUS_BYTES);
  a.per = reinterpret_cast<int64_t *>(w);
  a.starts = reinterpret_cast<int *>(w + 8);
  w += up256((kMaxB + 3) * 4);
  a.part_lse = reinterpret_cast<float *>(w);
  w += up256(2 * kMaxCtas * (size_t)H * 4);
  a.part_o = reinterpret_cast<float *>(w);
  switch (c.fmt) {
    case MOE_KV_BF16: return by_dim<MOE_KV_BF16>(a, c.head_dim, stream, launches);
    case MOE_KV_FP16: return by_dim<MOE_KV_FP16>(a, c.head_dim, stream, launches);
    case MOE_KV_FP8: return by_dim<MOE_KV_FP8>(a, c.head_dim, stream, launches);
    default: return by_dim<MOE_KV_NVFP4>(a, c.head_dim, stream, launches);
  }
}

}  // namespace moe4
