// The plan of a batch: pages given and taken back, block tables, and where each
// new token goes.
//
// Every CTA of one cluster reads all B sequences and sums their tokens and pages
// (a scan of 64-bit pairs, 4 sequences a thread); the work that the sums lay out
// is then shared by the cluster: token rows and fresh pages by number, each found
// by a binary search of the sums in shared memory. All inputs are read before the
// cluster's first barrier and nothing that was read is written before it, so that
// outputs may be the inputs; the pages of ended sequences are on the stack before
// the second, after which pages are taken.
//
// Bound by latency: 16 bytes a sequence and 12 a token. One launch, three rounds
// of memory (lengths, pages, rows).
#include "common.cuh"
#include "device.cuh"
#include "kernels.h"

namespace moe4 {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32, kMaxB = 4096, kEach = kMaxB / kThreads, kMaxCluster = 8;
constexpr unsigned kAll = 0xffffffffu;

struct PlanArgs {
  const int32_t *new_lens, *seq_lens, *free_count;
  int32_t *table, *free_pages, *lens_out, *count_out, *offsets, *slots, *positions, *seq_ids;
  unsigned int *status;
  int64_t ts;
  int B, T, page, num_pages, max_pages;
};

// What a sequence adds to the sums: tokens, pages needed, pages given back.
struct Sums {
  int64_t tokens, need, back;
};

__device__ __forceinline__ Sums add(const Sums &a, const Sums &b) { return {a.tokens + b.tokens, a.need + b.need, a.back + b.back}; }

__device__ __forceinline__ Sums shift_up(const Sums &s, int o) {
  return {__shfl_up_sync(kAll, s.tokens, o), __shfl_up_sync(kAll, s.need, o), __shfl_up_sync(kAll, s.back, o)};
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The first of n rising values above x (n where there is none).
__device__ __forceinline__ int upper(const int *v, int n, int x) {
  int lo = 0;
  while (n > 0) {
    const int half = n >> 1;
    if (v[lo + half] <= x)
      lo += half + 1, n -= half + 1;
    else
      n = half;
  }
  return lo;
}

__device__ __forceinline__ int clamp31(int64_t v) { return (int)min(v, (int64_t)INT32_MAX); }

__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs a) {
  // per sequence: end of its tokens, pages before its own on the stack's way down, length (-1: not served)
  extern __shared__ int shared[];
  int *ends = shared, *before = ends + a.B, *lens = before + a.B;
  __shared__ Sums warp_sums[kWarps];
  __shared__ int given;  // pages: the served that need some come before all others that do
  if (threadIdx.x == 0) given = 0;
  pdl_trigger();
  pdl_wait();
  uint32_t ranks, rank;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool first = rank == 0;
  const int64_t cap = (int64_t)a.max_pages * a.page;

  const int each = (a.B + kThreads - 1) / kThreads;  // sequences of a thread, side by side
  int L[kEach], n[kEach];
  bool fits[kEach];
  Sums own = {0, 0, 0}, mine[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = tid * each + i;
    const bool in = i < each && b < a.B;
    L[i] = in ? a.seq_lens[b] : 0;
    n[i] = in ? a.new_lens[b] : 0;
  }
  int count = *a.free_count;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const bool valid = L[i] >= 0 && L[i] <= cap;
    const int held = valid ? (int)(((int64_t)L[i] + a.page - 1) / a.page) : 0;
    fits[i] = valid && n[i] > 0 && (int64_t)L[i] + n[i] <= cap;
    mine[i].tokens = max(n[i], 0);
    mine[i].need = fits[i] ? ((int64_t)L[i] + n[i] + a.page - 1) / a.page - held : 0;
    mine[i].back = valid && n[i] < 0 ? held : 0;
    own = add(own, mine[i]);
    if (!valid && first) raise_status(a.status, MOE_ERR_BAD_INDEX);
  }
  // the sums before this thread's sequences, and of all
  Sums up = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums v = shift_up(up, o);
    if (lane >= o) up = add(up, v);
  }
  if (lane == 31) warp_sums[warp] = up;
  __syncthreads();
  if (warp == 0) {
    Sums w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums v = shift_up(w, o);
      if (lane >= o) w = add(w, v);
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const Sums all = warp_sums[kWarps - 1];
  Sums at = warp ? warp_sums[warp - 1] : Sums{0, 0, 0};
  at = {at.tokens + up.tokens - own.tokens, at.need + up.need - own.need, at.back + up.back - own.back};

  if (count < 0 || count > a.num_pages) {
    if (first && tid == 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
    count = max(0, min(count, a.num_pages));
  }
  if (count + all.back > a.num_pages && first && tid == 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
  const int top = (int)min(count + all.back, (int64_t)a.num_pages);
  cluster_sync();  // all has been read

  // who is served, and the ended sequences' pages onto the stack
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = tid * each + i;
    if (i < each && b < a.B) {
      const int64_t end = at.tokens + mine[i].tokens;
      const bool served = fits[i] && (mine[i].need == 0 || at.need + mine[i].need <= top) && end <= a.T;
      ends[b] = clamp31(end);
      before[b] = clamp31(at.need);
      lens[b] = served ? L[i] : -1;
      if (served && mine[i].need) atomicMax(&given, (int)(at.need + mine[i].need));
      if (first) {
        if (n[i] > 0 && L[i] >= 0 && L[i] <= cap && !served) raise_status(a.status, MOE_ERR_CAPACITY);
        a.lens_out[b] = served ? L[i] + n[i] : n[i] < 0 && L[i] >= 0 && L[i] <= cap ? 0 : L[i];
        if (a.offsets) a.offsets[b + 1] = clamp31(end);
      }
    }
    // a warp the pages of one lane's sequence after the other's
    for (unsigned who = __ballot_sync(kAll, mine[i].back > 0); who; who &= who - 1) {
      const int from = __ffs(who) - 1;
      const int64_t to = count + __shfl_sync(kAll, at.back, from), pages = __shfl_sync(kAll, mine[i].back, from);
      const int32_t *row = a.table + (int64_t)__shfl_sync(kAll, b, from) * a.ts;
      for (int64_t j = (int64_t)rank * 32 + lane; j < pages; j += ranks * 32)
        if (to + j < a.num_pages) a.free_pages[to + j] = row[j];
    }
    at = add(at, mine[i]);
  }
  __syncthreads();
  cluster_sync();  // the stack is whole

  const int64_t step = (int64_t)ranks * kThreads;
  auto fresh = [&](int j) {  // page number j of those that are given, -1 for one that is none
    const int p = a.free_pages[top - 1 - j];
    return p >= 0 && p < a.num_pages ? p : -1;
  };
  for (int64_t j = (int64_t)rank * kThreads + tid; j < given; j += step) {
    const int b = upper(before, a.B, (int)j) - 1;  // the last that no more than j pages lie before: it needs some
    const int held = (lens[b] + a.page - 1) / a.page, p = fresh((int)j);
    a.table[b * a.ts + held + ((int)j - before[b])] = p;
    if (p < 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
  }
  if (first && tid == 0) {
    *a.count_out = top - given;
    if (a.offsets) a.offsets[0] = 0;
  }
  // rows
  const int64_t tokens = all.tokens;
  for (int64_t t = (int64_t)rank * kThreads + tid; t < a.T; t += step) {
    int slot = -1, pos = 0, b = -1;
    if (t < tokens) {
      b = upper(ends, a.B, (int)t);
      if (lens[b] >= 0) {
        const int start = b ? ends[b - 1] : 0, held = (lens[b] + a.page - 1) / a.page;
        pos = lens[b] + ((int)t - start);
        const int pg = pos / a.page;
        int p;
        if (pg < held) {
          p = a.table[b * a.ts + pg];
          if (p < 0 || p >= a.num_pages) {
            raise_status(a.status, MOE_ERR_BAD_INDEX);
            p = -1;
          }
        } else {
          p = fresh(before[b] + pg - held);
        }
        slot = p < 0 ? -1 : p * a.page + (pos - pg * a.page);
      }
    }
    a.slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
    if (a.seq_ids) a.seq_ids[t] = b;
  }
}

}  // namespace

moe_status_t launch_batch_plan(const int32_t *new_lens, const int32_t *seq_lens, int B, int page, int num_pages,
                               int32_t *table, int64_t ts, int max_pages, int32_t *free_pages, const int32_t *free_count,
                               int32_t *lens_out, int32_t *count_out, int32_t *offsets, int T, int32_t *slots,
                               int32_t *positions, int32_t *seq_ids, unsigned int *status, cudaStream_t stream,
                               int *launches) {
  const PlanArgs a = {new_lens, seq_lens, free_count, table, free_pages, lens_out, count_out, offsets, slots,
                      positions, seq_ids, status, ts, B, T, page, num_pages, max_pages};
  static PerDevice configured;
  const int set = configured.get([] {
    return cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 12 * kMaxB) == cudaSuccess ? 1 : 0;
  });
  if (set < 1) return MOE_ERR_CUDA;
  // a CTA for every 2048 rows: two a thread
  int ctas = 1;
  while (ctas < kMaxCluster && T > 2048 * ctas) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 12 * B;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (launches) ++*launches;
  return cudaLaunchKernelEx(&cfg, plan_kernel, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe4
