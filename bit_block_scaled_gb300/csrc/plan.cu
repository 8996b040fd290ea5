// The plan of a batch: pages given and taken back, block tables, and where each
// new token goes.
//
// Every CTA of one cluster reads all B sequences and sums their tokens and pages
// (a scan, up to 4 sequences a thread, in 32 bits that saturate); the work that
// the sums lay out is then shared by the cluster: token rows and fresh pages by
// number, each found by a binary search of the sums in shared memory. All inputs are read before the first barrier and nothing that was read
// is written before it, so that outputs may be the inputs; the pages of ended
// sequences are on the stack before the second, after which pages are taken. The
// barriers are the cluster's only where there is something to keep apart.
//
// Bound by latency: 16 bytes a sequence and 12 a token. One launch, three rounds
// of memory (lengths, pages, rows): 64 sequences of one token each 2.5 us, 500
// with 65536 tokens 6.5, 4096 of one token 7.3.
#include "checks.h"
#include "common.cuh"
#include "device.cuh"
#include "kernels.h"

namespace moe4 {

namespace {

constexpr int kMaxThreads = 1024, kWarps = kMaxThreads / 32, kMaxB = 4096, kEach = kMaxB / kMaxThreads, kMaxCluster = 16;
constexpr unsigned kAll = 0xffffffffu;

// Division of numbers below 2^31: q = x m / 2^(31 + l), l = ceil(log2 d) and m = ceil(2^(31 + l) / d) (Granlund and
// Montgomery, "Division by invariant integers using multiplication").
struct Divisor {
  uint32_t m;
  int shift;
  explicit Divisor(uint32_t d) {  // d > 1
    int l = 1;
    while (((uint32_t)1 << l) < d) ++l;
    m = (uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d);
    shift = l - 1;
  }
  __device__ __forceinline__ int div(int x) const { return (int)(__umulhi((uint32_t)x, m) >> shift); }
};

struct PlanArgs {
  const int32_t *new_lens, *seq_lens, *free_count;
  int32_t *table, *free_pages, *lens_out, *count_out, *offsets, *slots, *positions, *seq_ids;
  unsigned int *status;
  int64_t ts;
  int B, T, rows_each, page, num_pages, max_pages, log_b, wide;  // 2^log_b > B; rows' outputs are 16-byte aligned
  Divisor by_page, by_rows;
};

// What a sequence adds to the sums: tokens, pages needed, pages given back. Sums stay at 2^31 - 1 once they are there.
struct Sums {
  int tokens, need, back;
};

__device__ __forceinline__ int add31(int a, int b) { return (int)min((uint32_t)a + (uint32_t)b, 0x7fffffffu); }
__device__ __forceinline__ Sums add(const Sums &a, const Sums &b) {
  return {add31(a.tokens, b.tokens), add31(a.need, b.need), add31(a.back, b.back)};
}
__device__ __forceinline__ Sums shift_up(const Sums &s, int o) {
  return {__shfl_up_sync(kAll, s.tokens, o), __shfl_up_sync(kAll, s.need, o), __shfl_up_sync(kAll, s.back, o)};
}
// Sums of the lanes up to this one.
__device__ __forceinline__ Sums scan(Sums s, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums v = shift_up(s, o);
    if (lane >= o) s = add(s, v);
  }
  return s;
}
// The lanes before this one's, of what scan() gave.
__device__ __forceinline__ Sums exclusive(const Sums &s, int lane) {
  const Sums v = shift_up(s, 1);
  return lane ? v : Sums{0, 0, 0};
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The first of the n rising values above x (n where there is none); 2^log_n > n.
__device__ __forceinline__ int upper(const int *v, int n, int log_n, int x) {
  int at = 0;
  for (int s = 1 << (log_n - 1); s; s >>= 1)
    if (at + s <= n && v[at + s - 1] <= x) at += s;
  return at;
}

// R rows of a thread side by side: one search finds the first's sequence, the next ones' is it or close behind, and a page
// is looked up once. (Four searches instead: 500 sequences with 65536 rows 8.5 us against 7.2.)
template <int R>
__device__ __forceinline__ void put_rows(const PlanArgs &a, const int *ends, const int *before, const int *lens, int top,
                                         int thread, int step) {
  for (int64_t t0 = (int64_t)thread * R; t0 < a.T; t0 += (int64_t)step * R) {
    int b[R], pos[R], slot[R];
    const int32_t *from[R];  // the page's place, or none: no page, or the row before's
    int seq = upper(ends, a.B, a.log_b, (int)t0), last = -1, last_seq = -1;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int t = (int)t0 + i;
      while (seq < a.B && ends[seq] <= t) ++seq;
      b[i] = seq;
      pos[i] = 0;
      from[i] = nullptr;
      slot[i] = -1;  // for now the place in the page
      const int len = seq < a.B ? lens[seq] : -1;
      if (len >= 0) {
        pos[i] = len + (t - (seq ? ends[seq - 1] : 0));
        const int pg = a.by_page.div(pos[i]);
        slot[i] = pos[i] - pg * a.page;
        if (pg != last || seq != last_seq) {
          const int held = a.by_page.div(len + a.page - 1);
          from[i] = pg < held ? a.table + seq * a.ts + pg : a.free_pages + (top - 1 - (before[seq] + pg - held));
          last = pg, last_seq = seq;
        }
      }
    }
    int p[R];
#pragma unroll
    for (int i = 0; i < R; ++i) p[i] = from[i] ? *from[i] : -1;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (from[i] && (p[i] < 0 || p[i] >= a.num_pages)) {
        if (t0 + i < a.T) raise_status(a.status, MOE_ERR_BAD_INDEX);
        p[i] = -1;
      }
      if (i > 0 && !from[i] && slot[i] >= 0) p[i] = p[i - 1];
      slot[i] = slot[i] < 0 || p[i] < 0 ? -1 : p[i] * a.page + slot[i];
      if (b[i] == a.B) b[i] = -1;
    }
    if (R == 4 && a.wide && t0 + 4 <= a.T) {
      *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[R / 4], slot[R / 2], slot[R - 1]);
      if (a.positions) *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[R / 4], pos[R / 2], pos[R - 1]);
      if (a.seq_ids) *reinterpret_cast<int4 *>(a.seq_ids + t0) = make_int4(b[0], b[R / 4], b[R / 2], b[R - 1]);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (t0 + i < a.T) {
          a.slots[t0 + i] = slot[i];
          if (a.positions) a.positions[t0 + i] = pos[i];
          if (a.seq_ids) a.seq_ids[t0 + i] = b[i];
        }
    }
  }
}

// Sequence b's rows are those from b * rows_each on.
__device__ __forceinline__ void put_fixed_rows(const PlanArgs &a, const int *tokens, const int *before, const int *lens, int top,
                                               int thread, int step) {
  for (int t = thread; t < a.T; t += step) {
    int b = a.rows_each > 1 ? a.by_rows.div(t) : t, pos = 0, slot = -1;
    const int i = t - b * a.rows_each;
    if (b >= a.B || i >= tokens[b]) {
      b = -1;
    } else if (lens[b] >= 0) {
      pos = lens[b] + i;
      const int pg = a.by_page.div(pos), held = a.by_page.div(lens[b] + a.page - 1);
      const int p = pg < held ? a.table[b * a.ts + pg] : a.free_pages[top - 1 - (before[b] + pg - held)];
      if (p < 0 || p >= a.num_pages)
        raise_status(a.status, MOE_ERR_BAD_INDEX);
      else
        slot = p * a.page + (pos - pg * a.page);
    }
    a.slots[t] = slot;
    if (a.positions) a.positions[t] = pos;
    if (a.seq_ids) a.seq_ids[t] = b;
  }
}

__global__ void __launch_bounds__(kMaxThreads) plan_kernel(const PlanArgs a) {
  // per sequence: end of its tokens (their number where rows are fixed), pages before its own on the stack's way down, length (-1: not served)
  extern __shared__ int shared[];
  int *ends = shared, *before = ends + a.B, *lens = before + a.B;
  __shared__ Sums warp_sums[kWarps];
  __shared__ int given;  // pages: the served that need some come before all others that do
  pdl_wait();
  pdl_trigger();
  uint32_t ranks, rank;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int tid = threadIdx.x, threads = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const bool first = rank == 0;
  const int cap = a.max_pages * a.page;
  // the cluster where what follows may write what others have yet to read, or read what they write; else the CTA
  auto everyone = [&](bool all_ranks) {
    if (ranks > 1 && all_ranks)
      cluster_sync();
    else
      __syncthreads();
  };
  auto pages_of = [&](int tokens) { return a.by_page.div(tokens + a.page - 1); };  // of at most (max_pages + 1) pages' tokens

  const int each = (a.B + threads - 1) / threads;  // sequences of a thread, side by side
  int L[kEach], n[kEach];
  uint32_t fits = 0, valid = 0;  // a bit for each of them
  Sums own = {0, 0, 0}, mine[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int b = tid * each + i;
    const bool in = i < each && b < a.B;
    L[i] = in ? a.seq_lens[b] : 0;
    n[i] = in ? a.new_lens[b] : 0;
  }
  int count = *a.free_count;
  if (tid == 0) given = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    mine[i] = {0, 0, 0};
    if (i < each) {
      const bool ok = L[i] >= 0 && L[i] <= cap;
      if (ok) {
        valid |= 1u << i;
        const int held = pages_of(L[i]);
        // where rows are fixed, a sequence that has too few of them asks for nothing
        const bool rows = !a.rows_each || (n[i] <= a.rows_each && (int64_t)(tid * each + i) * a.rows_each + n[i] <= a.T);
        if (n[i] > 0 && n[i] <= cap - L[i] && rows) {
          fits |= 1u << i;
          mine[i].need = pages_of(L[i] + n[i]) - held;
        }
        if (n[i] < 0) mine[i].back = held;
      } else if (first) {
        raise_status(a.status, MOE_ERR_BAD_INDEX);
      }
      mine[i].tokens = max(n[i], 0);
      own = add(own, mine[i]);
    }
  }
  // the sums before this thread's sequences, and of all
  const Sums up = scan(own, lane);
  if (lane == 31) warp_sums[warp] = up;
  __syncthreads();
  const Sums w = scan(lane < (threads >> 5) ? warp_sums[lane] : Sums{0, 0, 0}, lane), wx = exclusive(w, lane);
  const Sums all = {__shfl_sync(kAll, w.tokens, 31), __shfl_sync(kAll, w.need, 31), __shfl_sync(kAll, w.back, 31)};
  const Sums base = {__shfl_sync(kAll, wx.tokens, warp), __shfl_sync(kAll, wx.need, warp), __shfl_sync(kAll, wx.back, warp)};
  Sums at = add(base, exclusive(up, lane));

  if (count < 0 || count > a.num_pages) {
    if (first && tid == 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
    count = max(0, min(count, a.num_pages));
  }
  const int room = a.num_pages - count;
  if (all.back > room && first && tid == 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
  const int top = count + min(all.back, room);
  everyone(a.lens_out == a.seq_lens || a.count_out == a.free_count);  // all has been read

  // who is served, and the ended sequences' pages onto the stack
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (i >= each) break;
    const int b = tid * each + i, taken = add31(at.need, mine[i].need);
    const int64_t start = a.rows_each ? (int64_t)b * a.rows_each : at.tokens;  // of its rows
    const int end = (int)min(start + mine[i].tokens, (int64_t)INT32_MAX);
    if (b < a.B) {
      const bool served = (fits >> i & 1) && (mine[i].need == 0 || taken <= top) && end <= a.T;
      ends[b] = a.rows_each ? mine[i].tokens : end;
      before[b] = at.need;
      lens[b] = served ? L[i] : -1;
      if (served && mine[i].need) atomicMax(&given, taken);
      if (first) {
        if (n[i] > 0 && (valid >> i & 1) && !served) raise_status(a.status, MOE_ERR_CAPACITY);
        a.lens_out[b] = served ? L[i] + n[i] : n[i] < 0 && (valid >> i & 1) ? 0 : L[i];
        if (a.offsets) a.offsets[b + 1] = a.rows_each ? (int)min(start + a.rows_each, (int64_t)INT32_MAX) : end;
      }
    }
    // a warp the pages of one lane's sequence after the other's
    for (unsigned who = __ballot_sync(kAll, mine[i].back > 0); who; who &= who - 1) {
      const int from = __ffs(who) - 1;
      const int64_t to = (int64_t)count + __shfl_sync(kAll, at.back, from);
      const int pages = __shfl_sync(kAll, mine[i].back, from);
      const int32_t *row = a.table + (int64_t)__shfl_sync(kAll, b, from) * a.ts;
      for (int j = rank * 32 + lane; j < pages; j += ranks * 32)
        if (to + j < a.num_pages) a.free_pages[to + j] = row[j];
    }
    at = add(at, mine[i]);
  }
  everyone(all.back > 0);  // the sums are there, and the stack is whole

  const int step = ranks * threads;
  auto fresh = [&](int j) {  // page number j of those that are given, -1 for one that is none
    const int p = a.free_pages[top - 1 - j];
    return p >= 0 && p < a.num_pages ? p : -1;
  };
  // pages into the table: the first of a thread is on its way while its rows are made
  auto put_page = [&](int j, int b, int p) {
    a.table[b * a.ts + pages_of(lens[b]) + (j - before[b])] = p;
    if (p < 0) raise_status(a.status, MOE_ERR_BAD_INDEX);
  };
  // the last that no more than j pages lie before: it needs some
  auto owner = [&](int j) { return upper(before, a.B, a.log_b, j) - 1; };
  const int j0 = rank * threads + tid;
  int b0 = 0, p0 = 0;
  if (j0 < given) b0 = owner(j0), p0 = fresh(j0);
  for (int j = j0 + step; j < given; j += step) put_page(j, owner(j), fresh(j));
  if (first && tid == 0) {
    *a.count_out = top - given;
    if (a.offsets) a.offsets[0] = 0;
  }
  if (a.rows_each)
    put_fixed_rows(a, ends, before, lens, top, rank * threads + tid, step);
  else if (a.T <= step)
    put_rows<1>(a, ends, before, lens, top, rank * threads + tid, step);
  else
    put_rows<4>(a, ends, before, lens, top, rank * threads + tid, step);
  if (j0 < given) put_page(j0, b0, p0);
}

}  // namespace

moe_status_t launch_batch_plan(const int32_t *new_lens, const int32_t *seq_lens, int B, int page, int num_pages,
                               int32_t *table, int64_t ts, int max_pages, int32_t *free_pages, const int32_t *free_count,
                               int32_t *lens_out, int32_t *count_out, int32_t *offsets, int T, int rows_each, int32_t *slots,
                               int32_t *positions, int32_t *seq_ids, unsigned int *status, cudaStream_t stream,
                               int *launches) {
  int log_b = 1;
  while (1 << log_b <= B) ++log_b;
  const int wide = aligned16(slots) && (!positions || aligned16(positions)) && (!seq_ids || aligned16(seq_ids));
  const PlanArgs a = {new_lens, seq_lens, free_count, table, free_pages, lens_out, count_out, offsets, slots,
                      positions, seq_ids, status, ts, B, T, rows_each, page, num_pages, max_pages, log_b, wide, Divisor(page),
                      Divisor(rows_each > 1 ? rows_each : 2)};
  static PerDevice configured;
  const int set = configured.get([] {
    return cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 12 * kMaxB) == cudaSuccess &&
                   cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess
               ? 1
               : 0;
  });
  if (set < 1) return MOE_ERR_CUDA;
  // no more threads than rows or sequences, and a CTA for every 1024 rows, up to a cluster's 16
  int ctas = 1, threads = 128;
  while (threads < kMaxThreads && (threads < B || threads < T)) threads *= 2;
  while (ctas < kMaxCluster && T > kMaxThreads * ctas) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
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
