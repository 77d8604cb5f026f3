// Block tables and slot maps of a step, built on the GPU from the requests'
// lengths (sm_103a).
//
// With need_b = ceil((cached_b + new_b) / 16) pages, a request that holds more
// gives the rest back to the free list and one that holds fewer takes pages
// from its end; then token i of request b sits at position cached_b + i in
// cache slot table[b][position / 16] * 16 + position % 16.
//
// The work is a few integers per request and per token, so the call is bound
// by latency: dependent memory round trips and launches, not bytes.  One CTA
// resizes the tables (the free list is one stack, and three prefix sums over
// the requests fix every request's place in it): a thread owns IPT
// neighbouring requests, so one pass of warp shuffles makes each sum.  Then the
// tokens' positions and slots are written, a token per thread; past 1024 tokens
// the CTA is the first of a cluster that shares that part: the others find the
// rows' requests and positions while it works on the tables (114K tokens 8.0 us,
// 9.2 when they wait first).  When the cluster was chosen, 4096 tokens took 5.4
// us, 6.5 with one CTA alone, and 4.7 - 5.6 with a second kernel for the tokens,
// which cost 2 us more of host time.  A few requests and tokens get a CTA of 128
// threads, whose start and barriers are shorter: 3.1 us for 64 tokens of 8
// requests against 4.4 with 1024 (and three barriers a sum).
//
// Pages that move are loads with stores that wait for them, so the CTA shares the
// longer runs: 7 prompts of 8K - 16K tokens 11 us (46 with a request's run left to
// one warp), 8 requests that give 20K pages back 17 (52), 12 prompts beside 288
// other requests 13 (19); perf/more_cases.py measures these.
#include <limits.h>

#include "vg_device.cuh"
#include "vg_host.h"

namespace vg {
namespace {

constexpr int kTableThreads = 1024;
constexpr int kFewThreads = 128;       // of a CTA for a few requests and tokens
constexpr int kMaxTableCluster = 16;
constexpr int kMaxTableBatch = 8192;   // requests: 8 per thread
constexpr int kFillBatch = 4;          // tokens or pages of a thread whose loads are in flight together
constexpr int kRuns = 128;             // runs of pages that a CTA shares; a thread moves the others alone
constexpr int kRunBatch = 8;           // pages of a lane whose loads are in flight together in a shared run

struct TableParams {
  const int32_t* cached;
  const int32_t* fresh;
  int32_t* page_table;
  int32_t* owned;
  int32_t* free_pages;
  int32_t* free_count;
  int32_t* cu_tokens;
  int32_t* kv_lens;
  int32_t* positions;
  int32_t* slots;
  int32_t* error_flag;
  int batch, width, num_pages, free_capacity, max_tokens;
};

// A prefix sum over the CTA's threads in thread order, in two halves with a
// barrier between them, so that several sums share it: the inclusive sum within
// the warp, whose total goes to part[warp], ...
__device__ __forceinline__ long long warp_inclusive_sum(long long v, long long* part) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) part[threadIdx.x >> 5] = v;
  return v;
}

// ... and what the warps before this one add; `all` is the CTA's total.
template <int NT>
__device__ __forceinline__ long long sum_of_warps_before(const long long* part, long long* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long sum = lane < NT / 32 ? part[lane] : 0, before = lane < warp ? sum : 0;
#pragma unroll
  for (int o = 1; o < NT / 32; o <<= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  // lanes of one group of NT / 32 hold the entries
  *all = __shfl_sync(0xffffffffu, sum, 0);
  return __shfl_sync(0xffffffffu, before, 0);
}

// Positions and slots of token rows first, first + stride, ...; ends[b] =
// clamped end row of request b.  What needs no table comes before `tables_done`,
// which every thread calls once.
template <typename F>
__device__ __forceinline__ void fill_tokens(const TableParams& p, const int32_t* ends, int first,
                                            int stride, F tables_done) {
  for (int64_t t0 = first; t0 == first || t0 < p.max_tokens; t0 += (int64_t)kFillBatch * stride) {
    int req[kFillBatch], len[kFillBatch], page[kFillBatch];
    uint32_t pos[kFillBatch];  // means nothing where the request is refused
#pragma unroll
    for (int k = 0; k < kFillBatch; ++k) {
      const int64_t t = t0 + (int64_t)k * stride;
      int lo = 0, hi = t < p.max_tokens ? p.batch : 0;  // first request whose rows end past t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > t)
          hi = mid;
        else
          lo = mid + 1;
      }
      req[k] = t < p.max_tokens && lo < p.batch ? lo : -1;
      pos[k] = req[k] >= 0 ? (uint32_t)__ldg(p.cached + lo) + (uint32_t)(t - (lo > 0 ? ends[lo - 1] : 0)) : 0;
    }
    if (t0 == first) tables_done();
#pragma unroll
    for (int k = 0; k < kFillBatch; ++k) {
      const bool in = req[k] >= 0 && pos[k] / kPageSize < (uint32_t)p.width;
      len[k] = req[k] >= 0 ? __ldcg(p.kv_lens + req[k]) : 0;
      page[k] = in ? __ldcg(p.page_table + (size_t)req[k] * p.width + pos[k] / kPageSize) : -1;
    }
#pragma unroll
    for (int k = 0; k < kFillBatch; ++k) {
      const int64_t t = t0 + (int64_t)k * stride;
      if (t >= p.max_tokens) break;
      const bool served = len[k] > 0;
      int slot = -1;
      if (served) {
        if (page[k] >= 0 && page[k] < p.num_pages)
          slot = page[k] * kPageSize + (int)(pos[k] % kPageSize);
        else
          flag_error(p.error_flag, VG_DEVERR_PAGE);
      }
      p.positions[t] = served ? (int)pos[k] : 0;
      p.slots[t] = slot;
    }
  }
}

// Pages [lo, hi) of request b that move: page j goes to place at + j of the free
// list, or comes from place at - j.
struct PageRun {
  int b, lo, hi;
  long long at;
};

// Whether pages [lo, hi) of request b are page ids (those of this thread: first,
// first + step, ...).  Here and below the loads of N pages are issued together.
template <int N>
__device__ __forceinline__ bool pages_fine(const TableParams& p, int b, int lo, int hi, int first,
                                           int step) {
  const int32_t* row = p.page_table + (size_t)b * p.width;
  bool fine = true;
  for (int j = lo + first; j < hi; j += N * step) {
    int page[N];
#pragma unroll
    for (int k = 0; k < N; ++k) page[k] = j + k * step < hi ? row[j + k * step] : 0;
#pragma unroll
    for (int k = 0; k < N; ++k) fine &= page[k] >= 0 && page[k] < p.num_pages;
  }
  return fine;
}

template <int N>
__device__ __forceinline__ void push_pages(const TableParams& p, int b, int lo, int hi, long long at,
                                           int first, int step) {
  int32_t* row = p.page_table + (size_t)b * p.width;
  for (int j = lo + first; j < hi; j += N * step) {
    int page[N];
#pragma unroll
    for (int k = 0; k < N; ++k) page[k] = j + k * step < hi ? row[j + k * step] : 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (j + k * step < hi) {
        p.free_pages[at + j + k * step] = page[k];
        row[j + k * step] = -1;
      }
  }
}

template <int N>
__device__ __forceinline__ void pop_pages(const TableParams& p, int b, int lo, int hi, long long at,
                                          int first, int step) {
  int32_t* row = p.page_table + (size_t)b * p.width;
  for (int j = lo + first; j < hi; j += N * step) {
    int page[N];
#pragma unroll
    for (int k = 0; k < N; ++k)
      page[k] = j + k * step < hi ? p.free_pages[at - (j + k * step)] : 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (j + k * step < hi) {
        const bool fine = page[k] >= 0 && page[k] < p.num_pages;
        if (!fine) flag_error(p.error_flag, VG_DEVERR_PAGE);
        row[j + k * step] = fine ? page[k] : -1;
      }
  }
}

// f(run, lo, hi) for this warp's share of the runs' pieces.
template <int NT, typename F>
__device__ __forceinline__ void for_pieces(const PageRun* runs, int n, F f) {
  constexpr int kWarps = NT / 32, kPiece = 32 * kRunBatch;
  const int warp = threadIdx.x >> 5;
#pragma unroll 4
  for (int e = 0; e < n; ++e) {
    const int lo = runs[e].lo, count = runs[e].hi - lo;
    for (int k = (warp - e) & (kWarps - 1); k * kPiece < count; k += kWarps)
      f(e, lo + k * kPiece, lo + min(count, (k + 1) * kPiece));
  }
}

// The requests' end rows, in ends_s; and, by the grid's first CTA, the tables.
template <int NT, int IPT>
__device__ __forceinline__ void resize_tables(const TableParams& p, int32_t* ends_s,
                                              long long (*part)[NT / 32]) {
  __shared__ PageRun runs[kRuns];  // of pages that go back, then of pages that are taken
  __shared__ int runs_n[2], run_bad[kRuns];
  const int tid = threadIdx.x, lane = tid & 31;
  const int b0 = tid * IPT;
  if (tid < 2) runs_n[tid] = 0;
  // a fixed table has no free list: every request keeps the pages it has
  const bool fixed = p.owned == nullptr, leads = blockIdx.x == 0;
  const int top0 = fixed || !leads ? 0 : *p.free_count;
  int cached[IPT], fresh[IPT], own[IPT], need[IPT];
  bool ok[IPT];
  long long rows = 0;
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const int b = b0 + i;
    const bool in = b < p.batch;
    cached[i] = in ? p.cached[b] : 0;
    fresh[i] = in ? p.fresh[b] : 0;
    own[i] = in && !fixed && leads ? p.owned[b] : 0;
    rows += max(fresh[i], 0);
  }
  // -------- rows of the packed token buffer
  long long end = warp_inclusive_sum(rows, part[0]) - rows, all;
  __syncthreads();
  end += sum_of_warps_before<NT>(part[0], &all);
  int back = 0;
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    const int b = b0 + i;
    end += max(fresh[i], 0);
    const long long len = (long long)cached[i] + fresh[i];
    ok[i] = b < p.batch && cached[i] >= 0 && fresh[i] >= 0 &&
            len <= (long long)p.width * kPageSize && end <= p.max_tokens && own[i] >= 0 &&
            own[i] <= p.width;
    need[i] = ok[i] ? (int)((len + kPageSize - 1) / kPageSize) : 0;
    if (b < p.batch) {
      const int e = (int)(end < p.max_tokens ? end : p.max_tokens);
      ends_s[b] = e;
      if (!leads) continue;
      p.cu_tokens[b + 1] = e;
      if (!ok[i]) flag_error(p.error_flag, VG_DEVERR_LENGTH);
    }
  }
  if (!leads) return;
  if (tid == 0) p.cu_tokens[0] = 0;
  if (!fixed) {
    // -------- pages that go back: checked, then pushed.  A thread moves a few
    // pages of its request itself, longer runs are shared by the CTA.
    int run[IPT];
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
      run[i] = kRuns;
      if (ok[i] && own[i] > need[i]) {
        if (own[i] - need[i] > kFillBatch) run[i] = atomicAdd(&runs_n[0], 1);
        if (run[i] < kRuns) {
          runs[run[i]] = {b0 + i, need[i], own[i], 0};
          run_bad[run[i]] = 0;
        } else if (!pages_fine<kFillBatch>(p, b0 + i, need[i], own[i], 0, 1)) {
          ok[i] = false;
          flag_error(p.error_flag, VG_DEVERR_PAGE);
        }
      }
    }
    __syncthreads();
    const int returns = min(runs_n[0], kRuns);
    if (returns > 0) {
      for_pieces<NT>(runs, returns, [&](int e, int lo, int hi) {
        if (!pages_fine<kRunBatch>(p, runs[e].b, lo, hi, lane, 32)) run_bad[e] = 1;
      });
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
      if (run[i] < kRuns && run_bad[run[i]]) {
        ok[i] = false;
        flag_error(p.error_flag, VG_DEVERR_PAGE);
      }
      back += ok[i] ? max(own[i] - need[i], 0) : 0;
    }
    int grow = 0;  // a thread's own pages: at most 8 requests of < 2^27 pages
#pragma unroll
    for (int i = 0; i < IPT; ++i) grow += ok[i] ? max(need[i] - own[i], 0) : 0;
    long long back_sum = warp_inclusive_sum(back, part[1]), back_all;
    long long want = warp_inclusive_sum(grow, part[2]) - grow;  // asked for before this thread
    __syncthreads();
    back_sum += sum_of_warps_before<NT>(part[1], &back_all);
    want += sum_of_warps_before<NT>(part[2], &all);
    // a free list that is not one (its count is outside it, or the pages
    // coming back do not fit) changes nobody's pages
    const bool list_ok = top0 >= 0 && top0 + back_all <= p.free_capacity;
    const int top = top0 + (int)back_all;
    int at = top0 + (int)back_sum - back;  // this thread's first push
    if (list_ok) {
#pragma unroll
      for (int i = 0; i < IPT; ++i)
        if (ok[i] && own[i] > need[i]) {
          const long long to = (long long)at - need[i];
          if (run[i] < kRuns)
            runs[run[i]].at = to;
          else
            push_pages<kFillBatch>(p, b0 + i, need[i], own[i], to, 0, 1);
          at += own[i] - need[i];
        }
      if (returns > 0) {
        __syncthreads();
        for_pieces<NT>(runs, returns, [&](int e, int lo, int hi) {
          if (!run_bad[e]) push_pages<kRunBatch>(p, runs[e].b, lo, hi, runs[e].at, lane, 32);
        });
      }
    }
    __syncthreads();
    // -------- pages that are taken: the k-th page asked for is the k-th from
    // the list's end; a request past the end gets none
    int taken = 0;
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
      const int more = ok[i] ? max(need[i] - own[i], 0) : 0;
      const bool moves = ok[i] && need[i] != own[i];
      if (moves && (!list_ok || (more > 0 && want + more > top))) {
        ok[i] = false;
        flag_error(p.error_flag, VG_DEVERR_POOL);
      }
      if (ok[i] && more > 0) {
        const long long from = (long long)top - 1 - want + own[i];
        const int e = more > kFillBatch ? atomicAdd(&runs_n[1], 1) : kRuns;
        if (e < kRuns)
          runs[e] = {b0 + i, own[i], need[i], from};
        else
          pop_pages<kFillBatch>(p, b0 + i, own[i], need[i], from, 0, 1);
      }
      want += more;
      if (ok[i] && b0 + i < p.batch) {
        if (need[i] != own[i]) p.owned[b0 + i] = need[i];
        taken += more;
      }
    }
    warp_inclusive_sum(taken, part[3]);
    __syncthreads();
    for_pieces<NT>(runs, min(runs_n[1], kRuns), [&](int e, int lo, int hi) {
      pop_pages<kRunBatch>(p, runs[e].b, lo, hi, runs[e].at, lane, 32);
    });
    sum_of_warps_before<NT>(part[3], &all);
    if (tid == 0 && list_ok) *p.free_count = top - (int)all;
  }
#pragma unroll
  for (int i = 0; i < IPT; ++i)
    if (b0 + i < p.batch) p.kv_lens[b0 + i] = ok[i] ? cached[i] + fresh[i] : 0;
}

template <int NT, int IPT>
__global__ void __launch_bounds__(NT) step_tables_kernel(const TableParams p) {
  extern __shared__ int32_t ends_s[];  // [batch]
  __shared__ long long part[4][NT / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const bool cluster = gridDim.x > 1;  // the grid is one
  if (cluster && blockIdx.x > 0) cluster_arrive_release();
  resize_tables<NT, IPT>(p, ends_s, part);
  __syncwarp();  // the tables' work leaves a warp's lanes apart, the cluster's barrier wants them together
  if (cluster && blockIdx.x == 0) cluster_arrive_release();
  __syncthreads();
  fill_tokens(p, ends_s, blockIdx.x * NT + threadIdx.x, gridDim.x * NT, [&]() {
    __syncwarp();
    if (cluster) cluster_wait_acquire();
  });
}

template <int NT, int IPT>
cudaError_t launch_tables(const TableParams& p, int ctas, cudaStream_t stream) {
  if (ctas > 8) {
    static bool attr_set[64] = {false};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(step_tables_kernel<NT, IPT>,
                                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dev < 64) attr_set[dev] = true;
    }
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = (size_t)p.batch * sizeof(int32_t);  // at most 32 KB
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, step_tables_kernel<NT, IPT>, p);
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_step_tables(const int32_t* cached_lens, const int32_t* new_lens, int batch,
                                    int32_t* page_table, int max_pages_per_seq, int num_pages,
                                    int32_t* owned, int32_t* free_pages, int free_capacity,
                                    int32_t* free_count, int max_tokens, int32_t* cu_tokens,
                                    int32_t* kv_lens, int32_t* positions, int32_t* slots,
                                    int32_t* error_flag, cudaStream_t stream) {
  if (!cached_lens || !new_lens || !page_table || !cu_tokens || !kv_lens || batch <= 0 ||
      max_pages_per_seq <= 0 || num_pages <= 0 || max_tokens < 0)
    return VG_ERR_INVALID_ARGUMENT;
  if (max_tokens > 0 && (!positions || !slots)) return VG_ERR_INVALID_ARGUMENT;
  // the free list is given whole or not at all
  if ((owned != nullptr) != (free_pages != nullptr) || (owned != nullptr) != (free_count != nullptr) ||
      (owned && free_capacity <= 0))
    return VG_ERR_INVALID_ARGUMENT;
  // a slot number and a sequence length have to fit an int32
  if (batch > kMaxTableBatch || num_pages > INT_MAX / kPageSize ||
      max_pages_per_seq > INT_MAX / kPageSize)
    return VG_ERR_UNSUPPORTED;
  TableParams p = {};
  p.cached = cached_lens;
  p.fresh = new_lens;
  p.page_table = page_table;
  p.owned = owned;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.cu_tokens = cu_tokens;
  p.kv_lens = kv_lens;
  p.positions = positions;
  p.slots = slots;
  p.error_flag = error_flag;
  p.batch = batch;
  p.width = max_pages_per_seq;
  p.num_pages = num_pages;
  p.free_capacity = free_capacity;
  p.max_tokens = max_tokens;
  int ctas = 1;
  while (ctas < kMaxTableCluster && (int64_t)ctas * kTableThreads < max_tokens) ctas *= 2;
  const cudaError_t e =
      batch <= kFewThreads && max_tokens <= kFewThreads * kFillBatch
          ? launch_tables<kFewThreads, 1>(p, 1, stream)
          : batch <= kTableThreads ? launch_tables<kTableThreads, 1>(p, ctas, stream)
                                   : launch_tables<kTableThreads, 8>(p, ctas, stream);
  return e == cudaSuccess ? VG_OK : VG_ERR_LAUNCH;
}
