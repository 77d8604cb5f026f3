// Block tables of beams that continue other beams, on the GPU (sm_103a).
//
// Row j of a request becomes a continuation of its row parents[j].  The rows of
// a request share the pages that are full: a page stands in several of its rows,
// always at the column of its positions, so the rows themselves say who holds
// it and no counter is kept.  A column is one thread's: it reads the request's old
// entries there, finds the pages that no new row holds (they go on the free
// list), and writes the new entries.  A partly filled last page is written to by
// its row, so it stays with one row; each other one that takes it gets a page
// from the list's end, and the copy is left to vg_copy_pages.
//
// The call is bound by latency (lengths, entries, list: dependent round trips).
// The columns of all requests form one line that the CTAs of one cluster share;
// the places of the returned pages are in line order, so the CTAs exchange their
// counts through distributed shared memory, and a second cluster barrier lies
// between what is pushed and what is popped.  A share of one column per thread
// (16K columns in a full cluster) is read once.
#include <limits.h>

#include "vg_device.cuh"
#include "vg_host.h"

namespace vg {
namespace {

constexpr int kThreads = 1024;
constexpr int kFewThreads = 256;      // of a CTA for a few rows and columns
constexpr int kMaxCluster = 16;
constexpr int kMaxRows = 4096;
constexpr int kMaxBeams = 32;

struct BeamParams {
  const int32_t* parents;
  int32_t* lens;
  int32_t* page_table;
  int32_t* owned;
  int32_t* free_pages;
  int32_t* free_count;
  int32_t* copies;
  int32_t* error_flag;
  int batch, beams, width, num_pages, free_capacity;
};

// Shared memory of a CTA: numbers per row, per request, and the old entries of
// the columns being worked on, [beams][threads].
struct BeamShared {
  int *len, *own, *tail, *rank;  // [rows]; tail: page of a new row's partly filled last page, -1: none;
                                 // rank: which of the pages asked for is its copy's, -1: none
  int *ends, *alive;             // [batch]: columns up to the request's end; mask of rows that go on
  int* stage;
  int8_t* parent;                // [rows]; -1: the row is emptied, -2: the request is refused
};

__host__ __device__ inline size_t shared_bytes(int batch, int beams, int threads) {
  const size_t rows = (size_t)batch * beams;
  return (4 * rows + 2 * (size_t)batch + (size_t)beams * threads) * sizeof(int) + rows;
}

__device__ __forceinline__ BeamShared carve(int* s, const BeamParams& p, int threads) {
  const int rows = p.batch * p.beams;
  BeamShared sh;
  sh.len = s;
  sh.own = s + rows;
  sh.tail = s + 2 * rows;
  sh.rank = s + 3 * rows;
  sh.ends = s + 4 * rows;
  sh.alive = sh.ends + p.batch;
  sh.stage = sh.alive + p.batch;
  sh.parent = reinterpret_cast<int8_t*>(sh.stage + p.beams * threads);
  return sh;
}

// Inclusive sum of v over the CTA's threads in order; `all` is the total.  One
// barrier before and one after `part` is used.
template <int NT>
__device__ __forceinline__ int cta_inclusive_sum(int v, int* part, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  int sum = lane < NT / 32 ? part[lane] : 0, before = lane < warp ? sum : 0;
  sum = __reduce_add_sync(0xffffffffu, sum);
  before = __reduce_add_sync(0xffffffffu, before);
  __syncthreads();
  *all = sum;
  return v + before;
}

__device__ __forceinline__ int pages_of(int len) { return (int)(((unsigned)len + kPageSize - 1) / kPageSize); }

// A column of the line: its request and number, and the old entries (stage).
struct Column {
  int b, c;
};

template <int NT>
__device__ __forceinline__ Column load_column(const BeamParams& p, const BeamShared& sh, int x) {
  int lo = 0, hi = p.batch - 1;  // the first request that ends past x
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sh.ends[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  const Column col = {lo, x - (lo > 0 ? sh.ends[lo - 1] : 0)};
  const int r0 = lo * p.beams;
  int* old = sh.stage + threadIdx.x;
#pragma unroll 8
  for (int i = 0; i < p.beams; ++i)
    old[i * NT] = col.c < sh.own[r0 + i] ? p.page_table[(int64_t)(r0 + i) * p.width + col.c] : -1;
  return col;
}

// f(page) for each page of the column that no new row holds, once, rows in
// order.  What is no page id is passed over, and flagged if `report`.
template <int NT, typename F>
__device__ __forceinline__ void for_returned(const BeamParams& p, const BeamShared& sh, const Column& col,
                                             bool report, F f) {
  const int r0 = col.b * p.beams;
  const int alive = sh.alive[col.b];
  const int* old = sh.stage + threadIdx.x;
  for (int i = 0; i < p.beams; ++i) {
    if (col.c >= sh.own[r0 + i]) continue;
    if ((alive >> i & 1) && col.c < pages_of(sh.len[r0 + i])) continue;
    const int page = old[i * NT];
    bool held = false;
    for (int k = 0; k < p.beams && !held; ++k)
      held = k != i && col.c < sh.own[r0 + k] && old[k * NT] == page &&
             (k < i || ((alive >> k & 1) && col.c < pages_of(sh.len[r0 + k])));
    if (held) continue;
    if (page < 0 || page >= p.num_pages) {
      if (report) flag_error(p.error_flag, VG_DEVERR_PAGE);
      continue;
    }
    f(page);
  }
}

template <int NT>
__global__ void __launch_bounds__(NT) beam_tables_kernel(const BeamParams p) {
  extern __shared__ int shared[];
  __shared__ int part[NT / 32], counts[kMaxCluster];
  const BeamShared sh = carve(shared, p, NT);
  const int tid = threadIdx.x, cta = blockIdx.x, ctas = gridDim.x;  // the grid is one cluster
  const int rows = p.batch * p.beams;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int top0 = *p.free_count;
  for (int r = tid; r < rows; r += NT) {
    sh.len[r] = p.lens[r];
    sh.own[r] = p.owned[r];
    const int j = p.parents[r];
    sh.parent[r] = (int8_t)(j >= -1 && j < p.beams ? j : -2);
  }
  __syncthreads();
  // -------- the requests' columns
  int end = 0, columns;
  for (int b0 = 0; b0 < p.batch; b0 += NT) {
    const int b = b0 + tid;
    int cols = 0, alive = 0, bad = 0;
    if (b < p.batch) {
      for (int i = 0; i < p.beams; ++i) {
        const int r = b * p.beams + i, j = sh.parent[r];
        if (j == -2) bad |= VG_DEVERR_INDEX;
        if (j >= 0) alive |= 1 << j;
        if (sh.len[r] < 0 || sh.own[r] < 0 || sh.own[r] > p.width || pages_of(sh.len[r]) > sh.own[r])
          bad |= VG_DEVERR_LENGTH;
        cols = max(cols, sh.own[r]);
      }
      if (bad) {
        if (cta == 0) flag_error(p.error_flag, bad);
        cols = alive = 0;
        for (int i = 0; i < p.beams; ++i) sh.parent[b * p.beams + i] = -2;
      }
      sh.alive[b] = alive;
    }
    const int e = end + cta_inclusive_sum<NT>(cols, part, &columns);
    if (b < p.batch) sh.ends[b] = e;
    end += columns;
  }
  columns = end;
  __syncthreads();
  // -------- who asks for a copy of its last page
  for (int r = tid; r < rows; r += NT) {
    const int j = sh.parent[r];
    int tail = -1;
    if (j >= 0) {
      const int from = r - r % p.beams + j, len = sh.len[from];
      if (len % kPageSize) tail = p.page_table[(int64_t)from * p.width + len / kPageSize];
    }
    sh.tail[r] = tail;
  }
  __syncthreads();
  int asked = 0;
  for (int r0 = 0; r0 < rows; r0 += NT) {
    const int r = r0 + tid;
    int ask = 0, all;
    if (r < rows && sh.tail[r] >= 0) {
      const int first = r - r % p.beams, full = sh.len[first + sh.parent[r]] / kPageSize;
      for (int k = first; k < r && !ask; ++k)
        ask = sh.tail[k] == sh.tail[r] && sh.len[first + sh.parent[k]] / kPageSize == full;
    }
    const int at = asked + cta_inclusive_sum<NT>(ask, part, &all) - ask;
    if (r < rows) sh.rank[r] = ask ? at : -1;
    asked += all;
  }
  // -------- pages that go back: counted, by CTA
  const int share = (columns + ctas - 1) / ctas, x0 = cta * share, x1 = min(columns, x0 + share);
  const bool once = share <= NT;
  Column col = {0, 0};
  int mine = 0, total;
  for (int x = x0 + tid; x < x1; x += NT) {
    col = load_column<NT>(p, sh, x);
    for_returned<NT>(p, sh, col, true, [&](int) { ++mine; });
  }
  cta_inclusive_sum<NT>(mine, part, &total);
  int base = top0, back = total;
  if (ctas > 1) {
    if (tid < ctas) {
      const uint32_t to = mapa_shared(smem_u32(&counts[cta]), tid);
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(total) : "memory");
    }
    __syncwarp();
    cluster_arrive_release();
    cluster_wait_acquire();
    back = 0;
    for (int i = 0; i < ctas; ++i) {
      if (i < cta) base += counts[i];
      back += counts[i];
    }
  } else {
    __syncthreads();
  }
  // a free list that is not one changes nothing
  if (top0 < 0 || top0 > p.free_capacity || back > p.free_capacity - top0) {
    if (cta == 0 && tid == 0) flag_error(p.error_flag, VG_DEVERR_POOL);
    for (int r = cta * NT + tid; r < rows; r += ctas * NT) {
      p.copies[3 * r] = p.copies[3 * r + 1] = -1;
      p.copies[3 * r + 2] = 0;
    }
    return;
  }
  const int top = top0 + back;
  // -------- pushed, and the new entries (those of copies come last)
  for (int xa = x0; xa < x1; xa += NT) {
    const int x = xa + tid;
    int n = 0;
    if (x < x1) {
      if (!once) col = load_column<NT>(p, sh, x);
      for_returned<NT>(p, sh, col, false, [&](int) { ++n; });
    }
    if (total > 0) {  // of this CTA
      int all;
      int at = base + cta_inclusive_sum<NT>(n, part, &all) - n;
      if (n > 0) for_returned<NT>(p, sh, col, false, [&](int page) { p.free_pages[at++] = page; });
      base += all;
    }
    if (x < x1) {
      const int r0 = col.b * p.beams;
      const int* old = sh.stage + tid;
      for (int i = 0; i < p.beams; ++i) {
        const int r = r0 + i, j = sh.parent[r];
        int page = -1;
        if (j >= 0 && sh.rank[r] < top) {
          const int len = sh.len[r0 + j], full = len / kPageSize;
          if (col.c == full && sh.rank[r] >= 0) continue;
          if (col.c < full || (col.c == full && len % kPageSize)) page = old[j * NT];
        }
        const bool had = col.c < sh.own[r];
        if (had ? page != old[i * NT] : page != -1) p.page_table[(int64_t)r * p.width + col.c] = page;
      }
    }
  }
  if (back > 0) {
    __syncwarp();
    if (ctas > 1) {
      cluster_arrive_release();
      cluster_wait_acquire();
    } else {
      __syncthreads();
    }
  }
  // -------- rows, and the pages for copies from the list's end
  for (int r = cta * NT + tid; r < rows; r += ctas * NT) {
    int from = -1, to = -1, held = 0;
    const int j = sh.parent[r];
    if (j != -2) {
      int len = 0;
      const int rank = sh.rank[r];
      if (j >= 0 && rank < top) {
        len = sh.len[r - r % p.beams + j];
        if (rank >= 0) {
          int page = __ldcg(p.free_pages + (top - 1 - rank));
          if (page < 0 || page >= p.num_pages) {
            flag_error(p.error_flag, VG_DEVERR_PAGE);
            page = -1;
          } else {
            from = sh.tail[r];
            to = page;
            held = len % kPageSize;
          }
          p.page_table[(int64_t)r * p.width + len / kPageSize] = page;
        }
      } else if (j >= 0) {
        flag_error(p.error_flag, VG_DEVERR_POOL);
      }
      p.lens[r] = len;
      p.owned[r] = pages_of(len);
    }
    p.copies[3 * r] = from;
    p.copies[3 * r + 1] = to;
    p.copies[3 * r + 2] = held;
  }
  if (cta == 0 && tid == 0) *p.free_count = top - min(asked, top);
}

template <int NT>
cudaError_t launch(const BeamParams& p, int ctas, cudaStream_t stream) {
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(beam_tables_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(226 * 1024));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(beam_tables_kernel<NT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev] = true;
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
  cfg.dynamicSmemBytes = shared_bytes(p.batch, p.beams, NT);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, beam_tables_kernel<NT>, p);
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_beam_tables(const int32_t* parents, int batch, int beams, int32_t* lens,
                                    int32_t* page_table, int max_pages_per_seq, int num_pages,
                                    int32_t* owned, int32_t* free_pages, int free_capacity,
                                    int32_t* free_count, int32_t* copies, int32_t* error_flag,
                                    cudaStream_t stream) {
  if (!parents || !lens || !page_table || !owned || !free_pages || !free_count || !copies || batch <= 0 ||
      beams <= 0 || max_pages_per_seq <= 0 || num_pages <= 0 || free_capacity <= 0)
    return VG_ERR_INVALID_ARGUMENT;
  // a column's number on the line has to fit an int32
  if (beams > kMaxBeams || (int64_t)batch * beams > kMaxRows || num_pages > INT_MAX / kPageSize ||
      max_pages_per_seq > INT_MAX / kPageSize || (int64_t)batch * max_pages_per_seq > INT_MAX - kThreads * kMaxCluster)
    return VG_ERR_UNSUPPORTED;
  BeamParams p = {};
  p.parents = parents;
  p.lens = lens;
  p.page_table = page_table;
  p.owned = owned;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.copies = copies;
  p.error_flag = error_flag;
  p.batch = batch;
  p.beams = beams;
  p.width = max_pages_per_seq;
  p.num_pages = num_pages;
  p.free_capacity = free_capacity;
  const int64_t columns = (int64_t)batch * max_pages_per_seq;  // at most
  int ctas = 1;
  while (ctas < kMaxCluster && (int64_t)ctas * kThreads < columns) ctas *= 2;
  const cudaError_t e = batch * beams <= kFewThreads && columns <= 4 * kFewThreads
                            ? launch<kFewThreads>(p, 1, stream)
                            : launch<kThreads>(p, ctas, stream);
  return e == cudaSuccess ? VG_OK : VG_ERR_LAUNCH;
}
