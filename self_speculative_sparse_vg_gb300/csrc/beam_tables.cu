// Block tables of beams that continue other beams, on the GPU (sm_103a).
//
// Row j of a request becomes a continuation of its row parents[j].  The rows of
// a request share the pages that are full: a page stands in several of its rows,
// always at the column of its positions, so the rows themselves say who holds
// it and no counter is kept.  A column's old entries say which pages no new row
// holds (they go on the free list); then the new entries are written.  A partly
// filled last page is written to by its row, so it stays with one row; each other
// one that takes it gets a page from the list's end, and the copy is left to
// vg_copy_pages.
//
// The call is bound by latency (lengths, entries, list: dependent round trips, and
// barriers between them).  The columns of all requests, in tiles of 32, form one
// line that the CTAs of one cluster share; the places of the returned pages are in
// line order, so the CTAs exchange their counts through distributed shared memory,
// and a second cluster barrier lies between the columns (old entries read, pages
// pushed) and the copies (pages popped, their entries written).
//
// Three kinds of columns.  Most hold one full page in all rows and go on doing so:
// a tile of such is looked at, a thread per column and all its loads in flight,
// and left.  Where no column of a tile holds several pages (a prompt that one
// row holds, a request that ends), the tile is one item of the list: one page a
// column is read again and the rows' entries follow from their lengths.  Other
// columns are items of their own, gone through by lanes, one per row, several
// columns of a warp at a time: who holds the same page is one `match` (a thread
// per column took 4000 cycles for eight rows).  Rows part at neighbouring
// columns and a long request's tiles lie side by side, so a CTA's warps share what
// each of them has found.
//
// Measured, calls in a row: 4 beams of 2100 positions 5.5 us, a launch's latency
// and five round trips.  32 requests of eight beams with up to 32768 positions, each
// call on a new state: 11.8 us when all go on, 16.4 us when a fifth of the requests begins
// or ends in the call (35.6 us with every column by lanes, 24.4 us with all rows of such
// a tile read again).
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
constexpr int kBatch = 8;             // entries of a thread whose loads are in flight together
constexpr int kTiles = 31;            // tiles of 32 columns of a warp that are remembered
constexpr int kListed = 96;           // items of a warp that the CTA's warps can share

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
  int row_bits;  // log2 of the lanes that a column's rows take
};

// Shared memory of a CTA: numbers per row and per request.
struct BeamShared {
  int *len, *own, *tail, *rank;  // [rows]; tail: page of a new row's partly filled last page, -1: none;
                                 // rank: which of the pages asked for is its copy's, -1: none
  int *kept, *held;              // [rows]; columns of an old row that a new one takes, and of a new row
  int *ends, *alive, *full;      // [batch]: tiles up to the request's end; mask of rows that go on (after
                                 // its check); columns that are full pages in every row, 0 if one ends
  int *bad;                      // [batch]: error bits
  int8_t* parent;                // [rows]; -1: the row is emptied, -2: the request is refused
};

__host__ __device__ inline size_t shared_bytes(int batch, int beams) {
  const size_t rows = (size_t)batch * beams;
  return (6 * rows + 4 * (size_t)batch) * sizeof(int) + rows;
}

__device__ __forceinline__ BeamShared carve(int* s, const BeamParams& p) {
  const int rows = p.batch * p.beams;
  BeamShared sh;
  sh.len = s;
  sh.own = s + rows;
  sh.tail = s + 2 * rows;
  sh.rank = s + 3 * rows;
  sh.kept = s + 4 * rows;
  sh.held = s + 5 * rows;
  sh.ends = s + 6 * rows;
  sh.alive = sh.ends + p.batch;
  sh.full = sh.alive + p.batch;
  sh.bad = sh.full + p.batch;
  sh.parent = reinterpret_cast<int8_t*>(sh.bad + p.batch);
  return sh;
}

// Inclusive sum of v over the CTA's threads in order; `all` is the total.  One
// barrier; `part` is used again two sums later at the earliest.
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
  *all = sum;
  return v + before;
}

__device__ __forceinline__ int pages_of(int len) { return (int)(((unsigned)len + kPageSize - 1) / kPageSize); }

// What a warp's list holds: a column (its request and number), or a tile of 32 columns
// of which each holds one page at most: b = -2 - request, c = 2 * its first column
// + how many pages go back.  b = -1: nothing.
struct Column {
  int b, c;
};

// Whether the page that a column's rows hold goes back: no new row takes it (kept: the
// columns that any takes).  A foreign one is flagged and dropped.
__device__ __forceinline__ bool goes_back(const BeamParams& p, int c, int kept, int page) {
  if (c < kept) return false;
  if (page >= 0 && page < p.num_pages) return true;
  flag_error(p.error_flag, VG_DEVERR_PAGE);
  return false;
}

// The columns of request b that new rows take.
__device__ __forceinline__ int columns_kept(const BeamParams& p, const BeamShared& sh, int b) {
  const int lane = threadIdx.x & 31;
  return __reduce_max_sync(0xffffffffu, lane < p.beams ? sh.kept[b * p.beams + lane] : 0);
}

// What changes of the tile at column c0 of request b, listed in order: its columns, or
// the tile if no column holds several pages.  Returns how many.
__device__ __forceinline__ int list_tile(const BeamParams& p, const BeamShared& sh, int b, int c0, Column* list) {
  const int lane = threadIdx.x & 31, c = c0 + lane;
  bool works = false, many = false, back = false;
  if (c0 + 32 <= sh.full[b]) {  // full pages, in every row
    const int32_t* at = p.page_table + (int64_t)b * p.beams * p.width + c;
    const int first = at[0];
    for (int i0 = 1; i0 < p.beams; i0 += kBatch) {
      int page[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) page[k] = i0 + k < p.beams ? at[(int64_t)(i0 + k) * p.width] : first;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) many |= page[k] != first;
    }
    works = many;
  } else {
    const int own = lane < p.beams ? sh.own[b * p.beams + lane] : 0, kept = columns_kept(p, sh, b);
    const int32_t* at = p.page_table + (int64_t)b * p.beams * p.width + c;
    int lo = INT_MAX, hi = INT_MIN;
    for (int i0 = 0; i0 < p.beams; i0 += kBatch) {
      int page[kBatch];  // (entries past a row's pages are loaded, too, and not looked at)
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        page[k] = i0 + k < p.beams && c < p.width ? at[(int64_t)(i0 + k) * p.width] : 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const bool has = c < __shfl_sync(0xffffffffu, own, i0 + k);
        lo = has ? min(lo, page[k]) : lo;
        hi = has ? max(hi, page[k]) : hi;
      }
    }
    works = lo <= hi;
    many = lo < hi;
    if (lo == hi) back = goes_back(p, c, kept, lo);
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, works);
  if (!mask) return 0;
  const bool columns = __any_sync(0xffffffffu, many);
  const int goes = __popc(__ballot_sync(0xffffffffu, back));
  __syncwarp();
  if (columns) {
    if (works) list[__popc(mask & ((1u << lane) - 1u))] = {b, c};
  } else if (lane == 0) {
    list[0] = {-2 - b, 2 * c0 + goes};
  }
  __syncwarp();
  return columns ? __popc(mask) : 1;
}

// A listed tile: its pages that go back to the free list from `place` on, and its
// new entries.  A row's copy is written last, by another thread.
__device__ __forceinline__ void write_tile(const BeamParams& p, const BeamShared& sh, int b, int c0, int place,
                                           int top) {
  const int lane = threadIdx.x & 31, c = c0 + lane, r0 = b * p.beams;
  int own = 0, held = 0, copied = -1;  // row `lane`: its columns before and after, and its copy's
  if (lane < p.beams) {
    const int rank = sh.rank[r0 + lane];
    own = sh.own[r0 + lane];
    held = rank < top ? sh.held[r0 + lane] : 0;
    copied = rank >= 0 ? held - 1 : -1;
  }
  const int most = __reduce_max_sync(0xffffffffu, own), kept = columns_kept(p, sh, b);
  const int row = __ffs(__ballot_sync(0xffffffffu, own == most)) - 1;  // it holds what any row does
  int32_t* at = p.page_table + (int64_t)r0 * p.width + c;
  const int page = c < most ? at[(int64_t)row * p.width] : -1;
  const bool differs = min(max(own, c0), c0 + 32) != min(max(held, c0), c0 + 32);
  const uint32_t rows = __ballot_sync(0xffffffffu, differs);
  const bool back = c < most && goes_back(p, c, kept, page);
  const uint32_t goes = __ballot_sync(0xffffffffu, back);
  if (back) p.free_pages[place + __popc(goes & ((1u << lane) - 1u))] = page;
  for (int i0 = 0; i0 < p.beams; i0 += kBatch) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k;
      const bool had = c < __shfl_sync(0xffffffffu, own, i), has = c < __shfl_sync(0xffffffffu, held, i);
      const bool copy = c == __shfl_sync(0xffffffffu, copied, i);
      if ((rows >> i & 1) && had != has && !copy) at[(int64_t)i * p.width] = has ? page : -1;
    }
  }
}

// One row of a column, in a lane: its old entry, and whether the page goes back
// (no new row holds it; the first of the rows that did).
struct Entry {
  int b, c, r, page;  // b <= -2, in its first lane: a tile
  bool has, keeps, back;
};

__device__ __forceinline__ Entry load_entry(const BeamParams& p, const BeamShared& sh, const Column& col) {
  const int i = threadIdx.x & ((1 << p.row_bits) - 1);
  Entry e = {-1, 0, 0, -1, false, false, false};
  if (col.b < 0 ? i > 0 : i >= p.beams) return e;  // a tile is its first lane's
  e.b = col.b;
  e.c = col.c;
  if (col.b < 0) return e;
  e.r = col.b * p.beams + i;
  e.has = col.c < sh.own[e.r];
  if (e.has) e.page = p.page_table[(int64_t)e.r * p.width + col.c];
  e.keeps = e.has && col.c < sh.kept[e.r];
  return e;
}

// What goes back of the columns of a warp's entries; returns the lanes.
__device__ __forceinline__ uint32_t find_returned(const BeamParams& p, Entry& e, bool report) {
  const int lane = threadIdx.x & 31, bits = p.row_bits;
  const uint32_t column = bits == 5 ? 0xffffffffu : ((1u << (1 << bits)) - 1u) << (lane >> bits << bits);
  const uint32_t holders = __ballot_sync(0xffffffffu, e.has), keepers = __ballot_sync(0xffffffffu, e.keeps);
  const uint32_t same = __match_any_sync(0xffffffffu, e.page) & holders & column;
  e.back = e.has && !(same & keepers) && !(same & ((1u << lane) - 1u));
  if (e.back && (e.page < 0 || e.page >= p.num_pages)) {
    if (report) flag_error(p.error_flag, VG_DEVERR_PAGE);
    e.back = false;
  }
  return __ballot_sync(0xffffffffu, e.back);
}

template <int NT>
__global__ void __launch_bounds__(NT) beam_tables_kernel(const BeamParams p) {
  extern __shared__ int shared[];
  __shared__ int parts[2][NT / 32], counts[kMaxCluster];
  __shared__ Column lists[NT / 32][kListed], spread_list[NT / 32 * kListed];
  const BeamShared sh = carve(shared, p);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  const int ctas = gridDim.x;  // the grid is one cluster
  const int rows = p.batch * p.beams;
  int turn = 0;  // of `parts`
  auto sum = [&](int v, int* all) { return cta_inclusive_sum<NT>(v, parts[turn ^= 1], all); };
  for (int b = tid; b < p.batch; b += NT) {
    sh.alive[b] = sh.bad[b] = sh.ends[b] = 0;
    sh.full[b] = INT_MAX;
  }
  // another CTA's shared memory is there once that CTA has begun
  if (ctas > 1) {
    __syncwarp();
    cluster_arrive_relaxed();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int top0 = *p.free_count;
  __syncthreads();
  // -------- the rows, and what they mean for their requests
  for (int r = tid; r < rows; r += NT) {
    const int b = r / p.beams;
    const int len = p.lens[r], own = p.owned[r], j = p.parents[r];
    const bool known = j >= -1 && j < p.beams;
    sh.len[r] = len;
    sh.own[r] = own;
    sh.parent[r] = (int8_t)(known ? j : -2);
    int bad = known ? 0 : VG_DEVERR_INDEX;
    if (len < 0 || own < 0 || own > p.width || pages_of(len) > own) bad |= VG_DEVERR_LENGTH;
    if (bad) atomicOr(&sh.bad[b], bad);
    if (known && j >= 0) atomicOr(&sh.alive[b], 1 << j);
    atomicMax(&sh.ends[b], own);
    atomicMin(&sh.full[b], known && j >= 0 ? len / kPageSize : 0);
  }
  __syncthreads();
  // the page at the end of each new row: on its way during the sum
  constexpr int kEarly = NT == kThreads ? kMaxRows / NT : 1;  // (fewer threads: at most a row each)
  int tails[kEarly];
#pragma unroll
  for (int k = 0; k < kEarly; ++k) {
    const int r = tid + k * NT;
    tails[k] = -1;
    if (r >= rows) break;
    const int b = r / p.beams, j = sh.parent[r];
    sh.kept[r] = sh.alive[b] >> (r - b * p.beams) & 1 ? pages_of(sh.len[r]) : 0;
    const int from = b * p.beams + j, len = j >= 0 ? sh.len[from] : 0;
    sh.held[r] = pages_of(len);
    if (sh.bad[b]) continue;
    if (len % kPageSize) tails[k] = p.page_table[(int64_t)from * p.width + len / kPageSize];
  }
  int tiles = 0;  // of the line
  for (int b0 = 0; b0 < p.batch; b0 += NT) {
    const int b = b0 + tid;
    int n = 0, all;
    const int bad = b < p.batch ? sh.bad[b] : 0;
    if (b < p.batch && !bad) n = (sh.ends[b] + 31) / 32;
    const int end = tiles + sum(n, &all);
    if (b < p.batch) sh.ends[b] = end;
    if (bad) {
      if (cta == 0) flag_error(p.error_flag, bad);
      sh.alive[b] = 0;
      for (int i = 0; i < p.beams; ++i) sh.parent[b * p.beams + i] = -2;
    }
    tiles += all;
  }
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (tid + k * NT < rows) sh.tail[tid + k * NT] = tails[k];
  __syncthreads();
  // -------- who asks for a copy of its last page
  int asked = 0;
  for (int r0 = 0; r0 < rows; r0 += NT) {
    const int r = r0 + tid;
    int ask = 0, all;
    if (r < rows && sh.tail[r] >= 0) {
      const int first = r - r % p.beams, full = sh.len[first + sh.parent[r]] / kPageSize;
      for (int k = first; k < r && !ask; ++k)
        ask = sh.tail[k] == sh.tail[r] && sh.len[first + sh.parent[k]] / kPageSize == full;
    }
    const int at = asked + sum(ask, &all) - ask;
    if (r < rows) sh.rank[r] = ask ? at : -1;
    asked += all;
  }
  // -------- the columns that change, and the pages that go back: counted
  const int step = 32 >> p.row_bits, sub = lane >> p.row_bits;  // columns of a pass, and this lane's
  const int warps = ctas * (NT / 32), w = cta * (NT / 32) + warp;
  // a warp has a run of tiles, and lists what changes of them
  const int share = (tiles + warps - 1) / warps;
  const int tile0 = min(tiles, w * share), tile1 = min(tiles, tile0 + share);
  int first_b = 0;  // the request of the first: the one that ends past it
  for (int hi = p.batch - 1; first_b < hi;) {
    const int mid = (first_b + hi) >> 1;
    if (sh.ends[mid] > tile0)
      hi = mid;
    else
      first_b = mid + 1;
  }
  auto list_next = [&](int t, int* b, Column* to) {  // tile t; *b: a request no later than its own
    while (sh.ends[*b] <= t) ++*b;
    return list_tile(p, sh, *b, (t - (*b > 0 ? sh.ends[*b - 1] : 0)) * 32, to);
  };
  Column* list = lists[warp];
  int k_begin = 0, k_end = 0;
  uint32_t has_work = 0;  // tiles with columns that change; those past kTiles share a bit
  int found = 0, listed;
  bool fits = true;
  for (int t = tile0, b = first_b; t < tile1; ++t) {
    fits &= found <= kListed - 32;  // past its room the list is made again
    const int n = list_next(t, &b, list + (fits ? found : 0));
    if (n > 0) has_work |= 1u << min(t - tile0, kTiles);
    found += n;
  }
  // where a warp has several passes: one list of the CTA, if every warp's has
  // fitted, cut anew in warps' shares
  constexpr int kMany = 1 << 16, kNotAll = 1 << 24;
  const int at = sum(lane > 0 ? 0 : !fits ? kNotAll : found > step ? found + kMany : found, &listed);
  const bool spread = listed < kNotAll;
  k_end = found;
  if (spread && listed >= kMany) {
    listed %= kMany;
    const int first = __shfl_sync(0xffffffffu, at, 0) % kMany - found;
    for (int k = lane; k < found; k += 32) spread_list[first + k] = list[k];
    const int each = (listed + NT / 32 - 1) / (NT / 32);
    k_begin = min(listed, warp * each);
    k_end = min(listed, k_begin + each);
    list = spread_list;
    __syncthreads();
  }
  // entry of column k of the list
  auto entry = [&](int k) {
    Column col = {-1, 0};
    if (k + sub < k_end) col = list[k + sub];
    return load_entry(p, sh, col);
  };
  int mine = 0, passes = 0;
  Entry e = {-1, 0, 0, -1, false, false, false};
  for (int t = tile0, b = first_b; t < tile1 || (spread && t == tile0); ++t) {
    if (!spread) k_end = has_work >> min(t - tile0, kTiles) & 1 ? list_next(t, &b, list) : 0;
    Entry next = entry(k_begin);
    for (int k0 = k_begin; k0 < k_end; k0 += step, ++passes) {
      e = next;
      next = entry(k0 + step);
      mine += __popc(find_returned(p, e, true)) + __reduce_add_sync(0xffffffffu, e.b <= -2 ? e.c & 63 : 0);
    }
    if (spread) break;
  }
  int total;
  const int before = sum(lane == 0 ? mine : 0, &total) - (lane == 0 ? mine : 0);
  int base = top0 + __shfl_sync(0xffffffffu, before, 0), back = total;
  if (ctas > 1) {
    __syncwarp();
    cluster_wait_acquire();  // of the arrival at the beginning
    if (tid < ctas) {
      const uint32_t to = mapa_shared(smem_u32(&counts[cta]), tid);
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(total) : "memory");
    }
    __syncwarp();
    cluster_arrive_release();
    cluster_wait_acquire();
    const int count = lane < ctas ? counts[lane] : 0;
    back = __reduce_add_sync(0xffffffffu, count);
    base += __reduce_add_sync(0xffffffffu, lane < cta ? count : 0);
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
  const bool once = passes == 1;  // the pass is still in the registers
  for (int t = tile0, b = first_b; t < tile1 || (spread && t == tile0); ++t) {
    if (!spread) k_end = has_work >> min(t - tile0, kTiles) & 1 ? list_next(t, &b, list) : 0;
    Entry next = once ? e : entry(k_begin);
    for (int k0 = k_begin; k0 < k_end; k0 += step) {
      if (!once) {
        e = next;
        next = entry(k0 + step);
        find_returned(p, e, false);
      }
      const uint32_t goes = __ballot_sync(0xffffffffu, e.back);
      int place = base + __popc(goes & ((1u << lane) - 1u));
      base += __popc(goes);
      for (uint32_t marks = __ballot_sync(0xffffffffu, e.b <= -2); marks; marks &= marks - 1) {
        const int at = __ffs(marks) - 1, c = __shfl_sync(0xffffffffu, e.c, at), n = c & 63;
        write_tile(p, sh, -2 - __shfl_sync(0xffffffffu, e.b, at), (c & ~63) / 2,
                   __shfl_sync(0xffffffffu, place, at), top);
        __syncwarp();
        if (lane > at) place += n;
        base += n;
      }
      if (e.back) p.free_pages[place] = e.page;
      const int j = e.b >= 0 ? sh.parent[e.r] : -1, first = lane >> p.row_bits << p.row_bits;
      const int from = __shfl_sync(0xffffffffu, e.page, first + max(j, 0));
      if (e.b < 0) continue;
      const int rank = sh.rank[e.r], held = rank < top ? sh.held[e.r] : 0;
      if (rank >= 0 && e.c == held - 1) continue;  // a copy's, written last
      const int page = e.c < held ? from : -1;
      if (e.has ? page != e.page : page != -1) p.page_table[(int64_t)e.r * p.width + e.c] = page;
    }
    __syncwarp();
    if (spread) break;
  }
  // before an entry of a copy is written every warp has read the old ones (a row that
  // takes its own last page as a copy is another row's source), and what was pushed is
  // there to be popped; the same decision in all CTAs
  if (back > 0 || asked > 0) {
    __syncwarp();
    if (ctas > 1) {
      cluster_arrive_release();
      cluster_wait_acquire();
    } else {
      __syncthreads();
    }
  }
  if (asked > top) {  // rows are emptied: their entries of columns that would stay, too
    for (int r = cta; r < rows; r += ctas)
      if (sh.rank[r] >= top)
        for (int c = tid; c < sh.own[r]; c += NT) p.page_table[(int64_t)r * p.width + c] = -1;
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
                                         170 * 1024);
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
  cfg.dynamicSmemBytes = shared_bytes(p.batch, p.beams);
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
  // twice a column's number, and the tiles of all requests, have to fit an int32
  if (beams > kMaxBeams || (int64_t)batch * beams > kMaxRows || num_pages > INT_MAX / kPageSize ||
      max_pages_per_seq > INT_MAX / kPageSize || (int64_t)batch * max_pages_per_seq > INT_MAX)
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
  while ((1 << p.row_bits) < beams) ++p.row_bits;
  p.width = max_pages_per_seq;
  p.num_pages = num_pages;
  p.free_capacity = free_capacity;
  const int64_t tiles = (int64_t)batch * ((max_pages_per_seq + 31) / 32);  // at most
  int ctas = 1;
  while (ctas < kMaxCluster && (int64_t)ctas * kThreads / 32 < tiles) ctas *= 2;
  const cudaError_t e = batch * beams <= kFewThreads && tiles <= kFewThreads / 32
                            ? launch<kFewThreads>(p, 1, stream)
                            : launch<kThreads>(p, ctas, stream);
  return e == cudaSuccess ? VG_OK : VG_ERR_LAUNCH;
}
