// Selection over beams and vocabulary (sm_103a).
//
// Candidate (beam w, token t) of a request scores s_w + x_wt - log sum_u exp x_wu.
// The call keeps the num_out best of a request, ties to the lower beam, then
// the lower token.  Every logit is read once, so the call is bound by HBM.
//
//  * A row of logits is cut into slices, a CTA each, that lie in shared memory
//    (one bulk copy; several CTAs share an SM, so that copies and arithmetic of
//    different slices overlap).  A slice leaves its maximum m, its
//    sum of exp(x - m) and its best num_out logits in order: nothing else of a row
//    can be among a request's best.
//  * The best of a slice: threads are dealt to at least num_out groups; the
//    least of the groups' maxima has num_out logits at or above it, and few more
//    (num_out times the harmonic number of num_out, for logits in any order).  Those
//    are listed and ordered by counting.  Where more are listed than there is
//    room for (a row of equal values, most of it set to the type's lowest), the
//    num_out-th largest value is found by bisection and its ties in order.
//  * A second kernel, a CTA per request, merges the slices' lists per row and
//    the rows' lists by score, the front entries of up to 32 lists in the lanes
//    of a warp.
//
// A score decides between candidates that may lie close together, so it is held
// as an unevaluated pair of floats: s - m - log l by error-free sums, the
// logarithm split in exponent and mantissa.  What is left is the rounding of the
// sum of exponentials, about 2^-23 relative.
#include <float.h>
#include <limits.h>
#include <math.h>

#include <cuda_fp16.h>

#include "vg_device.cuh"
#include "vg_host.h"

namespace vg {
namespace {

constexpr int kSliceThreads = 256;
constexpr int kSliceWarps = kSliceThreads / 32;
constexpr int kMaxSlices = 32;           // of a row: a lane each in the merge
constexpr int kMaxBeams = 32;
constexpr int kMaxOut = 64;
constexpr int kListed = 1024;            // candidates that a slice has room for
constexpr int kSliceBytes = 32 * 1024;   // of a slice, longer only where a row has more than 32 of them
constexpr int kLeastSliceBytes = 4 * 1024;
constexpr int kMostSliceBytes = 96 * 1024;

struct SelectParams {
  const uint8_t* logits;
  const float* scores;
  const uint8_t* ended;
  float* out_scores;
  int32_t* out_tokens;
  int32_t* out_parents;
  uint8_t* out_ended;
  float2* slice_ml;      // [rows][slices]: maximum, sum of exponentials
  float2* slice_best;    // [rows][slices][num_out]: logit, token (its bits); -1: none
  int32_t* error_flag;
  int64_t stride;        // bytes between rows
  uint64_t wait_ns;
  int end_token, batch, beams, vocab, num_out, slices, slice;
};

// Row `row` offers candidates of its own logits.
__device__ __forceinline__ bool row_lives(const SelectParams& p, int row) {
  const float s = p.scores[row];
  return s > -INFINITY && s < INFINITY && !(p.ended && p.ended[row]);
}

// Order-preserving image of a float (-0 as +0; no NaN).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A 32-bit word of logits as floats: two of 16 bits, or one.
template <int TYPE>
struct Word {
  static constexpr int kPer = TYPE == VG_TYPE_FP32 ? 1 : 2;
  static constexpr int kSize = 4 / kPer;
  static __device__ __forceinline__ void get(uint32_t w, float (&x)[kPer]) {
    if constexpr (TYPE == VG_TYPE_FP32) {
      x[0] = __uint_as_float(w);
    } else if constexpr (TYPE == VG_TYPE_BF16) {
      x[0] = __uint_as_float(w << 16);
      x[1] = __uint_as_float(w & 0xffff0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
      x[0] = f.x;
      x[1] = f.y;
    }
  }
};

// The slice in shared memory: element i at byte `off` + i * size.
template <int TYPE>
struct Slice {
  static constexpr int kPer = Word<TYPE>::kPer;
  const uint32_t* words;   // the word that holds element 0
  bool odd;                // element 0 is its upper half
  int n;
  __device__ __forceinline__ int count() const { return (n + kPer - 1) / kPer; }
  // word w: elements kPer * w .., -inf past the end
  __device__ __forceinline__ void get(int w, float (&x)[kPer]) const {
    uint32_t v = words[w];
    if (kPer == 2 && odd) v = __funnelshift_r(v, words[w + 1], 16);
    Word<TYPE>::get(v, x);
    if (kPer == 2 && 2 * w + 1 >= n) x[kPer - 1] = -INFINITY;
  }
};

// The CTA's sum of v, for every thread (two barriers).
__device__ __forceinline__ int cta_sum(int v, int* part) {
  const int s = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kSliceWarps; ++i) sum += part[i];
  __syncthreads();
  return sum;
}

// The num_out best where the list overflows: the num_out-th largest value by
// bisection, the larger ones listed, then its ties in order.  `least` has at least
// num_out elements at or above it, or is -inf.  Returns the list's length.
template <int TYPE>
__device__ __noinline__ int list_by_bisection(const Slice<TYPE>& sl, float least, float most, int num_out,
                                              float2* list, int* counter, int* part) {
  const int tid = threadIdx.x, words = sl.count();
  float x[Slice<TYPE>::kPer];
  uint32_t lo = ordered(least), hi = ordered(most);
  while (lo < hi) {  // the largest key with num_out elements at or above it
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const float t = from_ordered(mid);
    int n = 0;
    for (int w = tid; w < words; w += kSliceThreads) {
      sl.get(w, x);
#pragma unroll
      for (int j = 0; j < Slice<TYPE>::kPer; ++j) n += x[j] >= t;
    }
    if (cta_sum(n, part) >= num_out)
      lo = mid;
    else
      hi = mid - 1;
  }
  const float t = from_ordered(lo);
  if (tid == 0) *counter = 0;
  __syncthreads();
  for (int w = tid; w < words; w += kSliceThreads) {
    sl.get(w, x);
#pragma unroll
    for (int j = 0; j < Slice<TYPE>::kPer; ++j)
      if (x[j] > t) {
        const int at = atomicAdd(counter, 1);
        list[at] = make_float2(x[j], __int_as_float(Slice<TYPE>::kPer * w + j));
      }
  }
  __syncthreads();
  int have = *counter;  // below num_out, or every element above -inf
  if (t > -INFINITY) {
    for (int w0 = 0; w0 < words && have < num_out; w0 += kSliceThreads) {
      const int w = w0 + tid;
      int own = 0;
      if (w < words) {
        sl.get(w, x);
#pragma unroll
        for (int j = 0; j < Slice<TYPE>::kPer; ++j) own += x[j] == t;
      }
      int before = own;  // inclusive sum over the warp, then the warps before
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if ((tid & 31) >= o) before += v;
      }
      if ((tid & 31) == 31) part[tid >> 5] = before;
      __syncthreads();
      int all = 0;
#pragma unroll
      for (int i = 0; i < kSliceWarps; ++i) {
        if (i < (tid >> 5)) before += part[i];
        all += part[i];
      }
      int at = have + before - own;
#pragma unroll
      for (int j = 0; j < Slice<TYPE>::kPer; ++j)
        if (w < words && x[j] == t && at < num_out)
          list[at++] = make_float2(t, __int_as_float(Slice<TYPE>::kPer * w + j));
      have = min(have + all, num_out);
      __syncthreads();
    }
  }
  return have;
}

template <int TYPE>
__global__ void __launch_bounds__(kSliceThreads) beam_slice_kernel(const SelectParams p) {
  constexpr int PER = Word<TYPE>::kPer, SIZE = Word<TYPE>::kSize;
  extern __shared__ __align__(16) uint8_t data[];  // 16 bytes more than a slice, twice
  __shared__ __align__(8) uint64_t bar;
  __shared__ float2 list[kListed];
  __shared__ float group_max[kSliceWarps][32], sums[kSliceWarps];
  __shared__ int counter, part[kSliceWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.slices, s = blockIdx.x - row * p.slices;
  if (tid == 0) {
    mbar_init(&bar, 1);
    fence_barrier_init();
    counter = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (!row_lives(p, row)) return;
  const int first = s * p.slice, n = min(p.slice, p.vocab - first);
  // whole 16-byte pieces by one bulk copy, the ends by element
  const uint8_t* src = p.logits + row * p.stride + (int64_t)first * SIZE;
  const int off = (int)(reinterpret_cast<uintptr_t>(src) & 15);
  const int begin = (16 - off) & 15, bytes = n * SIZE;
  const int middle = max(bytes - begin, 0) & ~15;
  uint8_t* dst = data + off;
  __syncthreads();
  if (tid == 0) {
    mbar_arrive_expect_tx(&bar, middle);
    if (middle > 0) bulk_load(dst + begin, src + begin, middle, &bar);
  }
  if (tid >= 32 && tid < 64) {  // at most 7 elements on either side (3 of 32 bits)
    const int i = (tid & 15) * SIZE, at = tid < 48 ? i : begin + middle + i;
    if (tid < 48 ? i < min(begin, bytes) : at < bytes) {
      if (SIZE == 2)
        *reinterpret_cast<uint16_t*>(dst + at) = *reinterpret_cast<const uint16_t*>(src + at);
      else
        *reinterpret_cast<uint32_t*>(dst + at) = *reinterpret_cast<const uint32_t*>(src + at);
    }
  }
  __syncthreads();
  const bool landed = mbar_wait_checked(&bar, 0, p.wait_ns, p.error_flag);
  if (!landed) return;  // flagged; after a second nothing more is expected
  const Slice<TYPE> sl = {reinterpret_cast<const uint32_t*>(data + (off & ~3)), (off & 2) != 0, n};
  const int words = sl.count();
  // -------- the groups' maxima (fmaxf passes a NaN over; the sum shows it)
  float mx = -INFINITY;
#pragma unroll 4
  for (int w = tid; w < words; w += kSliceThreads) {
    float x[PER];
    sl.get(w, x);
#pragma unroll
    for (int j = 0; j < PER; ++j) mx = fmaxf(mx, x[j]);
  }
  int groups = 4;
  while (groups < p.num_out) groups *= 2;
  for (int o = 16; o >= groups; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  group_max[warp][lane] = mx;
  __syncthreads();
  float even = -INFINITY, uneven = -INFINITY;
#pragma unroll
  for (int i = 0; i < kSliceWarps; i += 2) {
    even = fmaxf(even, group_max[i][lane]);
    uneven = fmaxf(uneven, group_max[i + 1][lane]);
  }
  float m = fmaxf(even, uneven), least = groups > 32 ? fminf(even, uneven) : m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
  }
  // -------- the sum of exponentials, and what is at or above `least`
  const float ref = safe_ref(m), floor = fmaxf(least, -FLT_MAX);  // -inf is never listed
  float sum = 0.f;
#pragma unroll 4
  for (int w = tid; w < words; w += kSliceThreads) {
    float x[PER];
    sl.get(w, x);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      sum += ex2((x[j] - ref) * kLog2e);
      if (x[j] >= floor) {
        const int at = atomicAdd(&counter, 1);
        if (at < kListed) list[at] = make_float2(x[j], __int_as_float(PER * w + j));
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < kSliceWarps; ++i) l += sums[i];
    p.slice_ml[(int64_t)row * p.slices + s] = make_float2(m, l);
  }
  int listed = counter;
  if (listed > kListed) {
    __syncthreads();
    listed = list_by_bisection<TYPE>(sl, least, m, p.num_out, list, &counter, part);
    __syncthreads();
  }
  // -------- their order, by counting
  float2* best = p.slice_best + ((int64_t)row * p.slices + s) * p.num_out;
  for (int i = tid; i < listed; i += kSliceThreads) {
    const float2 c = list[i];
    int rank = 0;
    for (int j = 0; j < listed; ++j) {
      const float2 o = list[j];
      rank += o.x > c.x || (o.x == c.x && __float_as_int(o.y) < __float_as_int(c.y));
    }
    if (rank < p.num_out) best[rank] = make_float2(c.x, __int_as_float(first + __float_as_int(c.y)));
  }
  for (int i = listed + tid; i < p.num_out; i += kSliceThreads) best[i] = make_float2(-INFINITY, __int_as_float(-1));
}

// ------------------------------------------------------------------ the merge
// hi + lo = a + b exactly
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}
// a (a pair) + b, normalised
__device__ __forceinline__ float2 pair_add(float2 a, float b) {
  const float2 s = two_sum(a.x, b);
  return two_sum(s.x, __fadd_rn(s.y, a.y));
}

// s - m - log l.  The exponent's part of the logarithm is exact in 24 bits up to
// 2^-12 and a remainder, the mantissa's is at most 0.35 in size.
__device__ __forceinline__ float2 row_offset(float s, float m, float l) {
  int e;
  float f = frexpf(l, &e);
  if (f < 0.70710678f) {
    f *= 2.f;
    --e;
  }
  constexpr float kLn2Hi = 0.693359375f, kLn2Lo = -2.12194440e-4f;  // ln 2, its first 9 bits and the rest
  float2 c = two_sum(s, -m);
  c = pair_add(c, -(float)e * kLn2Hi);
  return pair_add(c, -fmaf((float)e, kLn2Lo, logf(f)));
}

constexpr int kRequestThreads = 256;

// Shared memory: [warps][slices * num_out] entries of the rows being merged, then
// [beams][num_out] entries of the rows' lists.
__global__ void __launch_bounds__(kRequestThreads) beam_merge_kernel(const SelectParams p) {
  extern __shared__ __align__(16) float2 entries[];
  __shared__ float2 offset[kMaxBeams];
  __shared__ float own_score[kMaxBeams];
  __shared__ int length[kMaxBeams];  // of a row's list; -1: an ended beam's one entry
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  const int per_row = p.slices * p.num_out;
  float2* lists = entries + (kRequestThreads / 32) * per_row;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  for (int w = warp; w < p.beams; w += kRequestThreads / 32) {
    const int row = b * p.beams + w;
    const float s = p.scores[row];
    const bool ended = p.ended && p.ended[row];
    bool bad = s != s || s == INFINITY;
    int n = 0;
    float2 c = make_float2(0.f, 0.f);
    if (ended && !bad) {
      n = s > -INFINITY ? -1 : 0;
    } else if (row_lives(p, row)) {
      // the row's entries, and its normaliser meanwhile
      float2* mine = entries + warp * per_row;
      const float2* src = p.slice_best + (int64_t)row * per_row;
      for (int i = lane; i < per_row; i += 32) mine[i] = __ldcg(src + i);
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < p.slices) ml = __ldcg(p.slice_ml + (int64_t)row * p.slices + lane);
      float m = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      // NaN where a slice's sum is one (it holds a NaN or +inf)
      float l = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ml.y * expf(ml.x - safe_ref(m));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      bad = !(l < INFINITY);
      if (!bad && l > 0.f) {
        c = row_offset(s, m, l);
        __syncwarp();
        // the slices' lists, a lane each, by logit; a lower lane's tokens are lower
        const float2* head = mine + lane * p.num_out;
        int d = 0;
        float2 x = lane < p.slices ? head[0] : make_float2(0.f, __int_as_float(-1));
        for (; n < p.num_out; ++n) {
          const uint32_t key = __float_as_int(x.y) >= 0 ? ordered(x.x) : 0u;
          const uint32_t top = __reduce_max_sync(0xffffffffu, key);
          if (top == 0u) break;
          const int win = __ffs(__ballot_sync(0xffffffffu, key == top)) - 1;
          if (lane == win) {
            lists[w * p.num_out + n] = x;
            x = ++d < p.num_out ? head[d] : make_float2(0.f, __int_as_float(-1));
          }
        }
      }
    }
    if (lane == 0) {
      if (bad) flag_error(p.error_flag, VG_DEVERR_VALUE);
      offset[w] = c;
      own_score[w] = s;
      length[w] = bad ? 0 : n;
    }
    __syncwarp();
  }
  __syncthreads();  // scores and marks have been read: the outputs may be the same arrays
  if (warp > 0) return;
  // the rows' lists, a lane each, by score; a lower lane is a lower beam
  const int n = lane < p.beams ? length[lane] : 0;
  const bool ended = n < 0;
  const float2 c = lane < p.beams ? offset[lane] : make_float2(0.f, 0.f);
  int d = 0, token = -1;
  float2 y = make_float2(0.f, 0.f);
  bool has = false;
  auto front = [&]() {
    has = d < (ended ? 1 : n);
    if (!has) return;
    if (ended) {
      y = make_float2(own_score[lane], 0.f);
      token = p.end_token;
    } else {
      const float2 x = lists[lane * p.num_out + d];
      y = pair_add(c, x.x);
      token = __float_as_int(x.y);
      has = y.x > -INFINITY;  // a sum past float's range is no candidate
    }
  };
  front();
  for (int k = 0; k < p.num_out; ++k) {
    const uint32_t hi = has ? ordered(y.x) : 0u, top = __reduce_max_sync(0xffffffffu, hi);
    const int64_t at = (int64_t)b * p.num_out + k;
    if (top == 0u) {
      if (lane == 0) {
        p.out_scores[at] = -INFINITY;
        p.out_tokens[at] = p.out_parents[at] = -1;
        if (p.out_ended) p.out_ended[at] = 0;
      }
      continue;
    }
    const uint32_t lo = has && hi == top ? ordered(y.y) : 0u, low = __reduce_max_sync(0xffffffffu, lo);
    const int win = __ffs(__ballot_sync(0xffffffffu, has && hi == top && lo == low)) - 1;
    if (lane == win) {
      p.out_scores[at] = y.x;
      p.out_tokens[at] = token;
      p.out_parents[at] = lane;
      if (p.out_ended) p.out_ended[at] = ended || token == p.end_token;
      ++d;
      front();
    }
  }
}

struct SelectPlan {
  int slices, slice;  // of a row; elements of one
  size_t off_best, bytes;
};

// Slices of 32 KB; more and shorter ones (down to 4 KB) while they are too few
// to fill the GPU, longer ones where a row has more than the merge has lanes.
// slices = 0: rows too long.
SelectPlan make_select_plan(int64_t rows, int vocab, int size, int num_out) {
  SelectPlan pl = {};
  const int64_t row = (int64_t)vocab * size;
  int64_t n = (row + kSliceBytes - 1) / kSliceBytes;
  const int64_t most = (row + kLeastSliceBytes - 1) / kLeastSliceBytes;
  const int64_t fill = (3 * (int64_t)device_sm_count() + rows - 1) / rows;
  n = n > (fill < most ? fill : most) ? n : (fill < most ? fill : most);
  if (n > kMaxSlices) n = kMaxSlices;
  const int piece = 16 / size;
  int64_t slice = (vocab + n - 1) / n;
  slice = (slice + piece - 1) / piece * piece;
  if (slice * size > kMostSliceBytes) return pl;
  pl.slice = (int)slice;
  pl.slices = (int)((vocab + slice - 1) / slice);
  pl.off_best = align_up((size_t)rows * pl.slices * sizeof(float2), 256);
  pl.bytes = pl.off_best + align_up((size_t)rows * pl.slices * num_out * sizeof(float2), 256);
  return pl;
}

int type_size(int type) {
  return type == VG_TYPE_FP32 ? 4 : type == VG_TYPE_BF16 || type == VG_TYPE_FP16 ? 2 : 0;
}

template <typename K>
cudaError_t allow_smem(K kernel, int bytes, bool (&set)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && set[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) set[dev] = true;
  return e;
}

template <int TYPE>
cudaError_t launch_slices(cudaLaunchConfig_t cfg, const SelectParams& p) {
  static bool set[64] = {false};
  const cudaError_t e = allow_smem(beam_slice_kernel<TYPE>, kMostSliceBytes + 32, set);
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, beam_slice_kernel<TYPE>, p);
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" size_t vg_beam_select_workspace_bytes(int batch, int beams, int vocab, int type, int num_out) {
  if (batch <= 0 || beams <= 0 || vocab <= 0 || num_out <= 0 || !type_size(type) || beams > kMaxBeams ||
      num_out > kMaxOut)
    return 0;
  const SelectPlan pl = make_select_plan((int64_t)batch * beams, vocab, type_size(type), num_out);
  return pl.slices ? pl.bytes : 0;
}

extern "C" vg_status vg_beam_select(const void* logits, int type, int64_t logits_stride, const float* scores,
                                    const uint8_t* ended, int end_token, int batch, int beams, int vocab,
                                    int num_out, float* out_scores, int32_t* out_tokens,
                                    int32_t* out_parents, uint8_t* out_ended, void* workspace,
                                    size_t workspace_bytes, int32_t* error_flag, cudaStream_t stream) {
  if (!logits || !scores || !out_scores || !out_tokens || !out_parents || batch <= 0 || beams <= 0 ||
      vocab <= 0 || num_out <= 0 || logits_stride < vocab)
    return VG_ERR_INVALID_ARGUMENT;
  const int size = type_size(type);
  if (!size || beams > kMaxBeams || num_out > kMaxOut || (int64_t)batch * beams > (1 << 24) ||
      logits_stride > ((int64_t)1 << 40))
    return VG_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(logits) % size) return VG_ERR_INVALID_ARGUMENT;
  const SelectPlan pl = make_select_plan((int64_t)batch * beams, vocab, size, num_out);
  if (!pl.slices) return VG_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < pl.bytes) return VG_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return VG_ERR_INVALID_ARGUMENT;
  SelectParams p = {};
  p.logits = static_cast<const uint8_t*>(logits);
  p.scores = scores;
  p.ended = ended;
  p.out_scores = out_scores;
  p.out_tokens = out_tokens;
  p.out_parents = out_parents;
  p.out_ended = out_ended;
  p.slice_ml = static_cast<float2*>(workspace);
  p.slice_best = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + pl.off_best);
  p.error_flag = error_flag;
  p.stride = logits_stride * size;
  p.wait_ns = wait_report_ns();
  p.end_token = end_token;
  p.batch = batch;
  p.beams = beams;
  p.vocab = vocab;
  p.num_out = num_out;
  p.slices = pl.slices;
  p.slice = pl.slice;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(batch * beams * pl.slices);
  cfg.blockDim = dim3(kSliceThreads);
  cfg.dynamicSmemBytes = (size_t)pl.slice * size + 32;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cudaError_t e = type == VG_TYPE_FP32   ? launch_slices<VG_TYPE_FP32>(cfg, p)
                  : type == VG_TYPE_BF16 ? launch_slices<VG_TYPE_BF16>(cfg, p)
                                         : launch_slices<VG_TYPE_FP16>(cfg, p);
  if (e != cudaSuccess) return VG_ERR_LAUNCH;
  static bool set[64] = {false};
  constexpr int kMostMerge = ((kRequestThreads / 32) * kMaxSlices + kMaxBeams) * kMaxOut * (int)sizeof(float2);
  e = allow_smem(beam_merge_kernel, kMostMerge, set);
  if (e != cudaSuccess) return VG_ERR_LAUNCH;
  cfg.gridDim = dim3(batch);
  cfg.blockDim = dim3(kRequestThreads);
  cfg.dynamicSmemBytes = ((size_t)(kRequestThreads / 32) * pl.slices + beams) * num_out * sizeof(float2);
  e = cudaLaunchKernelEx(&cfg, beam_merge_kernel, p);
  return e == cudaSuccess ? VG_OK : VG_ERR_LAUNCH;
}
