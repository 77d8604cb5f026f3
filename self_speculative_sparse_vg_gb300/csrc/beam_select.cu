// Selection over beams and vocabulary (sm_103a).
//
// Candidate (beam w, token t) of a request scores s_w + x_wt - log sum_u exp x_wu.
// The call keeps the num_out best of a request, ties to the lower beam, then
// the lower token.  Every logit is read once, so the call is bound by HBM.
//
//  * A row of logits is cut into slices, a CTA each, that lie in shared memory
//    (one bulk copy; six CTAs share an SM, so that copies and arithmetic of
//    different slices overlap: fewer CTAs that load ahead of what they compute, in
//    two buffers of 32 KB or a ring of 16 KB stages, were slower, 512 rows of 128K
//    51 and 58 us against 42).  A slice leaves its maximum m, its sum of exp(x - m)
//    and its best num_out logits in order: nothing else of a row can be among a
//    request's best.
//  * The best of a slice: threads are dealt to groups, twice num_out at least; the
//    num_out-th largest of the groups' maxima has num_out logits at or above it, and
//    few more (1.4 num_out in all, for logits in any order).  Those are listed and
//    ordered by counting.  Where more are listed than there is room for (a row of
//    equal values, most of it set to the type's lowest), the num_out-th largest
//    value is found by bisection and its ties in order.
//  * A second kernel, a CTA per request, merges the slices' lists: of their front
//    entries it finds a bound as the slices do, and orders by counting what reaches it.
//    Where more reach it than there is room for, one warp takes the best front entry of
//    all lists, place after place.
//
// A score decides between candidates that may lie close together, so it is held
// as an unevaluated pair of floats: s - m - log l by error-free sums, the
// logarithm split in exponent and mantissa.  What is left is the rounding of the
// sum of exponentials, about 2^-23 relative.
//
// Measured, calls in a row.  One request of four beams, 32K bf16 logits: 6.8 us, two
// launches' latency.  8 of four beams, 151936 float32 logits: 10.0 us.  16 of five,
// 50257 fp16 logits from odd addresses: 11.2 us.  64 of eight, 128256 bf16 logits: 40.5
// us (117 MB: 17.3 at the rate of a copy); there the slices take 34 us, of which the
// load and the maxima 20.5, the exponentials 4.7, the candidates and their order 9:
// issue is active 63 % of the time, and the short phases wait at barriers.  One request
// of many beams that keep many takes the warp's way through the lists: 16 beams keeping
// 32 of 32K 91 us, of 128K 149; 32 beams keeping 64 of 128K 300.
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
constexpr int kMaxSlices = 96;           // of a row
constexpr int kMaxBeams = 32;
constexpr int kMaxOut = 64;
constexpr int kListed = 256;             // candidates that a slice, or a request, has room for (more cost a
                                         // slice's shared memory the sixth CTA of an SM)
constexpr int kSliceBytes = 32 * 1024;   // of a slice, at most
constexpr int kLeastSliceBytes = 4 * 1024;

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
  uint32_t by_slices, by_out;  // ceil(2^32 / slices), / num_out; 0 for 1
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

// Words of logits: two of 16 bits in each, or one of 32.
template <int TYPE>
struct Word {
  static constexpr int kPer = TYPE == VG_TYPE_FP32 ? 1 : 2;
  static constexpr int kSize = 4 / kPer;
  static constexpr uint32_t kNone = TYPE == VG_TYPE_FP32   ? 0xff800000u
                                    : TYPE == VG_TYPE_BF16 ? 0xff80ff80u
                                                           : 0xfc00fc00u;  // -inf
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
  // two floats, of a word or of two
  static __device__ __forceinline__ void two(const uint32_t* w, float (&x)[2]) {
    if constexpr (kPer == 2) {
      get(w[0], x);
    } else {
      x[0] = __uint_as_float(w[0]);
      x[1] = __uint_as_float(w[1]);
    }
  }
  // maximum by element (a NaN gives way)
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (TYPE == VG_TYPE_FP32)
      r = __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    else if constexpr (TYPE == VG_TYPE_BF16)
      asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
      asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // the larger element of a word
  static __device__ __forceinline__ float top(uint32_t w) {
    float x[kPer];
    get(w, x);
    return kPer == 1 ? x[0] : fmaxf(x[0], x[kPer - 1]);
  }
};

// A slice lies in shared memory in pieces of 16 bytes, element 0 at the beginning
// of piece 0 wherever its row begins, -inf past the end; thread t takes pieces
// t + 256 j.  So equal rows have equal sums.
//
// A slice on a 16-byte boundary comes as one bulk copy (which completes on `bar`),
// but for the last piece if it is not whole.
template <int TYPE>
__device__ __forceinline__ void copy_slice(uint4* data, const uint8_t* src, int bytes, uint64_t* bar) {
  const int whole = bytes & ~15;
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(bar, whole);
    if (whole > 0) bulk_load(data, src, whole, bar);
  }
  if (bytes > whole && threadIdx.x >= 32 && threadIdx.x < 48) {
    constexpr int SIZE = Word<TYPE>::kSize;
    const int at = whole + (threadIdx.x - 32) * SIZE;
    uint8_t* dst = reinterpret_cast<uint8_t*>(data) + at;
    if (at < whole + 16) {
      if (SIZE == 2)
        *reinterpret_cast<uint16_t*>(dst) =
            at < bytes ? *reinterpret_cast<const uint16_t*>(src + at) : (uint16_t)Word<TYPE>::kNone;
      else
        *reinterpret_cast<uint32_t*>(dst) = at < bytes ? *reinterpret_cast<const uint32_t*>(src + at) : Word<TYPE>::kNone;
    }
  }
}

// Any other slice, `off` = 4 SHIFT (+ 2 if odd) bytes past a boundary: a piece out
// of two aligned loads (`base`), of which no more are made than hold an element
// of the slice (an allocation begins and ends on such a boundary).
template <int TYPE, int SHIFT>
__device__ __forceinline__ void shift_slice(uint4* data, const uint8_t* base, int off, int bytes) {
  const uint32_t none = Word<TYPE>::kNone;
  const bool odd = (off & 2) != 0;
#pragma unroll 4
  for (int at = 16 * threadIdx.x; at < bytes; at += 16 * kSliceThreads) {
    uint4 a = __ldg(reinterpret_cast<const uint4*>(base + at)), b = make_uint4(none, none, none, none);
    if (at + 16 - off < bytes) b = __ldg(reinterpret_cast<const uint4*>(base + at + 16));
    const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = TYPE != VG_TYPE_FP32 && odd ? __funnelshift_r(x[SHIFT + i], x[SHIFT + i + 1], 16) : x[SHIFT + i];
      const int left = bytes - at - 4 * i;  // of the slice, from this word on
      if (left <= 0)
        w[i] = none;
      else if (left < 4)
        w[i] = (w[i] & 0xffffu) | (none & 0xffff0000u);
    }
    data[at / 16] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// f(element number, value) for the elements of a thread's pieces that `may` let
// through (by the largest of a piece).
template <int TYPE, typename M, typename F>
__device__ __forceinline__ void for_elements(const uint4* data, int pieces, M may, F f) {
  constexpr int PER = Word<TYPE>::kPer;
#pragma unroll 2
  for (int q = threadIdx.x; q < pieces; q += kSliceThreads) {
    const uint4 v = data[q];
    using W = Word<TYPE>;
    if (!may(W::top(W::most(W::most(v.x, v.y), W::most(v.z, v.w))))) continue;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[PER];
      W::get(w[i], x);
#pragma unroll
      for (int j = 0; j < PER; ++j) f((4 * q + i) * PER + j, x[j]);
    }
  }
}

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

// Groups that the threads are dealt to: twice num_out at least, so that some 1.4
// num_out elements reach the num_out-th largest of their maxima.
constexpr int kGroups = 2 * kMaxOut;
__device__ __forceinline__ int groups_for(int num_out) { return num_out <= 16 ? 32 : num_out <= 32 ? 64 : kGroups; }

// The num_out-th largest of the groups' maxima: the least of those that fewer than
// num_out exceed.  One warp; group[]: its room.
__device__ __forceinline__ float kth_of_groups(const float* thread_max, float* group, int num_out) {
  const int lane = threadIdx.x & 31, groups = groups_for(num_out);
  for (int g = lane; g < groups; g += 32) {
    float v = thread_max[g];
    for (int t = g + groups; t < kSliceThreads; t += groups) v = fmaxf(v, thread_max[t]);
    group[g] = v;
  }
  __syncwarp();
  uint32_t least = 0xffffffffu;
  for (int g = lane; g < groups; g += 32) {
    const float v = group[g];
    int over = 0;
#pragma unroll 4
    for (int j = 0; j < groups; j += 4) {
      const float4 o = *reinterpret_cast<const float4*>(group + j);
      over += (o.x > v) + (o.y > v) + (o.z > v) + (o.w > v);
    }
    if (over < num_out) least = min(least, ordered(v));
  }
  return from_ordered(__reduce_min_sync(0xffffffffu, least));
}

// The num_out best where the list overflows: the num_out-th largest value by
// bisection, the larger ones listed, then its ties in order.  `least` has at least
// num_out elements at or above it, or is -inf.  Returns the list's length.
template <int TYPE>
__device__ __noinline__ int list_by_bisection(const uint4* data, int pieces, float least, float most, int num_out,
                                              float2* list, int* counter, int* part) {
  const int tid = threadIdx.x;
  uint32_t lo = ordered(least), hi = ordered(most);
  while (lo < hi) {  // the largest key with num_out elements at or above it
    const uint32_t mid = lo + (hi - lo + 1) / 2;
    const float t = from_ordered(mid);
    int n = 0;
    for_elements<TYPE>(data, pieces, [&](float top) { return top >= t; }, [&](int, float x) { n += x >= t; });
    if (cta_sum(n, part) >= num_out)
      lo = mid;
    else
      hi = mid - 1;
  }
  const float t = from_ordered(lo);
  if (tid == 0) *counter = 0;
  __syncthreads();
  for_elements<TYPE>(data, pieces, [&](float top) { return top > t; }, [&](int e, float x) {
    if (x > t) list[atomicAdd(counter, 1)] = make_float2(x, __int_as_float(e));
  });
  __syncthreads();
  int have = *counter;  // below num_out, or every element above -inf
  if (t == -INFINITY) return have;
  for (int q0 = 0; q0 < pieces && have < num_out; q0 += kSliceThreads) {
    // this thread's piece of the 256 from q0 on; their elements are in order
    const int end = min(pieces, q0 + kSliceThreads);
    int own = 0;
    if (q0 + tid < end)
      for_elements<TYPE>(data + q0, end - q0, [&](float top) { return top >= t; }, [&](int, float x) { own += x == t; });
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
    if (own > 0)
      for_elements<TYPE>(data + q0, end - q0, [&](float top) { return top >= t; }, [&](int e, float x) {
        if (x == t && at < num_out)
          list[at++] = make_float2(t, __int_as_float(q0 * 4 * Word<TYPE>::kPer + e));
      });
    have = min(have + all, num_out);
    __syncthreads();
  }
  return have;
}

template <int TYPE>
__global__ void __launch_bounds__(kSliceThreads, 6) beam_slice_kernel(const SelectParams p) {
  constexpr int PER = Word<TYPE>::kPer, SIZE = Word<TYPE>::kSize;
  extern __shared__ __align__(16) uint4 data[];
  __shared__ __align__(8) uint64_t bar;
  __shared__ float2 list[kListed];
  __shared__ __align__(16) float group_max[kGroups];
  __shared__ float thread_max[kSliceThreads];
  __shared__ float warp_max[kSliceWarps], warp_sum[kSliceWarps], kth;
  __shared__ uint16_t piece_list[kListed];
  __shared__ int counter, elements, dead, part[kSliceWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.slices, s = blockIdx.x - row * p.slices;
  if (tid == 0) {
    mbar_init(&bar, 1);
    fence_barrier_init();
    counter = elements = dead = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (!row_lives(p, row)) return;
  const int first = s * p.slice, n = min(p.slice, p.vocab - first), bytes = n * SIZE;
  const uint8_t* src = p.logits + row * p.stride + (int64_t)first * SIZE;
  const int off = (int)(reinterpret_cast<uintptr_t>(src) & 15);
  if (off == 0)
    copy_slice<TYPE>(data, src, bytes, &bar);
  else if (off < 4)
    shift_slice<TYPE, 0>(data, src - off, off, bytes);
  else if (off < 8)
    shift_slice<TYPE, 1>(data, src - off, off, bytes);
  else if (off < 12)
    shift_slice<TYPE, 2>(data, src - off, off, bytes);
  else
    shift_slice<TYPE, 3>(data, src - off, off, bytes);
  __syncthreads();
  if (off == 0) {
    // one warp looks, the others wait for it (256 threads that poll take issue
    // slots from the SM's other slices)
    if (warp == 0 && !mbar_wait_checked(&bar, 0, p.wait_ns, p.error_flag)) dead = 1;
    __syncthreads();
    if (dead) return;
  }
  const int pieces = (bytes + 15) / 16;
  using W = Word<TYPE>;
  auto piece_top = [](const uint4& v) { return W::most(W::most(v.x, v.y), W::most(v.z, v.w)); };
  // -------- maxima (a NaN is passed over; the sum shows it)
  uint32_t most = W::kNone;
#pragma unroll 4
  for (int q = tid; q < pieces; q += kSliceThreads) most = W::most(most, piece_top(data[q]));
  float m_warp = W::top(most);
  thread_max[tid] = m_warp;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m_warp = fmaxf(m_warp, __shfl_xor_sync(0xffffffffu, m_warp, o));
  if (lane == 0) warp_max[warp] = m_warp;
  __syncthreads();
  // -------- a value that at least num_out elements reach, and few more
  if (warp == 0) {
    const float v = kth_of_groups(thread_max, group_max, p.num_out);
    if (lane == 0) kth = v;
  }
  __syncthreads();
  // -------- sum of exponentials relative to the warp's maximum m, as 2^(c x - r)
  // with r = c m rounded, which is put right at the end (where c m is no float,
  // x - m is taken first); and the pieces that reach the value (never -inf)
  const float least = kth, floor = fmaxf(least, -FLT_MAX);
  const float base = safe_ref(m_warp);
  const bool plain = fabsf(base) < 1e30f;
  const float r = plain ? base * kLog2e : 0.f;
  uint64_t acc = 0;
  auto reached = [&](const uint4& v, int q) {
    if (W::top(piece_top(v)) >= floor) {
      const int at = atomicAdd(&counter, 1);
      if (at < kListed) piece_list[at] = q;
    }
  };
  if (plain) {
    const uint64_t c2 = pair(kLog2e, kLog2e), r2 = pair(-r, -r);
    auto add = [&](const uint4& v) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; i += 2 / PER) {
        float x[2];
        W::two(w + i, x);
        const float2 y = unpair(fma2(pair(x[0], x[1]), c2, r2));
        acc = add2(acc, pair(ex2(y.x), ex2(y.y)));
      }
    };
    int q = tid;
    for (; q + kSliceThreads < pieces; q += 2 * kSliceThreads) {  // two pieces, one look at both
      const uint4 v0 = data[q], v1 = data[q + kSliceThreads];
      add(v0);
      add(v1);
      if (W::top(W::most(piece_top(v0), piece_top(v1))) >= floor) {
        reached(v0, q);
        reached(v1, q + kSliceThreads);
      }
    }
    if (q < pieces) {
      add(data[q]);
      reached(data[q], q);
    }
  } else {
    for (int q = tid; q < pieces; q += kSliceThreads) {
      const uint4 v = data[q];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
      for (int i = 0; i < 4; i += 2 / PER) {
        float x[2];
        W::two(w + i, x);
        acc = add2(acc, pair(ex2((x[0] - base) * kLog2e), ex2((x[1] - base) * kLog2e)));
      }
      reached(v, q);
    }
  }
  const float2 a = unpair(acc);
  float sum = (a.x + a.y) * ex2(plain ? -fmaf(base, kLog2e, -r) : 0.f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) warp_sum[warp] = sum;
  __syncthreads();
  float m = warp_max[lane % kSliceWarps], m_own = m;
#pragma unroll
  for (int o = 1; o < kSliceWarps; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (warp == 0) {
    const float own = warp_sum[lane % kSliceWarps];
    float l = own == 0.f ? 0.f : own * expf(safe_ref(m_own) - safe_ref(m));
#pragma unroll
    for (int o = 1; o < kSliceWarps; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) p.slice_ml[(int64_t)row * p.slices + s] = make_float2(m, l);
  }
  // -------- the elements of those pieces, a thread each
  int listed = counter;
  constexpr int E = 4 * PER;
  if (listed <= kListed) {
    for (int i = tid; i < listed * E; i += kSliceThreads) {
      const int e = piece_list[i / E] * E + i % E;
      float x[PER];
      W::get(reinterpret_cast<const uint32_t*>(data)[e / PER], x);
      const float y = PER == 2 && (e & 1) ? x[PER - 1] : x[0];
      if (y >= floor) {
        const int at = atomicAdd(&elements, 1);
        if (at < kListed) list[at] = make_float2(y, __int_as_float(e));
      }
    }
    __syncthreads();
    listed = elements;
  }
  if (listed > kListed) {
    __syncthreads();
    listed = list_by_bisection<TYPE>(data, pieces, least, m, p.num_out, list, &counter, part);
    __syncthreads();
  }
  // -------- their order, by counting: four threads for each
  float2* best = p.slice_best + ((int64_t)row * p.slices + s) * p.num_out;
  for (int i0 = 0; i0 + (tid & ~31) / 4 < listed; i0 += kSliceThreads / 4) {
    const int i = i0 + tid / 4;
    const float2 c = list[i < listed ? i : 0];
    int rank = 0;
    for (int j = tid & 3; j < listed; j += 4) {
      const float2 o = list[j];
      rank += o.x > c.x || (o.x == c.x && __float_as_int(o.y) < __float_as_int(c.y));
    }
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    if (i < listed && (tid & 3) == 0 && rank < p.num_out)
      best[rank] = make_float2(c.x, __int_as_float(first + __float_as_int(c.y)));
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

constexpr int kRequestThreads = 256, kRequestWarps = kRequestThreads / 32;
constexpr int kHeads = 2 * kMaxOut;  // front entries that a bound is found from
constexpr int kEarly = 4;            // entries of a thread that are loaded with the normalisers

// A row of the request: what it adds to its logits, or that it offers one entry
// (it has ended) or nothing.
struct alignas(16) Row {
  float2 offset;
  float score;
  int kind;  // 0: nothing, 1: its entries, 2: the end token
};

struct Pick {
  uint64_t key;  // order of the score (hi, then lo); 0: none
  uint64_t tie;  // order among equal keys: beam, logit (largest first), where it stands in
                 // the lists.  (A key does not tell logits of a beam apart that differ
                 // by less than 2^-47 of its offset: 1e-20 and 2e-20 beside -10.)
};
constexpr int kAtBits = 18;  // list * num_out + depth
static_assert(kMaxBeams * kMaxSlices * kMaxOut <= 1 << kAtBits, "");

__device__ __forceinline__ uint64_t score_key(float2 y) {
  return y.x > -INFINITY ? (uint64_t)ordered(y.x) << 32 | ordered(y.y) : 0;  // past float's range: none
}

// n / d for the numbers of a request's entries, m = ceil(2^32 / d): exact while
// n d < 2^32.
__device__ __forceinline__ int quotient(int n, uint32_t m) { return m == 0 ? n : (int)__umulhi((uint32_t)n, m); }

// Key of entry `depth` of list `list` (a slice of a row), given what lies there.
__device__ __forceinline__ uint64_t key_of(const SelectParams& p, const Row* rows, int list, int depth, float2 raw) {
  const int w = quotient(list, p.by_slices);
  const Row r = rows[w];
  if (r.kind == 1 && __float_as_int(raw.y) >= 0) return score_key(pair_add(r.offset, raw.x));
  if (r.kind == 2 && depth == 0 && list == w * p.slices) return score_key(make_float2(r.score, 0.f));
  return 0;
}
__device__ __forceinline__ uint64_t tie_of(const SelectParams& p, int list, int at, float logit) {
  return (uint64_t)quotient(list, p.by_slices) << (32 + kAtBits) | (uint64_t)~ordered(logit) << kAtBits | (uint64_t)at;
}
__device__ __forceinline__ bool before(const Pick& a, const Pick& b) {
  return a.key > b.key || (a.key == b.key && a.tie < b.tie);
}

__device__ __forceinline__ void write_place(const SelectParams& p, const Row* rows, int b, int place, const Pick& k,
                                            int token) {
  const int64_t at = (int64_t)b * p.num_out + place;
  const bool none = k.key == 0;
  const int w = none ? -1 : (int)(k.tie >> (32 + kAtBits));
  if (!none && rows[w].kind == 2) token = p.end_token;
  p.out_scores[at] = none ? -INFINITY : from_ordered((uint32_t)(k.key >> 32));
  p.out_tokens[at] = none ? -1 : token;
  p.out_parents[at] = w;
  if (p.out_ended) p.out_ended[at] = !none && (rows[w].kind == 2 || token == p.end_token);
}

// Where more entries reach the bound than there is room for: the best front entry of
// all lists, one place after another (one warp, a lane takes every 32nd list).  That is
// so where many are level, and where the bound is low: past 128 lists it comes from 64
// maxima of four threads' fronts, of which it is the 32nd or 64th where as many are
// kept, and from fewer where beams do not live (a first step) or lie far apart.
// About 3 us a place (256 lists), 5 (928).
__device__ __noinline__ void merge_one_by_one(const SelectParams& p, const Row* rows, const float2* best, int b,
                                              uint8_t* depth) {
  const int lane = threadIdx.x & 31, lists = p.beams * p.slices;
  for (int l = lane; l < lists; l += 32) depth[l] = 0;
  for (int place = 0; place < p.num_out; ++place) {
    Pick top = {0, ~0ull};
    int token = -1;
    constexpr int kAhead = 4;  // lists of a lane whose loads are in flight together
    for (int l0 = lane; l0 < lists; l0 += 32 * kAhead) {
      float2 raw[kAhead];
      int d[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int l = l0 + 32 * i;
        d[i] = l < lists ? depth[l] : p.num_out;
        if (d[i] < p.num_out) raw[i] = __ldcg(best + l * p.num_out + d[i]);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (d[i] >= p.num_out) continue;
        const int l = l0 + 32 * i;
        const uint64_t key = key_of(p, rows, l, d[i], raw[i]);
        if (key == 0 || key < top.key) continue;
        const Pick k = {key, tie_of(p, l, l * p.num_out + d[i], raw[i].x)};
        if (before(k, top)) {
          top = k;
          token = __float_as_int(raw[i].y);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Pick k = {__shfl_xor_sync(0xffffffffu, top.key, o), __shfl_xor_sync(0xffffffffu, top.tie, o)};
      const int other = __shfl_xor_sync(0xffffffffu, token, o);
      if (before(k, top)) {
        top = k;
        token = other;
      }
    }
    if (lane == 0) write_place(p, rows, b, place, top, token);
    const int l = (int)(top.tie & ((1u << kAtBits) - 1u)) / p.num_out;
    if (top.key && l % 32 == lane) ++depth[l];
    __syncwarp();
  }
}

// A CTA per request.  Its rows' slices left sorted lists; a bound that num_out
// entries reach is the num_out-th largest of front entries, as in the slices.
__global__ void __launch_bounds__(kRequestThreads) beam_merge_kernel(const SelectParams p) {
  __shared__ Row rows[kMaxBeams];
  __shared__ __align__(16) float heads[kHeads];
  __shared__ Pick picks[kListed];
  __shared__ int tokens[kListed];
  __shared__ uint32_t bound;
  __shared__ int counter;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  const int lists = p.beams * p.slices, entries = lists * p.num_out, row0 = b * p.beams;
  const float2* best = p.slice_best + (int64_t)row0 * p.slices * p.num_out;
  // how many front entries of each list, and how many values to bound from
  const int front = (p.num_out + lists - 1) / lists, values = lists * front;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  // -------- loads (of rows that left nothing as well: whatever lies there)
  float2 early[kEarly], head = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kEarly; ++k)
    if (tid + k * kRequestThreads < entries) early[k] = __ldcg(best + tid + k * kRequestThreads);
  const int head_list = tid % lists, head_depth = tid / lists;
  if (tid < values) head = __ldcg(best + (int64_t)head_list * p.num_out + head_depth);
  constexpr int kRowsPerWarp = kMaxBeams / kRequestWarps;
  float2 ml[kRowsPerWarp];
  float score[kRowsPerWarp];
  bool ended[kRowsPerWarp];
#pragma unroll
  for (int k = 0; k < kRowsPerWarp; ++k) {
    const int w = warp + k * kRequestWarps;
    if (w >= p.beams) break;
    score[k] = p.scores[row0 + w];
    ended[k] = p.ended && p.ended[row0 + w];
    ml[k] = lane < p.slices ? __ldcg(p.slice_ml + (int64_t)(row0 + w) * p.slices + lane) : make_float2(-INFINITY, 0.f);
  }
  if (tid == 0) {
    bound = 0xffffffffu;
    counter = 0;
  }
  if (tid < kHeads) heads[tid] = -INFINITY;
  // -------- the rows' normalisers
#pragma unroll
  for (int k = 0; k < kRowsPerWarp; ++k) {
    const int w = warp + k * kRequestWarps;
    if (w >= p.beams) break;
    Row r = {make_float2(0.f, 0.f), score[k], 0};
    bool bad = !(score[k] < INFINITY);
    if (!bad && score[k] > -INFINITY) {
      if (ended[k]) {
        r.kind = 2;
      } else {
        float m = ml[k].x;
        for (int s = lane + 32; s < p.slices; s += 32)
          m = fmaxf(m, __ldcg(p.slice_ml + (int64_t)(row0 + w) * p.slices + s).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        // NaN where a slice's sum is one (it holds a NaN or +inf)
        auto part = [&](float2 x) { return x.y == 0.f ? 0.f : x.y * expf(x.x - safe_ref(m)); };
        float l = part(ml[k]);
        for (int s = lane + 32; s < p.slices; s += 32)
          l += part(__ldcg(p.slice_ml + (int64_t)(row0 + w) * p.slices + s));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        bad = !(l < INFINITY);
        if (!bad && l > 0.f) {
          r.kind = 1;
          r.offset = row_offset(score[k], m, l);
        }
      }
    }
    if (lane == 0) {
      if (bad) flag_error(p.error_flag, VG_DEVERR_VALUE);
      rows[w] = r;
    }
  }
  __syncthreads();  // scores and marks have been read: the outputs may be the same arrays
  // -------- the bound: on scores rounded to floats, whose order is that of scores
  auto rounded = [&](uint64_t key) { return key ? from_ordered((uint32_t)(key >> 32)) : -INFINITY; };
  float front_score = -INFINITY;
  if (tid < values) front_score = rounded(key_of(p, rows, head_list, head_depth, head));
  int n = values;
  if (values > kHeads) {  // many lists: the best front entry of every four threads
    for (int l = tid + kRequestThreads; l < lists; l += kRequestThreads)
      front_score = fmaxf(front_score, rounded(key_of(p, rows, l, 0, __ldcg(best + (int64_t)l * p.num_out))));
    front_score = fmaxf(front_score, __shfl_xor_sync(0xffffffffu, front_score, 1));
    front_score = fmaxf(front_score, __shfl_xor_sync(0xffffffffu, front_score, 2));
    n = kRequestThreads / 4;
    if ((tid & 3) == 0) heads[tid >> 2] = front_score;
  } else if (tid < values) {
    heads[tid] = front_score;
  }
  __syncthreads();
  if (tid < n) {
    const float v = heads[tid];
    int over = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 4) {
      const float4 o = *reinterpret_cast<const float4*>(heads + j);
      over += (o.x > v) + (o.y > v) + (o.z > v) + (o.w > v);
    }
    if (over < p.num_out) atomicMin(&bound, ordered(v));
  }
  __syncthreads();
  // -------- what reaches it
  const uint64_t least = max((uint64_t)bound << 32, (uint64_t)1);
  for (int i0 = 0, k = 0; i0 < entries; i0 += kRequestThreads, ++k) {
    const int i = i0 + tid;
    if (i >= entries) break;
    const float2 raw = k == 0 ? early[0] : k == 1 ? early[1] : k == 2 ? early[2] : k == 3 ? early[3] : __ldcg(best + i);
    const int list = quotient(i, p.by_out);
    const uint64_t key = key_of(p, rows, list, i - list * p.num_out, raw);
    if (key >= least) {
      const int at = atomicAdd(&counter, 1);
      if (at < kListed) {
        picks[at] = {key, tie_of(p, list, i, raw.x)};
        tokens[at] = __float_as_int(raw.y);
      }
    }
  }
  __syncthreads();
  const int listed = counter;
  if (listed > kListed) {
    if (warp == 0) merge_one_by_one(p, rows, best, b, reinterpret_cast<uint8_t*>(picks));
    return;
  }
  // -------- their order: eight threads count for each
  for (int c0 = 0; c0 < listed; c0 += kRequestThreads / 8) {
    const int c = c0 + (tid >> 3);
    const Pick own = picks[c < listed ? c : 0];
    int rank = 0;
    for (int j = tid & 7; j < listed; j += 8) {
      rank += before(picks[j], own);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (c < listed && rank < p.num_out && (tid & 7) == 0) write_place(p, rows, b, rank, own, tokens[c]);
  }
  for (int place = listed + tid; place < p.num_out; place += kRequestThreads)
    write_place(p, rows, b, place, Pick{0, 0}, -1);
}

struct SelectPlan {
  int slices, slice;  // of a row; elements of one
  size_t off_best, bytes;
};

// Slices of 32 KB; more and shorter ones (down to 4 KB) while they are too few
// to fill the GPU.  slices = 0: rows too long.
SelectPlan make_select_plan(int64_t rows, int vocab, int size, int num_out) {
  SelectPlan pl = {};
  const int64_t row = (int64_t)vocab * size;
  const int64_t least = (row + kSliceBytes - 1) / kSliceBytes;
  if (least > kMaxSlices) return pl;
  const int64_t most = (row + kLeastSliceBytes - 1) / kLeastSliceBytes;
  const int64_t fill = (3 * (int64_t)device_sm_count() + rows - 1) / rows;
  int64_t n = fill < most ? fill : most;
  if (n > 32) n = 32;
  if (n < least) n = least;
  const int piece = 16 / size;
  int64_t slice = (vocab + n - 1) / n;
  slice = (slice + piece - 1) / piece * piece;
  pl.slice = (int)slice;
  pl.slices = (int)((vocab + slice - 1) / slice);
  pl.off_best = align_up((size_t)rows * pl.slices * sizeof(float2), 256);
  pl.bytes = pl.off_best + align_up((size_t)rows * pl.slices * num_out * sizeof(float2), 256);
  return pl;
}

int type_size(int type) {
  return type == VG_TYPE_FP32 ? 4 : type == VG_TYPE_BF16 || type == VG_TYPE_FP16 ? 2 : 0;
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
  p.by_slices = pl.slices == 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + pl.slices - 1) / pl.slices);
  p.by_out = num_out == 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + num_out - 1) / num_out);
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(batch * beams * pl.slices);
  cfg.blockDim = dim3(kSliceThreads);
  cfg.dynamicSmemBytes = (size_t)pl.slice * size;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg,
                                     type == VG_TYPE_FP32   ? beam_slice_kernel<VG_TYPE_FP32>
                                     : type == VG_TYPE_BF16 ? beam_slice_kernel<VG_TYPE_BF16>
                                                            : beam_slice_kernel<VG_TYPE_FP16>,
                                     p);
  if (e != cudaSuccess) return VG_ERR_LAUNCH;
  cfg.gridDim = dim3(batch);
  cfg.blockDim = dim3(kRequestThreads);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, beam_merge_kernel, p);
  return e == cudaSuccess ? VG_OK : VG_ERR_LAUNCH;
}
