// Rotary positions and the append of new K/V rows to the paged cache (sm_103a).
//
// A pair (x_u, x_w) of a query or key head is turned by the angle
// a = position * inv_freq[i]:  y_u = x_u cos a - x_w sin a,
// y_w = x_w cos a + x_u sin a, with (u, w) = (i, i + rot / 2) or (2i, 2i + 1)
// and the position taken from the axis freq_axis[i] (time, height, width ...).
// Turned queries go to q_out; turned keys and the values go straight to their
// cache slots, so a layer's new rows are read once and written once.
//
// The call moves 2 (Hq + 2 Hkv) d bf16 per token and is bound by HBM; for a
// few tokens by latency.  An item is two 16-byte pieces of one head that hold
// eight pairs (pieces c and c + rot / 16, or 2c and 2c + 1), so a thread turns
// its item without shuffles.  A thread keeps one (head, c) of kUnroll tokens:
// its pointers move by a stride and nothing is divided per item (with a
// division and 64-bit offsets for each item the call was bound by the
// instructions, 43 us for 8192 tokens of 32 + 2 * 8 heads).  It loads all its
// items before it waits; meanwhile the CTA makes its tokens' angles, each once.
//
// Angles: a far position times a frequency has more than 24 significant bits,
// so the product is kept exactly until whole turns are taken off; only the
// sine and cosine are single precision.
#include <limits.h>

#include "vg_device.cuh"
#include "vg_host.h"

namespace vg {
namespace {

// Most threads of a CTA, tokens of a thread.  8192 tokens of 32 + 2 * 8 heads:
// 34.6 us (5.8 TB/s) as set, 35.4 with one token of a thread, 35.1 with 256
// threads, 35.6 with 512.  (Streaming stores: 33.2, but the next call reads what
// this one wrote.)
constexpr int kRopeThreads = 128;
constexpr int kUnroll = 2;
constexpr int kAxesMax = 8;

struct RopeParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_pages;
  __nv_bfloat16* v_pages;
  const int32_t* positions;
  const int32_t* slots;
  const float* inv_freq;
  const int32_t* freq_axis;
  int32_t* error_flag;
  int64_t q_stride, k_stride, v_stride, q_out_stride, pos_stride;  // elements between tokens / axes
  int num_tokens, num_q_heads, num_kv_heads, num_slots, n_axes, half;
  int per_cta;  // (head, c) columns of a CTA; its threads are some tokens' columns
  int side;     // tokens side by side
};

// (cos a, sin a) of a = pos * f, as a fraction of a turn.  A position below
// 2^24 is exact in single precision, so an fma gives the rest of its product
// with f, and another the rest of the product with 1 / (2 pi) (Dekker's exact
// product): the fraction is good to 1e-8 of a turn, in six operations of the
// full-rate pipe.  Farther positions go through double precision.
__device__ __forceinline__ float2 turn_of(int pos, float f) {
  float frac;
  if (pos > -(1 << 24) && pos < (1 << 24)) {
    constexpr double kInvTwoPi = 0.15915494309189533577;
    constexpr float kHi = (float)kInvTwoPi, kLo = (float)(kInvTwoPi - (double)kHi);
    const float x = (float)pos, hi = x * f, lo = fmaf(x, f, -hi);
    const float turns = hi * kHi;
    frac = (turns - rintf(turns)) + fmaf(lo, kHi, fmaf(hi, kLo, fmaf(hi, kHi, -turns)));
  } else {
    const double turns = (double)pos * (double)f * 0.15915494309189533577;
    frac = (float)(turns - rint(turns));
  }
  // the hardware sine and cosine: within 2^-21 on half a turn either way, far
  // below the one rounding to bf16 that follows
  float s, c;
  __sincosf(6.2831853071795865f * frac, &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// cs[j * stride] holds the cosines of the item's frequencies 2j and 2j + 1, then
// their sines.
template <bool NEAR>
__device__ __forceinline__ void turn_item(uint4& x0, uint4& x1, const float4* cs, int stride) {
  uint32_t a[4] = {x0.x, x0.y, x0.z, x0.w}, b[4] = {x1.x, x1.y, x1.z, x1.w};
  if (NEAR) {  // a word is a pair; frequencies 0 .. 3 in the first piece
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 w = cs[j * stride];
      uint32_t& p0 = j < 2 ? a[2 * j] : b[2 * j - 4];
      uint32_t& p1 = j < 2 ? a[2 * j + 1] : b[2 * j - 3];
      const float2 u = unpack_bf16(p0), v = unpack_bf16(p1);
      p0 = pack_bf16(u.x * w.x - u.y * w.z, u.y * w.x + u.x * w.z);
      p1 = pack_bf16(v.x * w.y - v.y * w.w, v.y * w.y + v.x * w.w);
    }
  } else {     // pairs run across the two pieces: two of them in each operation
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 w = cs[j * stride];
      const float2 u = unpack_bf16(a[j]), v = unpack_bf16(b[j]);
      const uint64_t u2 = pair(u.x, u.y), v2 = pair(v.x, v.y);
      const uint64_t c2 = pair(w.x, w.y), s2 = pair(w.z, w.w), m2 = pair(-w.z, -w.w);
      const float2 y = unpair(fma2(u2, c2, mul2(v2, m2))), z = unpair(fma2(v2, c2, mul2(u2, s2)));
      a[j] = pack_bf16(y.x, y.y);
      b[j] = pack_bf16(z.x, z.y);
    }
  }
  x0 = make_uint4(a[0], a[1], a[2], a[3]);
  x1 = make_uint4(b[0], b[1], b[2], b[3]);
}

template <int HD, bool NEAR>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams p) {
  extern __shared__ float4 cs_s[];  // [token of the CTA][4][half / 8]
  constexpr int IPH = HD / 16;      // items of a head
  const int tokens = p.side * kUnroll, t0 = blockIdx.x * tokens;
  const int nt = min(tokens, p.num_tokens - t0);
  int32_t* slot_s = reinterpret_cast<int32_t*>(cs_s + tokens * (p.half / 2));  // [token of the CTA]
  const int qk = p.num_q_heads + p.num_kv_heads;
  const int turning = p.half / 8;   // items of a head that turn; the others pass
  // this thread's column and first token
  const int tl0 = threadIdx.x / p.per_cta;
  const int col = blockIdx.y * p.per_cta + threadIdx.x - tl0 * p.per_cta;
  const int c = col % IPH, hh = col / IPH;
  const bool is_q = hh < p.num_q_heads, is_k = !is_q && hh < qk;
  const bool on = tl0 < p.side && hh < qk + p.num_kv_heads;
  // element offsets of the item's two pieces within its head; passing items
  // follow the turning dims two pieces at a time
  const bool turns = c < turning;
  const int off0 = !turns ? 2 * p.half + (c - turning) * 16 : NEAR ? c * 16 : c * 8;
  const int off1 = turns && !NEAR ? p.half + off0 : off0 + 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  uint4 x0[kUnroll], x1[kUnroll];
  if (on) {
    const int64_t stride = is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride;
    const __nv_bfloat16* src = (is_q   ? p.q + hh * HD
                                : is_k ? p.k + (hh - p.num_q_heads) * HD
                                       : p.v + (hh - qk) * HD) +
                               (t0 + tl0) * stride;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (tl0 + u * p.side < nt) {
        x0[u] = __ldcs(reinterpret_cast<const uint4*>(src + u * p.side * stride + off0));
        x1[u] = __ldcs(reinterpret_cast<const uint4*>(src + u * p.side * stride + off1));
      }
  }
  for (int i = threadIdx.x; i < nt; i += blockDim.x) slot_s[i] = p.slots[t0 + i];
  for (int i = threadIdx.x; i < nt * p.half; i += blockDim.x) {
    const int tl = i / p.half, f = i - tl * p.half;
    int axis = p.freq_axis ? p.freq_axis[f] : 0;
    if (axis < 0 || axis >= p.n_axes) {
      flag_error(p.error_flag, VG_DEVERR_INDEX);
      axis = 0;
    }
    float* at = reinterpret_cast<float*>(cs_s + tl * (p.half / 2) + (f % 8 / 2) * turning + f / 8) + f % 2;
    const float2 cs = turn_of(p.positions[axis * p.pos_stride + t0 + tl], p.inv_freq[f]);
    at[0] = cs.x;
    at[2] = cs.y;
  }
  __syncthreads();
  if (!on) return;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int tl = tl0 + u * p.side;
    if (tl >= nt) break;
    if (turns && hh < qk) turn_item<NEAR>(x0[u], x1[u], cs_s + tl * (p.half / 2) + c, turning);
    __nv_bfloat16* dst;
    if (is_q) {
      dst = p.q_out + (t0 + tl) * p.q_out_stride + hh * HD;
    } else {
      const int slot = slot_s[tl];
      if (slot < 0) continue;
      if (slot >= p.num_slots) {
        flag_error(p.error_flag, VG_DEVERR_INDEX);
        continue;
      }
      const int h = is_k ? hh - p.num_q_heads : hh - qk;
      dst = (is_k ? p.k_pages : p.v_pages) +
            (((int64_t)(slot / kPageSize) * p.num_kv_heads + h) * kPageSize + slot % kPageSize) * HD;
    }
    *reinterpret_cast<uint4*>(dst + off0) = x0[u];
    *reinterpret_cast<uint4*>(dst + off1) = x1[u];
  }
}

template <int HD>
cudaError_t launch_rope(const RopeParams& p, dim3 grid, int threads, bool near, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = (size_t)p.side * kUnroll * (p.half * sizeof(float2) + sizeof(int32_t));
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return near ? cudaLaunchKernelEx(&cfg, rope_append_kernel<HD, true>, p)
              : cudaLaunchKernelEx(&cfg, rope_append_kernel<HD, false>, p);
}

bool rows_ok(const void* base, int64_t stride, int heads, int head_dim) {
  return base && (reinterpret_cast<uintptr_t>(base) & 15) == 0 && stride % 8 == 0 &&
         stride >= (int64_t)heads * head_dim;
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_rope_append(const vg_paged_kv* kv, const void* q, int64_t q_stride,
                                    const void* k, int64_t k_stride, const void* v,
                                    int64_t v_stride, void* q_out, int64_t q_out_stride,
                                    int num_tokens, int num_q_heads, const int32_t* positions,
                                    int64_t pos_stride, int n_axes, const float* inv_freq,
                                    const int32_t* freq_axis, int rot_dim, int interleaved,
                                    const int32_t* slots, int32_t* error_flag,
                                    cudaStream_t stream) {
  const vg_status st = check_paged_kv(kv);
  if (st != VG_OK) return st;
  const int d = kv->head_dim;
  if (num_tokens < 0 || num_q_heads < 0 || rot_dim < 0 || rot_dim > d) return VG_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return VG_OK;
  if (!slots || !rows_ok(k, k_stride, kv->num_kv_heads, d) || !rows_ok(v, v_stride, kv->num_kv_heads, d))
    return VG_ERR_INVALID_ARGUMENT;
  if (num_q_heads > 0 && (!rows_ok(q, q_stride, num_q_heads, d) || !rows_ok(q_out, q_out_stride, num_q_heads, d)))
    return VG_ERR_INVALID_ARGUMENT;
  if (rot_dim > 0 && (!positions || !inv_freq || n_axes <= 0 || (n_axes > 1 && pos_stride < num_tokens)))
    return VG_ERR_INVALID_ARGUMENT;
  if (rot_dim % 16 || n_axes > kAxesMax || kv->num_pages > INT_MAX / kPageSize ||
      num_q_heads > 1024 || kv->num_kv_heads > 1024)
    return VG_ERR_UNSUPPORTED;
  RopeParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.k_pages = static_cast<__nv_bfloat16*>(const_cast<void*>(kv->k_pages));
  p.v_pages = static_cast<__nv_bfloat16*>(const_cast<void*>(kv->v_pages));
  p.positions = positions;
  p.slots = slots;
  p.inv_freq = inv_freq;
  p.freq_axis = freq_axis;
  p.error_flag = error_flag;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_out_stride = q_out_stride;
  p.pos_stride = pos_stride;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = kv->num_kv_heads;
  p.num_slots = kv->num_pages * kPageSize;
  p.n_axes = n_axes;
  p.half = rot_dim / 2;
  // Threads: as many tokens' columns side by side as fit kRopeThreads (at most
  // 32 tokens, whose angles fit 48 KB); a token of more columns than that is
  // cut over grid.y into equal parts of whole warps.
  const int columns = (num_q_heads + 2 * kv->num_kv_heads) * (d / 16);
  const int parts = ceil_div(columns, kRopeThreads);
  p.per_cta = parts == 1 ? columns : ceil_div(ceil_div(columns, parts), 32) * 32;
  p.side = kRopeThreads / p.per_cta < 32 ? kRopeThreads / p.per_cta : 32;
  const int threads = ceil_div(p.side * p.per_cta, 32) * 32;
  const dim3 grid(ceil_div(num_tokens, p.side * kUnroll), parts);
  const cudaError_t e = d == 128 ? launch_rope<128>(p, grid, threads, interleaved != 0, stream)
                                 : launch_rope<64>(p, grid, threads, interleaved != 0, stream);
  return e == cudaSuccess ? VG_OK : VG_ERR_LAUNCH;
}
