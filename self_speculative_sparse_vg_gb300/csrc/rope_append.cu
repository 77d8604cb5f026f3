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
// its item without shuffles.  A CTA takes as many tokens as give every thread
// several items; a thread loads up to kUnroll items before it waits, and the
// CTA computes each of its angles once while those loads are in flight.
//
// Angles: position * frequency is formed in double (a far position times a
// frequency has more than 24 significant bits) and reduced there to half a
// turn either way; only the sine and cosine are single precision.
#include <limits.h>

#include "vg_device.cuh"
#include "vg_host.h"

namespace vg {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnroll = 4;
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
  int num_tokens, num_q_heads, num_kv_heads, head_dim, num_slots, n_axes, half;
  int tokens_per_cta;
};

// (cos a, sin a) of a = pos * f, reduced to a fraction of a turn in double.
__device__ __forceinline__ float2 turn_of(int pos, float f) {
  constexpr double kInvTwoPi = 0.15915494309189533577;
  const double turns = (double)pos * (double)f * kInvTwoPi;
  float s, c;
  sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
  return make_float2(c, s);
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

template <bool NEAR>
__device__ __forceinline__ void turn_item(uint4& x0, uint4& x1, const float2* cs) {
  uint32_t a[4] = {x0.x, x0.y, x0.z, x0.w}, b[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (NEAR) {  // a word is a pair; frequencies i (first piece) and 4 + i
      const float2 u = unpack_bf16(a[i]), w = unpack_bf16(b[i]), c0 = cs[i], c1 = cs[4 + i];
      a[i] = pack_bf16(u.x * c0.x - u.y * c0.y, u.y * c0.x + u.x * c0.y);
      b[i] = pack_bf16(w.x * c1.x - w.y * c1.y, w.y * c1.x + w.x * c1.y);
    } else {     // pairs run across the two pieces; frequencies 2i, 2i + 1
      const float2 u = unpack_bf16(a[i]), w = unpack_bf16(b[i]), c0 = cs[2 * i], c1 = cs[2 * i + 1];
      a[i] = pack_bf16(u.x * c0.x - w.x * c0.y, u.y * c1.x - w.y * c1.y);
      b[i] = pack_bf16(w.x * c0.x + u.x * c0.y, w.y * c1.x + u.y * c1.y);
    }
  }
  x0 = make_uint4(a[0], a[1], a[2], a[3]);
  x1 = make_uint4(b[0], b[1], b[2], b[3]);
}

template <int HD, bool NEAR>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams p) {
  extern __shared__ float2 cs_s[];  // [tokens of the CTA][half]
  constexpr int IPH = HD / 16;      // items of a head
  const int t0 = blockIdx.x * p.tokens_per_cta;
  const int nt = min(p.tokens_per_cta, p.num_tokens - t0);
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int per_token = heads * IPH;
  const int items = nt * per_token;
  const int turning = p.half / 8;   // items of a head that turn; the others pass
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  bool have_angles = false;
  for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < items; i0 += kRopeThreads * kUnroll) {
    uint4 x0[kUnroll], x1[kUnroll];
    __nv_bfloat16* dst[kUnroll];
    int off0[kUnroll], off1[kUnroll], cs_at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kRopeThreads;
      dst[u] = nullptr;
      cs_at[u] = -1;
      if (i >= items) continue;
      const int c = i % IPH, hi = i / IPH, tl = hi / heads, hh = hi - tl * heads;
      const int64_t t = t0 + tl;
      // element offsets of the item's two pieces within the head
      const bool turns = c < turning;
      off0[u] = turns && !NEAR ? c * 8 : c * 16;
      off1[u] = turns && !NEAR ? p.half + c * 8 : c * 16 + 8;
      if (turns && hh < p.num_q_heads + p.num_kv_heads) {
        cs_at[u] = tl * p.half + c * 8;
      } else if (!turns) {
        // passing items follow the turning dims two pieces at a time
        off0[u] = 2 * p.half + (c - turning) * 16;
        off1[u] = off0[u] + 8;
      }
      const __nv_bfloat16* src;
      if (hh < p.num_q_heads) {
        src = p.q + t * p.q_stride + (int64_t)hh * HD;
        dst[u] = p.q_out + t * p.q_out_stride + (int64_t)hh * HD;
      } else {
        const bool is_k = hh < p.num_q_heads + p.num_kv_heads;
        const int h = hh - p.num_q_heads - (is_k ? 0 : p.num_kv_heads);
        const int slot = p.slots[t];
        if (slot < 0) continue;
        if (slot >= p.num_slots) {
          flag_error(p.error_flag, VG_DEVERR_INDEX);
          continue;
        }
        src = is_k ? p.k + t * p.k_stride + (int64_t)h * HD : p.v + t * p.v_stride + (int64_t)h * HD;
        dst[u] = (is_k ? p.k_pages : p.v_pages) +
                 (((int64_t)(slot / kPageSize) * p.num_kv_heads + h) * kPageSize + slot % kPageSize) * HD;
      }
      x0[u] = *reinterpret_cast<const uint4*>(src + off0[u]);
      x1[u] = *reinterpret_cast<const uint4*>(src + off1[u]);
    }
    if (!have_angles) {
      for (int i = threadIdx.x; i < nt * p.half; i += kRopeThreads) {
        const int tl = i / p.half, f = i - tl * p.half;
        int axis = p.freq_axis ? p.freq_axis[f] : 0;
        if (axis < 0 || axis >= p.n_axes) {
          flag_error(p.error_flag, VG_DEVERR_INDEX);
          axis = 0;
        }
        cs_s[i] = turn_of(p.positions[axis * p.pos_stride + t0 + tl], p.inv_freq[f]);
      }
      __syncthreads();
      have_angles = true;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!dst[u]) continue;
      if (cs_at[u] >= 0) turn_item<NEAR>(x0[u], x1[u], cs_s + cs_at[u]);
      *reinterpret_cast<uint4*>(dst[u] + off0[u]) = x0[u];
      *reinterpret_cast<uint4*>(dst[u] + off1[u]) = x1[u];
    }
  }
}

template <int HD>
cudaError_t launch_rope(const RopeParams& p, bool near, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ceil_div(p.num_tokens, p.tokens_per_cta));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.dynamicSmemBytes = (size_t)p.tokens_per_cta * p.half * sizeof(float2);
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
  p.head_dim = d;
  p.num_slots = kv->num_pages * kPageSize;
  p.n_axes = n_axes;
  p.half = rot_dim / 2;
  // as many tokens as give every thread kUnroll items, at most 64 (their
  // angles then fit 32 KB), at least one
  const int items = (num_q_heads + 2 * kv->num_kv_heads) * (d / 16);
  int tpc = kRopeThreads * kUnroll / items;
  p.tokens_per_cta = tpc < 1 ? 1 : tpc > 64 ? 64 : tpc;
  const cudaError_t e = d == 128 ? launch_rope<128>(p, interleaved != 0, stream)
                                 : launch_rope<64>(p, interleaved != 0, stream);
  return e == cudaSuccess ? VG_OK : VG_ERR_LAUNCH;
}
