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
  extern __shared__ float2 cs_s[];  // [tokens of the CTA][half], then their slots
  constexpr int IPH = HD / 16;      // items of a head
  const int t0 = blockIdx.x * p.tokens_per_cta;
  const int nt = min(p.tokens_per_cta, p.num_tokens - t0);
  int32_t* slot_s = reinterpret_cast<int32_t*>(cs_s + p.tokens_per_cta * p.half);
  const int heads = p.num_q_heads + 2 * p.num_kv_heads, qk = p.num_q_heads + p.num_kv_heads;
  const int items = nt * heads * IPH;
  const int turning = p.half / 8;   // items of a head that turn; the others pass
  // element offsets of an item's two pieces within its head
  auto pieces = [&](int c, int& off0, int& off1) {
    if (c < turning) {
      off0 = NEAR ? c * 16 : c * 8;
      off1 = NEAR ? off0 + 8 : p.half + off0;
    } else {  // passing items follow the turning dims two pieces at a time
      off0 = 2 * p.half + (c - turning) * 16;
      off1 = off0 + 8;
    }
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  bool ready = false;
  for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < items; i0 += kRopeThreads * kUnroll) {
    uint4 x0[kUnroll], x1[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kRopeThreads;
      if (i >= items) continue;
      const int hi = i / IPH, tl = hi / heads, hh = hi - tl * heads;
      const int64_t t = t0 + tl;
      const __nv_bfloat16* src =
          hh < p.num_q_heads ? p.q + t * p.q_stride + hh * HD
          : hh < qk          ? p.k + t * p.k_stride + (hh - p.num_q_heads) * HD
                             : p.v + t * p.v_stride + (hh - qk) * HD;
      int off0, off1;
      pieces(i % IPH, off0, off1);
      x0[u] = __ldcs(reinterpret_cast<const uint4*>(src + off0));
      x1[u] = __ldcs(reinterpret_cast<const uint4*>(src + off1));
    }
    if (!ready) {
      for (int i = threadIdx.x; i < nt; i += kRopeThreads) slot_s[i] = p.slots[t0 + i];
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
      ready = true;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kRopeThreads;
      if (i >= items) continue;
      const int c = i % IPH, hi = i / IPH, tl = hi / heads, hh = hi - tl * heads;
      if (c < turning && hh < qk) turn_item<NEAR>(x0[u], x1[u], cs_s + tl * p.half + c * 8);
      __nv_bfloat16* dst;
      if (hh < p.num_q_heads) {
        dst = p.q_out + (int64_t)(t0 + tl) * p.q_out_stride + hh * HD;
      } else {
        const int slot = slot_s[tl];
        if (slot < 0) continue;
        if (slot >= p.num_slots) {
          flag_error(p.error_flag, VG_DEVERR_INDEX);
          continue;
        }
        const int h = hh < qk ? hh - p.num_q_heads : hh - qk;
        dst = (hh < qk ? p.k_pages : p.v_pages) +
              (((int64_t)(slot / kPageSize) * p.num_kv_heads + h) * kPageSize + slot % kPageSize) * HD;
      }
      int off0, off1;
      pieces(c, off0, off1);
      *reinterpret_cast<uint4*>(dst + off0) = x0[u];
      *reinterpret_cast<uint4*>(dst + off1) = x1[u];
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
  cfg.dynamicSmemBytes = (size_t)p.tokens_per_cta * (p.half * sizeof(float2) + sizeof(int32_t));
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
