// Attention of a chunk of new tokens over the paged cache (sm_103a).
//
// Row (token i of sequence b, query head q) sits at position
// P = kv_len_b - n_b + i and computes softmax(scale q . k_j) v over the
// positions j <= P: one warp per row, lanes over the head's dimensions, the
// running maximum, sum and output in registers (fp32).
#include "vg_device.cuh"
#include "vg_host.h"

namespace vg {
namespace {

constexpr int kRowWarps = 8;

struct ChunkParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_pages;
  const __nv_bfloat16* v_pages;
  const int32_t* page_table;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  __nv_bfloat16* out;
  float* lse;
  int32_t* error_flag;
  int64_t q_stride, out_stride;
  float scale_log2;
  int batch, num_tokens, num_q_heads, num_kv_heads, num_pages, width;
};

template <int HD>
__global__ void __launch_bounds__(kRowWarps * 32) chunk_rows_kernel(const ChunkParams p) {
  constexpr int E = HD / 32;  // elements of the head per lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.batch; b += blockDim.x)
      if (p.cu_q[b] < 0 || p.cu_q[b + 1] < p.cu_q[b] || p.cu_q[b + 1] > p.num_tokens ||
          p.kv_lens[b] < 0 || p.kv_lens[b] > p.width * kPageSize)
        flag_error(p.error_flag, VG_DEVERR_LENGTH);
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const int t = (int)(row / p.num_q_heads), qh = (int)(row % p.num_q_heads);
  if (t >= p.num_tokens) return;
  int lo = 0, hi = p.batch;  // first sequence that ends past t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_q[mid + 1] > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  const int b = lo;
  if (b >= p.batch) return;
  const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], len = p.kv_lens[b];
  if (q0 < 0 || q0 > t || q1 > p.num_tokens || len < 0 || len > p.width * kPageSize) return;
  const int n = len - (q1 - q0) + (t - q0) + 1;  // attended positions
  const int h = qh / (p.num_q_heads / p.num_kv_heads);
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[t * p.q_stride + (int64_t)qh * HD + lane * E + e]) * p.scale_log2;
    o[e] = 0.f;
  }
  for (int j = 0; j < n; ++j) {
    const int page = p.page_table[(size_t)b * p.width + j / kPageSize];
    float k[E], v[E];
    const bool ok = page >= 0 && page < p.num_pages;
    if (!ok && lane == 0) flag_error(p.error_flag, VG_DEVERR_PAGE);
    const size_t at = ok ? (((size_t)page * p.num_kv_heads + h) * kPageSize + j % kPageSize) * HD + lane * E : 0;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      k[e] = ok ? __bfloat162float(p.k_pages[at + e]) : 0.f;
      v[e] = ok ? __bfloat162float(p.v_pages[at + e]) : 0.f;
      s = fmaf(q[e], k[e], s);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float m_new = fmaxf(m, s), ref = safe_ref(m_new);
    const float corr = ex2(m - ref), w = ex2(s - ref);
    l = l * corr + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * corr + w * v[e];
    m = m_new;
  }
  const float inv = n > 0 ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.out[t * p.out_stride + (int64_t)qh * HD + lane * E + e] = __float2bfloat16(o[e] * inv);
  if (p.lse && lane == 0)
    p.lse[(int64_t)t * p.num_q_heads + qh] = n > 0 ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <int HD>
cudaError_t launch_rows(const ChunkParams& p, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)p.num_tokens * p.num_q_heads + kRowWarps - 1) / kRowWarps));
  cfg.blockDim = dim3(kRowWarps * 32);
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_rows_kernel<HD>, p);
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" size_t vg_chunk_workspace_bytes(int batch, int num_tokens, int num_q_heads,
                                           int num_kv_heads, int head_dim) {
  (void)batch, (void)num_tokens, (void)num_q_heads, (void)num_kv_heads, (void)head_dim;
  return 0;
}

extern "C" vg_status vg_chunk_attention(const vg_paged_kv* kv, const void* q, int64_t q_stride,
                                        const int32_t* cu_q, const int32_t* kv_lens, int batch,
                                        int num_tokens, int num_q_heads, float softmax_scale,
                                        void* out, int64_t out_stride, float* lse, void* workspace,
                                        size_t workspace_bytes, int32_t* error_flag,
                                        cudaStream_t stream) {
  (void)workspace, (void)workspace_bytes;
  const vg_status st = check_paged_kv(kv);
  if (st != VG_OK) return st;
  if (!cu_q || !kv_lens || batch <= 0 || num_tokens < 0 || num_q_heads <= 0 ||
      !(softmax_scale > 0.f) || softmax_scale == INFINITY)
    return VG_ERR_INVALID_ARGUMENT;
  if (num_q_heads % kv->num_kv_heads) return VG_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return VG_OK;
  const int64_t row = (int64_t)num_q_heads * kv->head_dim;
  if (!q || !out || (reinterpret_cast<uintptr_t>(q) & 15) || (reinterpret_cast<uintptr_t>(out) & 15) ||
      q_stride < row || out_stride < row || q_stride % 8 || out_stride % 8)
    return VG_ERR_INVALID_ARGUMENT;
  if (num_q_heads / kv->num_kv_heads > 16 || batch > 4096 || kv->max_pages_per_seq > (1 << 26))
    return VG_ERR_UNSUPPORTED;
  ChunkParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.k_pages = static_cast<const __nv_bfloat16*>(kv->k_pages);
  p.v_pages = static_cast<const __nv_bfloat16*>(kv->v_pages);
  p.page_table = kv->page_table;
  p.cu_q = cu_q;
  p.kv_lens = kv_lens;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.error_flag = error_flag;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.scale_log2 = softmax_scale * kLog2e;
  p.batch = batch;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = kv->num_kv_heads;
  p.num_pages = kv->num_pages;
  p.width = kv->max_pages_per_seq;
  const cudaError_t e = kv->head_dim == 128 ? launch_rows<128>(p, stream) : launch_rows<64>(p, stream);
  return e == cudaSuccess ? VG_OK : VG_ERR_LAUNCH;
}
