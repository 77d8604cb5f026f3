// Copies of the first positions of cache pages, for all layers in one launch
// (sm_103a): what vg_beam_tables leaves to copy.
//
// A page of a pool is [heads][16][head_dim]; the held positions of a head are one
// run of bytes.  A CTA copies one page of one pool (K or V of a layer), all
// its loads in flight before the first store; bound by HBM, or by the launch for
// a layer's few pages.
//
// Measured: 32 rows' pages of one layer (8 heads of 128) 3.9 us a call, 2.3 on the
// device; 128 rows' of 32 layers, 161 MB moved, 26 - 30 us a call, 27.4 in a graph
// (5.9 TB/s; 256 threads a page 29.7).
#include "vg_device.cuh"
#include "vg_host.h"

namespace vg {
namespace {

constexpr int kThreads = 128;
constexpr int kPoolsPerLaunch = 128;  // K and V of 64 layers
constexpr int kBatch = 8;             // 16-byte pieces of a thread in flight

struct CopyParams {
  uint4* pool[kPoolsPerLaunch];
  const int32_t* copies;
  int32_t* error_flag;
  int num_pages, num_kv_heads, pieces;  // 16-byte pieces of a position of a head
};

__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int32_t* c = p.copies + 3 * (int64_t)blockIdx.x;
  const int from = c[0], to = c[1], held = c[2];
  if (held == 0) return;
  if (from < 0 || from >= p.num_pages || to < 0 || to >= p.num_pages || held < 0 || held > kPageSize) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(p.error_flag, VG_DEVERR_PAGE);
    return;
  }
  const int per_head = kPageSize * p.pieces, run = held * p.pieces, all = p.num_kv_heads * run;
  uint4* pool = p.pool[blockIdx.y];
  const uint4* src = pool + (int64_t)from * p.num_kv_heads * per_head;
  uint4* dst = pool + (int64_t)to * p.num_kv_heads * per_head;
  for (int i0 = threadIdx.x; i0 < all; i0 += kBatch * kThreads) {
    uint4 v[kBatch];
    int at[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kThreads, head = i / run;
      at[k] = head * per_head + (i - head * run);
      if (i < all) v[k] = src[at[k]];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k * kThreads < all) dst[at[k]] = v[k];
  }
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" vg_status vg_copy_pages(void* const* k_pages, void* const* v_pages, int num_layers, int num_pages,
                                   int num_kv_heads, int head_dim, const int32_t* copies, int num_copies,
                                   int32_t* error_flag, cudaStream_t stream) {
  if (num_layers < 0 || num_copies < 0 || num_pages <= 0 || num_kv_heads <= 0 || head_dim <= 0)
    return VG_ERR_INVALID_ARGUMENT;
  if (head_dim != 64 && head_dim != 128) return VG_ERR_UNSUPPORTED;
  if ((int64_t)num_kv_heads * head_dim > (1 << 24)) return VG_ERR_UNSUPPORTED;
  if (num_layers == 0 || num_copies == 0) return VG_OK;
  if (!k_pages || !v_pages || !copies) return VG_ERR_INVALID_ARGUMENT;
  for (int i = 0; i < num_layers; ++i)
    if (!k_pages[i] || !v_pages[i] || (reinterpret_cast<uintptr_t>(k_pages[i]) & 15) ||
        (reinterpret_cast<uintptr_t>(v_pages[i]) & 15))
      return VG_ERR_INVALID_ARGUMENT;
  CopyParams p = {};
  p.copies = copies;
  p.error_flag = error_flag;
  p.num_pages = num_pages;
  p.num_kv_heads = num_kv_heads;
  p.pieces = head_dim / 8;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  for (int l0 = 0; l0 < num_layers; l0 += kPoolsPerLaunch / 2) {
    const int n = num_layers - l0 < kPoolsPerLaunch / 2 ? num_layers - l0 : kPoolsPerLaunch / 2;
    for (int i = 0; i < n; ++i) {
      p.pool[2 * i] = static_cast<uint4*>(k_pages[l0 + i]);
      p.pool[2 * i + 1] = static_cast<uint4*>(v_pages[l0 + i]);
    }
    cfg.gridDim = dim3(num_copies, 2 * n);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, copy_pages_kernel, p);
    if (e != cudaSuccess) return VG_ERR_LAUNCH;
  }
  return VG_OK;
}
