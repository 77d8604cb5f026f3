// Host-side helpers shared by the three entry points (internal header).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/vg.h"

namespace vg {

constexpr int kPageSize = 16;

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Multiprocessor count of the current device (cached per device).
int device_sm_count();

// Bound after which a pipeline wait reports VG_DEVERR_TIMEOUT (set with
// vg_set_wait_limit_ns; 1 s by default).  Kernels take it as a parameter.
uint64_t wait_report_ns();

// 4-D tiled TMA descriptor over a page pool viewed as
// [num_pages][num_kv_heads][16][head_dim] bf16, box = 64 x 16 x 1 x 1 with the
// 128-byte swizzle.  Cached per (pointer, shape).  Returns false on failure.
bool page_pool_tensor_map(const void* base, int num_pages, int num_kv_heads, int head_dim,
                          CUtensorMap* out);

// 3-D tiled TMA descriptor over packed token rows [num_tokens][num_heads]
// [head_dim] bf16 with token_stride elements between tokens, box = 64 dims x
// box_heads x box_tokens with the 128-byte swizzle (tokens past the end read
// zeros).  Made anew on every call.
bool token_rows_tensor_map(const void* base, int num_tokens, int num_heads, int head_dim,
                           int64_t token_stride, int box_heads, int box_tokens, CUtensorMap* out);

// 4-D tiled TMA descriptor over a page pool viewed as [num_pages * num_kv_heads
// * 2][head_dim / 64][8][64] bf16: index ((page * num_kv_heads + head) * 2 + i)
// is the i-th 8-position group of a page, so that one box of 64 x 8 x head_dim
// / 64 x 2 is a whole (page, head) chunk, laid down group by group, 64-dim
// block by block, with the 128-byte swizzle.  Made anew on every call.
bool page_chunk_tensor_map(const void* base, int num_pages, int num_kv_heads, int head_dim,
                           CUtensorMap* out);

// 4-D tiled TMA descriptor over token rows [num_tokens][num_heads][head_dim] of
// 16-bit values with token_stride elements between tokens, viewed as
// [num_heads][head_dim / 64][num_tokens][64], so that one box of 64 x box_tokens
// x head_dim / 64 x 1 is a tile of one head, 64-dim block by block, with the
// 128-byte swizzle (tokens past the end read zeros).  Made anew on every call.
bool head_tile_tensor_map(const void* base, int num_tokens, int num_heads, int head_dim,
                          int64_t token_stride, int box_tokens, CUtensorMap* out);

// Basic checks of a vg_paged_kv; VG_OK or an error status.
vg_status check_paged_kv(const vg_paged_kv* kv);

}  // namespace vg
