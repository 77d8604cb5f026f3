// Pieces of the attention kernels whose CTAs take equal shares of a line of
// units (up to two 128-row tiles of one KV head): bounded waits, tensor-memory
// loads, and the merges of units that a cut divides.
#pragma once

#include <cuda_fp16.h>

#include "vg_device.cuh"

namespace vg {
namespace {

constexpr int kUnitTile = 128;  // rows of a row tile

// a / b of non-negative numbers that mostly fit 32 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

__device__ __forceinline__ long long warp_inclusive_sum(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// Waits for the phase with the given parity, as mbar_wait_checked does, in less
// code.  Past the report bound the wait flags VG_DEVERR_TIMEOUT, past
// kWaitLimitNs it gives up.  (The timer is slow to read: with a look at it after
// every poll the whole kernel was 5 % slower; polls is 1 under a report bound
// shorter than the limit, and the polls then do not sleep.)  P: a kernel's parameters.
template <typename P>
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, const P& p) {
  uint64_t t0 = 0;
  while (true) {
#pragma unroll 1
    for (int i = 0; i < p.polls; ++i)
      if (p.polls > 1 ? mbar_try_wait(bar, parity) : mbar_test_wait(bar, parity)) return true;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > p.wait_ns) flag_error(p.error_flag, VG_DEVERR_TIMEOUT);
    if (now - t0 > kWaitLimitNs) return false;
  }
}
// The same for a whole warp, which stays together: mostly one look and one vote
// (a loop that the lanes leave one by one costs some 50 cycles more, and the
// tensor-core warp waits six times for a tile).
template <typename P>
__device__ __forceinline__ bool wait_phase_warp(uint64_t* bar, uint32_t parity, const P& p) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_phase(bar, parity, p));
}

// 64 consecutive columns of this warp's lanes, load and wait in one statement
// (no register is read before it has landed).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 32-byte store (a whole sector of a row per lane).
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A unit that several CTAs share, written by the CTA where it begins.
struct MergeUnit {
  int parts;          // 0: none
  int tok0, ntok, h;
};

// What the merges need of a call.  `out` has rows of bf16 or (F16) fp16.
struct MergeParams {
  uint16_t* out;
  float* lse;
  const float* part_o;     // [grid][2][HD / 4][rows][4]
  const float* part_ml;    // [grid][2][rows][2]
  const MergeUnit* merge;  // [grid]
  int64_t out_stride;
  int num_q_heads, group, rows;
};

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (!F16) return pack_bf16(lo, hi);
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Merge of the units that several CTAs share, weights 2^(m - max m) of the
// parts, which sit in slot 1 of the CTA where the unit begins and in slot 0 of
// the following ones.  A CTA takes 32 rows, a lane each (the parts' layout);
// a warp takes an eighth of the dimensions, and the rows leave through shared
// memory in whole lines.  No part is left out for its weight: one that a row does
// not attend is zero, and a NaN or an infinity of one whose weight underflows
// still has to show (as NaN), as it does where no cut falls.
constexpr int kMergeWarps = 8, kMergeRows = 32;
constexpr int kMergeBatch = 2;  // parts whose loads are in flight together (most units have two)
// MORE: units may have more rows than the launch has CTAs for, so a CTA goes on with
// the next ones.  Where none does the loop is left out: the kernel by rows then takes 32
// registers for 48, so that more of the CTAs that find no unit run at once (one token
// of 32/8 heads of 128 over 2K: 11.9 us, 12.2 with the loop; a chunk of 1000 beside
// seven sequences 104.9 and 105.2).

template <int HD, bool F16, bool MORE>
__global__ void __launch_bounds__(kMergeWarps * 32) unit_merge_kernel(const MergeParams p) {
  constexpr int NP = HD / 4 / kMergeWarps;   // 4-dim pieces of a warp
  constexpr int kRow = HD / 2 + 4;           // words of a staged row (spread over the banks)
  __shared__ __align__(16) uint32_t out_s[kMergeRows][kRow];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const MergeUnit mu = p.merge[c];
  if (mu.parts == 0) return;
  const int g = p.group, tt = kUnitTile / g;
  const int rows = mu.ntok > tt ? kUnitTile + (mu.ntok - tt) * g : mu.ntok * g;
  for (int row0 = blockIdx.y * kMergeRows; row0 < rows; row0 += gridDim.y * kMergeRows) {
    const int row = row0 + lane;  // row of the partial
    const int tr = row % kUnitTile, tok = row / kUnitTile * tt + tr / g;
    const bool mine = tr < tt * g && tok < mu.ntok;  // else no token's row
    auto slot = [&](int part) { return (size_t)(part == 0 ? 2 * c + 1 : 2 * (c + part)); };
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    const float4* po = reinterpret_cast<const float4*>(p.part_o) + (size_t)(warp * NP) * p.rows + row;
    float m = -INFINITY, l = 0.f, acc[NP][4];
#pragma unroll
    for (int k = 0; k < NP; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
    if (mine) {
      for (int i0 = 0; i0 < mu.parts; i0 += kMergeBatch) {
        float2 x[kMergeBatch];
        float4 v[kMergeBatch][NP];
#pragma unroll
        for (int i = 0; i < kMergeBatch; ++i)
          if (i0 + i < mu.parts) {
            x[i] = __ldcg(&ml[slot(i0 + i) * p.rows + row]);
#pragma unroll
            for (int k = 0; k < NP; ++k) v[i][k] = __ldcg(po + (slot(i0 + i) * (HD / 4) + k) * p.rows);
          }
#pragma unroll
        for (int i = 0; i < kMergeBatch; ++i) {
          if (i0 + i >= mu.parts) break;
          const float mn = fmaxf(m, x[i].x), ref = safe_ref(mn);
          const float f = ex2(m - ref), w = ex2(x[i].x - ref);
          l = fmaf(l, f, w * x[i].y);
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            const float y[4] = {v[i][k].x, v[i][k].y, v[i][k].z, v[i][k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[k][e] = fmaf(w, y[e], acc[k][e] * f);
          }
          m = mn;
        }
      }
    }
    const float inv = l > 0.f ? 1.f / l : l == l ? 0.f : NAN;
    if (MORE && row0 >= gridDim.y * kMergeRows) __syncthreads();  // the rows before are read
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      out_s[lane][(warp * NP + k) * 2] = pack2<F16>(acc[k][0] * inv, acc[k][1] * inv);
      out_s[lane][(warp * NP + k) * 2 + 1] = pack2<F16>(acc[k][2] * inv, acc[k][3] * inv);
    }
    if (mine && warp == 0 && p.lse)
      p.lse[(int64_t)(mu.tok0 + tok) * p.num_q_heads + mu.h * g + tr % g] =
          (m + log2f(l)) * 0.6931471805599453f;
    __syncthreads();
    constexpr int kPieces = HD / 8;  // 16-byte pieces of a row
    for (int i = threadIdx.x; i < kMergeRows * kPieces; i += kMergeWarps * 32) {
      const int r = row0 + i / kPieces, rr = r % kUnitTile, tk = r / kUnitTile * tt + rr / g;
      if (rr >= tt * g || tk >= mu.ntok) continue;
      *reinterpret_cast<uint4*>(p.out + (int64_t)(mu.tok0 + tk) * p.out_stride +
                                (int64_t)(mu.h * g + rr % g) * HD + (i % kPieces) * 8) =
          *reinterpret_cast<const uint4*>(&out_s[i / kPieces][(i % kPieces) * 4]);
    }
    if (!MORE) break;
  }
}

// The same for calls of few rows (single tokens), whose units have many parts:
// a CTA per row at a time, its warps over the parts, every load in flight at once.
template <int HD, bool F16, bool MORE>
__global__ void __launch_bounds__(kMergeWarps * 32) unit_merge_row_kernel(const MergeParams p) {
  constexpr int E = HD / 32;
  __shared__ float acc_s[kMergeWarps][HD], l_s[kMergeWarps], m_s[kMergeWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const MergeUnit mu = p.merge[c];
  const int g = p.group;
  if (mu.parts == 0) return;
  auto slot = [&](int part) { return (size_t)(part == 0 ? 2 * c + 1 : 2 * (c + part)); };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  for (int row = blockIdx.y; row < mu.ntok * g; row += gridDim.y) {
    if (MORE && row >= gridDim.y) __syncthreads();  // the row before is read
    float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < mu.parts; i += kMergeWarps) {
      const float2 x = __ldcg(&ml[slot(i) * p.rows + row]);
      const float* src = p.part_o + ((slot(i) * (HD / 4) + lane * E / 4) * p.rows + row) * 4 + lane * E % 4;
      float v[E];
      if (E == 4) {
        const float4 y = __ldcg(reinterpret_cast<const float4*>(src));
        v[0] = y.x, v[1] = y.y, v[E - 2] = y.z, v[E - 1] = y.w;
      } else {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(src));
        v[0] = y.x, v[1] = y.y;
      }
      const float mn = fmaxf(m, x.x), ref = safe_ref(mn);
      const float f = ex2(m - ref), w = ex2(x.x - ref);
      // a part without weight is passed over if all of it is finite (one token of
      // 8 heads over 2K: 9.9 us for the call, 10.4 when none is)
      bool finite = fabsf(x.y) < INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) finite &= fabsf(v[e]) < INFINITY;
      l *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] *= f;
      if (w != 0.f || !finite) {
        l += w * x.y;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, v[e], acc[e]);
      }
      m = mn;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc_s[warp][lane * E + e] = acc[e];
    if (lane == 0) {
      l_s[warp] = l;
      m_s[warp] = m;
    }
    __syncthreads();
    if (threadIdx.x < HD / 2) {
      float m_all = m_s[0];
#pragma unroll
      for (int i = 1; i < kMergeWarps; ++i) m_all = fmaxf(m_all, m_s[i]);
      const float ref = safe_ref(m_all);
      float l_all = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
      for (int i = 0; i < kMergeWarps; ++i) {
        const float w = ex2(m_s[i] - ref);
        l_all += w * l_s[i];
        o0 = fmaf(w, acc_s[i][2 * threadIdx.x], o0);
        o1 = fmaf(w, acc_s[i][2 * threadIdx.x + 1], o1);
      }
      const float inv = l_all > 0.f ? 1.f / l_all : l_all == l_all ? 0.f : NAN;
      const int t = mu.tok0 + row / g, qh = mu.h * g + row % g;
      *reinterpret_cast<uint32_t*>(p.out + t * p.out_stride + (int64_t)qh * HD + 2 * threadIdx.x) =
          pack2<F16>(o0 * inv, o1 * inv);
      if (p.lse && threadIdx.x == 0)
        p.lse[(int64_t)t * p.num_q_heads + qh] = (m_all + log2f(l_all)) * 0.6931471805599453f;
    }
    if (!MORE) break;
  }
}

// Launches the merge behind a kernel whose calls have at most `rows` rows of a
// unit to merge (all of the call's rows of a KV head), of which a unit is expected
// to have `usual` (a CTA takes 32, and more where a unit has them).
template <int HD, bool F16>
cudaError_t launch_unit_merge(cudaLaunchConfig_t cfg, int grid, long long rows, long long usual,
                              const MergeParams& p) {
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  // Up to 32 rows: a CTA per row, whose units have many parts (one token of 8
  // heads over 2K: 9.9 us for the call, 12.7 with the other merge; eight tokens
  // over 16K - 64K: the same).  Units of several sequences have fewer, so that most of
  // 32 CTAs a unit would find no row: 16, or as many as expected, take two where one
  // sequence has them all (a token each of 8 sequences to 6404 states, 32/8 heads:
  // 30.6 us, 33.0 with 32; eight tokens of one 19.6 and 19.2).  More rows mean fewer parts,
  // and a CTA takes 32.
  if (rows <= 32) {
    const long long some = usual > 16 ? usual : 16;
    cfg.gridDim = dim3(grid, (int)(some < rows ? some : rows));
    return some < rows ? cudaLaunchKernelEx(&cfg, unit_merge_row_kernel<HD, F16, true>, p)
                       : cudaLaunchKernelEx(&cfg, unit_merge_row_kernel<HD, F16, false>, p);
  }
  const int most = p.rows == kUnitTile ? (int)rows : p.rows;
  cfg.gridDim = dim3(grid, ((usual < most ? (int)usual : most) + kMergeRows - 1) / kMergeRows);
  return usual < most ? cudaLaunchKernelEx(&cfg, unit_merge_kernel<HD, F16, true>, p)
                      : cudaLaunchKernelEx(&cfg, unit_merge_kernel<HD, F16, false>, p);
}

}  // namespace
}  // namespace vg
