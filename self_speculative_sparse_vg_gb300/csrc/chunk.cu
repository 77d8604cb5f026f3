// Attention of a chunk of new tokens over the paged cache (sm_103a).
//
// Row (token i of sequence b, query head q) sits at position
// P = kv_len_b - n_b + i and computes softmax(scale q . k_j) v over the
// positions j <= P.
//
// Design (one persistent CTA per SM):
//  * A unit is two 128-row tiles of one KV head of one sequence: the
//    floor(128 / g) tokens of a tile times their g query heads, packed token
//    by token, so K and V are read once for all heads of the group.  Its work
//    is the 128-position tiles up to its last row's position.
//  * All units' tiles form one line (sequence, KV head, row tiles; weighted by
//    what they cost), cut into equal shares, one per CTA: any mix of long
//    prompts and single tokens is balanced to a tile.  KV heads outrank row
//    tiles on the line so that the
//    CTAs of a long prompt stream the same few heads, which L2 holds.  A unit
//    that a cut divides leaves fp32 partials (m, l, O) in the workspace; a
//    small chained kernel merges them.  Every CTA finds its own share from
//    the lengths, so the call needs no plan from the host.
//  * Two softmax warpgroups, one row per thread, each with its own S (128
//    fp32 columns of tensor memory, P written back over it as bf16) and O:
//    while one does its exponentials the tensor cores run the other's
//    O += P V and S = Q K^T.  A unit of one row tile (single tokens) gives
//    both warpgroups the same rows and alternate position tiles; O's rows are
//    in the same tensor-memory lanes, so their merge needs only (m, l) from
//    the other side.
//  * S(t + 1) of a warpgroup is issued after its P(t) V, so its arrival also
//    says that O may be rescaled.  The exponent reference moves only when a
//    row maximum grows by more than 2^8: P stays below 2^8 times a weight of
//    one, exact range in bf16 and far from the fp32 range in l and O.
//  * A producer warp streams K and V tiles (TMA, 128-byte swizzle) through a
//    ring of stages and publishes the CTA's units; one warp issues every
//    tensor-core operation (a warp for each warpgroup was slower: the two
//    streams of products then mix on the tensor cores and finish together).  A page of a head is one TMA box: at about 100
//    cycles a box, two boxes a page (one per 64-dim block) held a CTA to one
//    64 KB tile of K and V in 3300 cycles.
//  * Position tiles that some row of the unit does not attend in full (the
//    diagonal and the end of the cache) pass through two checking warps
//    first: a weight of zero times a NaN or an infinity in V would still
//    spoil the row, so they zero V past the length and take non-finite values
//    out of the tile, noting per dimension the first position of each kind;
//    rows that attend it get it back at the end.
#include <limits.h>
#include <math.h>

#include "units.cuh"
#include "vg_device.cuh"
#include "vg_host.h"

namespace vg {
namespace {

constexpr int kTile = kUnitTile;       // positions of a KV tile, rows of a row tile
constexpr int kPagesPerTile = kTile / kPageSize;
constexpr int kChunkThreads = 384;
constexpr int kProducer = 8, kMma = 9, kChecker = 10;  // warps (0..7: softmax; two checkers)
constexpr int kMaxBatch = 4096;
constexpr float kRescale = 8.f;        // log2 growth of a row maximum that moves the reference
constexpr int kRowsMax = 2 * kTile;    // rows of a unit
// Costs on the line that the CTAs share: a position tile of a unit with two row
// tiles or with one, and what a unit costs beside its tiles (Q, first scores,
// epilogue).  Measured: 2900, 2400 and 7000 - 10000 cycles.
constexpr int kTwoCost = 5, kOneCost = 4, kUnitCost = 15;

struct ChunkParams {
  const int32_t* page_table;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  __nv_bfloat16* out;
  float* lse;
  float* part_o;      // [grid][2][HD / 4][rows][4]
  float* part_ml;     // [grid][2][rows][2]
  MergeUnit* merge;   // [grid]
  int32_t* error_flag;
  int64_t out_stride;
  uint64_t wait_ns;    // a longer wait is reported
  int polls;           // polls of a wait between two looks at the timer
  float scale_log2;
  int batch, num_tokens, num_q_heads, num_kv_heads, group, num_pages, width, rows;
};

// A unit of work as the CTA's roles see it.
struct Unit {
  int tok0, ntok;     // first token row, tokens (at most 2 * tile_tokens)
  int pos0;           // position of the first token (may be negative)
  int len;            // positions of the sequence
  int h;
  int kt0, kt1;       // position tiles of this CTA; kt0 == kt1: no more units
  int n0;             // position tiles of the first row tile
  int two;            // two row tiles (else one, position tiles alternate)
  int part;           // partial slot of the workspace, -1: writes its rows
};

template <int HD>
struct ChunkLayout {
  static constexpr int kBlocks = HD / 64;              // 64-dim blocks of a row
  // Q: [block][row][128 bytes].  K and V: [8-position group][block][8][128
  // bytes], the order in which one TMA box brings a page.
  static constexpr int kQBlockBytes = kTile * 128;
  static constexpr int kGroupBytes = kBlocks * 1024;
  static constexpr int kPageBytes = 2 * kGroupBytes;
  static constexpr int kStageBytes = kPagesPerTile * kPageBytes;
  static constexpr int kStages = HD == 128 ? 5 : 10;
  static constexpr int kQBytes = kStageBytes;          // one row tile
  static constexpr int kRing = 2 * kQBytes;
  static constexpr int kSmall = kRing + kStages * kStageBytes;
  // small area: barriers, units, (m, l) exchange, non-finite notes
  static constexpr int kBars = kSmall;
  static constexpr int kBarCount = 3 * kStages + 15;
  static constexpr int kUnits = kBars + (kBarCount + 1) / 2 * 16;
  static constexpr int kFlags = kUnits + 2 * 48;
  static constexpr int kNotes = kFlags + 32;
  static constexpr int kMl = kNotes + 2 * 3 * HD * 2;
  static constexpr int kBytes = kMl + kTile * 8;
  static constexpr int kSCol = 0, kOCol = 2 * kTile;

  // Byte offset of 16-byte piece `ch` of position `row` in a K or V tile.
  static __device__ __forceinline__ uint32_t kv_offset(int row, int ch) {
    return (row >> 3) * kGroupBytes + (ch >> 3) * 1024 + (row & 7) * 128 + (((ch & 7) ^ (row & 7)) << 4);
  }
};
static_assert(ChunkLayout<128>::kBytes <= 227 * 1024 && ChunkLayout<64>::kBytes <= 227 * 1024, "");
static_assert(sizeof(Unit) <= 48, "");

struct ChunkBars {
  // Ring stages.  `landed`: a V tile that is to be checked has landed; `full`:
  // a tile may be read (it has landed, or it was checked); `empty`: its
  // products are done.  Whoever waits on `full` or `landed`
  // waits for every phase of it, so that a parity names one phase.
  uint64_t *full, *landed, *empty;         // [stages]
  uint64_t *sfull, *pfull, *ofull;         // [2]: S, P, all of O of a warpgroup
  uint64_t *qfull, *qempty, *ufull, *uempty, *xfull, *xdone, *drain;
};

__device__ __forceinline__ ChunkBars chunk_bars(uint64_t* b, int stages) {
  ChunkBars r;
  r.full = b;
  r.landed = b + stages;
  r.empty = b + 2 * stages;
  b += 3 * stages;
  r.sfull = b;
  r.pfull = b + 2;
  r.ofull = b + 4;
  r.ufull = b + 6;
  r.uempty = b + 8;
  r.qfull = b + 10;
  r.qempty = b + 11;
  r.xfull = b + 12;
  r.xdone = b + 13;
  r.drain = b + 14;
  return r;
}

// Position tiles up to position `pos`, at least one (a unit whose rows attend
// nothing still writes them).
__device__ __forceinline__ int tiles_to(int pos) { return pos < 0 ? 1 : pos / kTile + 1; }

// Rows and lengths of sequence b; n = 0 when it has none or makes no sense.
__device__ __forceinline__ bool sequence_of(const ChunkParams& p, int b, int& q0, int& n, int& len) {
  q0 = p.cu_q[b];
  const int q1 = p.cu_q[b + 1];
  len = p.kv_lens[b];
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= p.num_tokens && len >= 0 && len <= p.width * kPageSize;
  n = ok ? q1 - q0 : 0;
  return ok;
}

__device__ __forceinline__ int tile_cost(int ntok, int tu) { return 2 * ntok > tu ? kTwoCost : kOneCost; }

// Length on the line of row-tile pair `rt` (tu tokens each) of a sequence: its
// overhead, then its position tiles.
__device__ __forceinline__ long long unit_length(int n, int len, int tu, int rt) {
  const int ntok = min(tu, n - rt * tu);
  return kUnitCost + (long long)tile_cost(ntok, tu) * tiles_to(len - n + rt * tu + ntok - 1);
}

// A unit's position tiles that end before offset y of its length; a CTA whose
// share holds [y0, y1) of it takes tiles [tiles_before(y0), tiles_before(y1)).
__device__ __forceinline__ int tiles_before(long long y, int cost) {
  return y <= kUnitCost ? 0 : (int)((y - kUnitCost) / cost);
}

// Whether some row of the unit does not attend all of tile kt (its first row
// ends before the tile does): V is then checked.
__device__ __forceinline__ bool checked_tile(int pos0, int kt) {
  return kt * kTile + kTile - 1 > pos0;
}

// Non-zero when one of two packed bf16 is an infinity or a NaN (an exponent of
// ones: adding the exponent's lowest bit carries out of it).
__device__ __forceinline__ uint32_t not_finite(uint32_t v) {
  return ((v & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// note_flags[slot * 2 + half]: the unit in this slot has notes of that half of
// the dimensions.  The producer clears both before it publishes the unit, a
// checking warp sets its own once its notes are laid out.  A row tile may end
// while later tiles are still checked, so the store and the load are ordered.
__device__ __forceinline__ void raise_notes(int* flag) {
  asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(smem_u32(flag)), "r"(1) : "memory");
}
__device__ __forceinline__ bool has_notes(const int* flag) {
  uint32_t v;
  asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(flag)) : "memory");
  return v != 0;
}

// The non-finite value that dimension c of a row attends, or 0: rel = the row's
// token within the unit, notes = first token distance of a NaN, +inf and -inf.
template <int HD>
__device__ __forceinline__ float noted(const uint16_t* notes, int c, int rel) {
  const bool n = rel >= notes[c], pi = rel >= notes[HD + c], ni = rel >= notes[2 * HD + c];
  if (n || (pi && ni)) return NAN;
  return pi ? INFINITY : ni ? -INFINITY : 0.f;
}

// ---------------------------------------------------------------- softmax
// One warp of warpgroup S (0 or 1) through all units of the CTA.
template <int HD>
__device__ __forceinline__ void softmax_role(const ChunkParams& p, const ChunkBars& bars,
                                             const Unit* units, const int* note_flags,
                                             const uint16_t* notes_s, float2* ml_s, uint32_t tmem,
                                             int wg, int warp, int lane) {
  using Lay = ChunkLayout<HD>;
  const int g = p.group, tt = kTile / g;
  const int r = (warp & 3) * 32 + lane;  // row within the tile
  const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  const uint32_t scol = trow + Lay::kSCol + wg * kTile;
  const uint32_t ocol = trow + Lay::kOCol + wg * HD;
  const int tok_r = r / g, head_r = r - tok_r * g;
  uint32_t sc = 0, oc = 0, xc = 0;
  for (uint32_t u = 0;; ++u) {
    const int slot = u & 1;
    if (!wait_phase_warp(&bars.ufull[slot], (u >> 1) & 1, p)) return;
    const Unit un = units[slot];
    if (un.kt0 == un.kt1) return;
    const int tok = un.two ? wg * tt + tok_r : tok_r;       // token within the unit
    const bool valid = tok_r < tt && tok < un.ntok;
    const int lim = valid ? un.pos0 + tok : -1;             // last attended position
    const bool rows = __any_sync(0xffffffffu, valid);       // a warp without rows only keeps step
    const int first = un.two ? un.kt0 : un.kt0 + wg;
    const int step = un.two ? 1 : 2;
    const int end = un.two && wg == 0 ? min(un.kt1, un.n0) : un.kt1;
    float m_used = -INFINITY, lsum = 0.f;
    for (int kt = first; kt < end; kt += step) {
      if (!wait_phase_warp(&bars.sfull[wg], sc & 1, p)) return;
      ++sc;
      tc_fence_after();
      if (rows) {
        uint32_t s[2][64];
        tmem_ld64(scol, s[0]);
        tmem_ld64(scol + 64, s[1]);
        const int rem = lim - kt * kTile;  // last attended column
        if (!__all_sync(0xffffffffu, rem >= kTile - 1 || !valid)) {
#pragma unroll
          for (int w = 0; w < kTile / 32; ++w) {
            const int last = rem - 32 * w;  // last attended column of these 32
            const uint32_t keep = last >= 31 ? 0xffffffffu : last < 0 ? 0u : (2u << last) - 1u;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((keep >> j) & 1u)) s[w >> 1][(w & 1) * 32 + j] = 0xff800000u;  // -inf
          }
        }
        float mx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(__uint_as_float(s[0][j]), __uint_as_float(s[1][j]));
#pragma unroll
        for (int j = 4; j < 64; ++j)
          mx[j & 3] = max3(mx[j & 3], __uint_as_float(s[0][j]), __uint_as_float(s[1][j]));
        // scale > 0: the maximum commutes with it
        const float m_tile = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * p.scale_log2;
        const bool need = m_tile > m_used + kRescale;
        if (__any_sync(0xffffffffu, need)) {
          const float mn = need ? m_tile : m_used;
          if (kt != first) {  // P(t - 1) V is done: S(t) was issued after it
            const float corr = mn == -INFINITY ? 1.f : ex2(m_used - mn);
            lsum *= corr;
#pragma unroll 1
            for (int c = 0; c < HD; c += 16) {
              float o[16];
              tmem_ld16(ocol + c, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] *= corr;
              tmem_st16(ocol + c, o);
            }
            tmem_st_wait();
          }
          m_used = mn;
        }
        // P = 2^(s scale - m).  (Handing it over in two halves, so that the
        // product with V starts earlier, changed nothing.)
        const float nref = -safe_ref(m_used);
        const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), nref2 = pair(nref, nref);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float2 x = unpair(fma2(pair(__uint_as_float(s[h][2 * j]), __uint_as_float(s[h][2 * j + 1])), scale2, nref2));
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            pk[j] = pack_bf16(x.x, x.y);
            s[h][2 * j] = __float_as_uint(x.x);
            s[h][2 * j + 1] = __float_as_uint(x.y);
          }
          tmem_st32u(scol + h * 32, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.pfull[wg]);
        // the row sum, off the tensor cores' path
        uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 64; ++j) {
          const uint32_t* x = &s[j >> 5][(j & 31) * 2];
          acc[j & 3] = add2(acc[j & 3], pair(__uint_as_float(x[0]), __uint_as_float(x[1])));
        }
        const float2 sum = unpair(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])));
        lsum += sum.x + sum.y;
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.pfull[wg]);
      }
    }
    // -------- epilogue
    const bool has = end > first;
    if (has) {
      if (!wait_phase_warp(&bars.ofull[wg], oc & 1, p)) return;
      ++oc;
      tc_fence_after();
    }
    const bool other = !un.two && un.kt0 + 1 < un.kt1;  // alternate tiles: both sides have O
    float w_own = 1.f, w_other = 0.f, m_all = m_used, l_all = lsum;
    if (other) {
      if (wg == 1) {
        ml_s[r] = make_float2(m_used, lsum);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.xfull);
      } else {
        if (!wait_phase_warp(bars.xfull, xc & 1, p)) return;
        tc_fence_after();
        const float2 o = ml_s[r];
        m_all = fmaxf(m_used, o.x);
        const float ref = safe_ref(m_all);
        w_own = ex2(m_used - ref);
        w_other = ex2(o.x - ref);
        l_all = w_own * lsum + w_other * o.y;
      }
    }
    if (rows && (un.two || wg == 0)) {
      const uint16_t* notes = notes_s + slot * 3 * HD;
      const bool direct = un.part < 0;
      const int t = un.tok0 + tok, qh = un.h * g + head_r;
      const int prow = (un.two ? wg * kTile : 0) + r;       // row of the partial
      const float inv = direct ? (l_all > 0.f ? 1.f / l_all : l_all == l_all ? 0.f : NAN) : 1.f;
      const float f_own = has ? w_own * inv : 0.f, f_other = w_other * inv;
      const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_stride * 2)) & 31) == 0;
#pragma unroll 1
      for (int c = 0; c < HD; c += 64) {
        uint32_t o[64];
        if (has) {
          tmem_ld64(ocol + c, o);
#pragma unroll
          for (int j = 0; j < 64; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f_own);
        } else {
#pragma unroll
          for (int j = 0; j < 64; ++j) o[j] = 0u;
        }
        if (other) {
          uint32_t x[64];
          tmem_ld64(ocol + HD + c, x);
#pragma unroll
          for (int j = 0; j < 64; ++j)
            o[j] = __float_as_uint(fmaf(__uint_as_float(x[j]), f_other, __uint_as_float(o[j])));
        }
        if (valid && direct) {
          __nv_bfloat16* dst = p.out + t * p.out_stride + (int64_t)qh * HD + c;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = pack_bf16(__uint_as_float(o[16 * j + 2 * i]), __uint_as_float(o[16 * j + 2 * i + 1]));
            if (wide) {
              store32(dst + 16 * j, w);
            } else {
              *reinterpret_cast<uint4*>(dst + 16 * j) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(dst + 16 * j + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        } else if (valid) {
          // [4-dim piece][row][4]: a warp's rows are neighbours
          uint4* dst = reinterpret_cast<uint4*>(p.part_o) + ((size_t)un.part * (HD / 4) + c / 4) * p.rows + prow;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            dst[(size_t)j * p.rows] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
        __syncwarp();
      }
      const bool noted_lo = has_notes(&note_flags[slot * 2]), noted_hi = has_notes(&note_flags[slot * 2 + 1]);
      if (valid && (noted_lo || noted_hi)) {
        // rows that attend a non-finite value of a checked tile: added to what
        // this thread has just stored, which may hold another from a tile that
        // was not checked, or a NaN of the row's scores
#pragma unroll 1
        for (int c = 0; c < HD; ++c) {
          if (!(c < HD / 2 ? noted_lo : noted_hi)) continue;
          const float x = noted<HD>(notes, c, tok);
          if (x == 0.f) continue;
          if (direct) {
            __nv_bfloat16* e = p.out + t * p.out_stride + (int64_t)qh * HD + c;
            *e = __float2bfloat16(__bfloat162float(*e) + x);
          } else {
            p.part_o[(((size_t)un.part * (HD / 4) + c / 4) * p.rows + prow) * 4 + c % 4] += x;
          }
        }
      }
      if (valid && direct && p.lse)
        p.lse[(int64_t)t * p.num_q_heads + qh] = (m_all + log2f(l_all)) * 0.6931471805599453f;
      if (valid && !direct)
        reinterpret_cast<float2*>(p.part_ml)[(size_t)un.part * p.rows + prow] = make_float2(m_all, l_all);
    }
    if (other) {
      if (wg == 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars.xdone);
      } else if (!wait_phase_warp(bars.xdone, xc & 1, p)) {
        return;
      }
      ++xc;
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.uempty[slot]);
  }
}

// ------------------------------------------------------- tensor-core issue
// The warp runs in step (every value it uses is the same in all lanes) and an
// elected lane issues.
template <int HD>
struct MmaIssuer {
  using Lay = ChunkLayout<HD>;
  const ChunkBars& bars;
  uint32_t tmem, ring_lo, q_lo, v_lo;  // low descriptor words of stage 0 and of Q
  static constexpr uint32_t kIdQk = umma_idesc_bf16(kTile, kTile, 0, 0);
  static constexpr uint32_t kIdPv = umma_idesc_bf16(kTile, HD, 0, 1);
  static constexpr uint32_t kHiQ = umma_desc_hi(1024), kHiKv = umma_desc_hi(Lay::kGroupBytes);

  // S of warpgroup `wg` = Q (row tile qt) K^T of the stage
  __device__ __forceinline__ void qk(int wg, int qt, uint32_t stage) {
    const uint32_t k = ring_lo + stage * (Lay::kStageBytes >> 4);
    const uint32_t q = q_lo + qt * (Lay::kQBytes >> 4);
#pragma unroll
    for (int ks = 0; ks < HD / 16; ++ks) {
      const int block = ks >> 2, in = (ks & 3) * 32;
      umma_bf16_elect(tmem + Lay::kSCol + wg * kTile, q + ((block * Lay::kQBlockBytes + in) >> 4), kHiQ,
                      k + ((block * 1024 + in) >> 4), kHiKv, kIdQk, ks > 0);
    }
    umma_commit_elect(&bars.sfull[wg]);
  }
  // O of warpgroup `wg` (+)= P V of the stage
  __device__ __forceinline__ void pv(int wg, uint32_t stage, bool accumulate) {
    const uint32_t v = v_lo + stage * (Lay::kStageBytes >> 4);
#pragma unroll
    for (int ks = 0; ks < kTile / 16; ++ks)
      umma_bf16_ts_elect(tmem + Lay::kOCol + wg * HD, tmem + Lay::kSCol + wg * kTile + ks * 8,
                         v + ks * (Lay::kPageBytes >> 4), kHiKv, kIdPv, accumulate || ks > 0);
  }
};

template <int HD>
__device__ __forceinline__ bool mma_role(const ChunkParams& p, const ChunkBars& bars,
                                         const Unit* units, uint32_t tmem, uint32_t ring, uint32_t q,
                                         int lane) {
  using Lay = ChunkLayout<HD>;
  constexpr uint32_t NST = Lay::kStages;
  MmaIssuer<HD> mma{bars, tmem, umma_desc_lo(ring, 16), umma_desc_lo(q, 16),
                    umma_desc_lo(ring, 1024)};
  uint32_t pc = 0;            // parities of the warpgroups' next P
  // next K's and V's ring stage and parity; entries are K(0), V(0), K(1) ...
  uint32_t sk = 0, pk = 0, sv = 1, pv = 0;
  auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_phase_warp(bar, parity, p); };
  auto next = [](uint32_t& st, uint32_t& par) {
    st += 2;
    if (st >= NST) {
      st -= NST;
      par ^= 1;
    }
  };
  // O(wg) (+)= P V
  auto pv_product = [&](int wg, uint32_t st, bool accumulate) {
    const uint32_t par = (pc >> wg) & 1;
    pc ^= 1u << wg;
    if (!wait_phase_warp(&bars.pfull[wg], par, p)) return false;
    tc_fence_after();
    mma.pv(wg, st, accumulate);
    return true;
  };
  for (uint32_t u = 0;; ++u) {
    const int slot = u & 1;
    if (!wait_phase_warp(&bars.ufull[slot], (u >> 1) & 1, p)) return false;
    const int kt0 = same(units[slot].kt0), kt1 = same(units[slot].kt1), n0 = same(units[slot].n0);
    const int two = same(units[slot].two);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.uempty[slot]);
    if (kt0 == kt1) return true;
    if (!wait_phase_warp(bars.qfull, u & 1, p)) return false;
    const int n = kt1 - kt0;
    if (two) {
      const int e0 = min(kt1, n0) - kt0;  // tiles of the first row tile
      if (!wait(&bars.full[sk], pk)) return false;
      tc_fence_after();
      if (e0 > 0) mma.qk(0, 0, sk);
      mma.qk(1, 1, sk);
      umma_commit_elect(&bars.empty[sk]);
      if (n == 1) umma_commit_elect(bars.qempty);
      next(sk, pk);
      for (int j = 0; j < n; ++j) {
        const bool more = j + 1 < n;
        // the tiles are waited for first, while the warpgroups are at P(j)
        if (!wait(&bars.full[sv], pv) || (more && !wait(&bars.full[sk], pk))) return false;
        // (one copy of this code for both warpgroups: with two the kernel was
        // 6 % slower, its roles share the instruction cache)
#pragma unroll 1
        for (int wg = 0; wg < 2; ++wg) {
          const int e = wg ? n : e0;
          if (j >= e) continue;
          if (!pv_product(wg, sv, j > 0)) return false;
          if (j + 1 < e)
            mma.qk(wg, wg, sk);
          else
            umma_commit_elect(&bars.ofull[wg]);
        }
        umma_commit_elect(&bars.empty[sv]);
        if (more) {
          umma_commit_elect(&bars.empty[sk]);
          if (j + 2 == n) umma_commit_elect(bars.qempty);
          next(sk, pk);
        }
        next(sv, pv);
      }
    } else {
      for (int j = 0; j < min(n, 2); ++j) {
        if (!wait(&bars.full[sk], pk)) return false;
        tc_fence_after();
        mma.qk(j, 0, sk);
        umma_commit_elect(&bars.empty[sk]);
        next(sk, pk);
      }
      if (n <= 2) umma_commit_elect(bars.qempty);
      for (int j = 0; j < n; ++j) {
        const int wg = j & 1;
        if (!wait(&bars.full[sv], pv) || !pv_product(wg, sv, j > 1)) return false;
        if (j >= n - 2) umma_commit_elect(&bars.ofull[wg]);
        umma_commit_elect(&bars.empty[sv]);
        next(sv, pv);
        if (j + 2 < n) {
          // only now: a stream from HBM is behind, and V(j)'s stage is wanted
          if (!wait(&bars.full[sk], pk)) return false;
          tc_fence_after();
          mma.qk(wg, 0, sk);
          umma_commit_elect(&bars.empty[sk]);
          if (j + 3 == n) umma_commit_elect(bars.qempty);
          next(sk, pk);
        }
      }
    }
  }
}

// ------------------------------------------------------------ V checks
// Warp `half` of two owns half of the dimensions of every checked V tile.
template <int HD>
__device__ __forceinline__ void check_role(const ChunkParams& p, const ChunkBars& bars,
                                           const Unit* units, int* note_flags, uint16_t* notes_s,
                                           uint8_t* ring, int half, int lane) {
  using Lay = ChunkLayout<HD>;
  constexpr int NST = Lay::kStages;
  constexpr int CPW = HD / 16;       // 16-byte pieces of a row per warp
  constexpr int RPI = 32 / CPW;      // rows per pass
  uint32_t tiles = 0, landed = 0;
  for (uint32_t u = 0;; ++u) {
    const int slot = u & 1;
    if (!wait_phase_warp(&bars.ufull[slot], (u >> 1) & 1, p)) return;
    const Unit un = units[slot];
    if (un.kt0 == un.kt1) return;
    uint16_t* notes = notes_s + slot * 3 * HD;
    bool noting = false;
    // the checked tiles are the last ones, from the first that has a position
    // past the first row's
    const int from = max(un.kt0, un.pos0 < 0 ? 0 : (un.pos0 + 1) / kTile);
    for (int kt = from; kt < un.kt1; ++kt) {
      const uint32_t st = (2 * (tiles + kt - un.kt0) + 1) % NST;
      if (!wait_phase_warp(&bars.landed[st], (landed >> st) & 1, p)) return;
      landed ^= 1u << st;
      uint8_t* tile = ring + st * Lay::kStageBytes;
      // rows past the length are zeroed, those past the first row's position
      // looked at (earlier ones are attended by every row)
      const int last = min(un.len - kt * kTile, kTile);
      const int begin = max(un.pos0 + 1 - kt * kTile, 0);
      const int ch = half * CPW + lane % CPW, r = lane / CPW;  // piece of the row, row of the pass
      uint32_t bad = 0;
#pragma unroll 8
      for (int r0 = begin; r0 < last; r0 += RPI) {
        const uint4 v = *reinterpret_cast<const uint4*>(tile + Lay::kv_offset(min(r0 + r, last - 1), ch));
        bad |= not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w);
      }
#pragma unroll 4
      for (int r0 = max(last, 0); r0 < kTile; r0 += RPI)
        if (r0 + r < kTile)
          *reinterpret_cast<uint4*>(tile + Lay::kv_offset(r0 + r, ch)) = make_uint4(0u, 0u, 0u, 0u);
      if (__any_sync(0xffffffffu, bad != 0)) {
        if (!noting) {  // clear this warp's notes: no position sees them
          for (int c = lane; c < 3 * HD / 2; c += 32)
            notes[c / (HD / 2) * HD + half * (HD / 2) + c % (HD / 2)] = 0xffff;
          noting = true;
          __syncwarp();
          if (lane == 0) raise_notes(&note_flags[slot * 2 + half]);
        }
        __syncwarp();
        // a lane per dimension, rows in order
        for (int c = half * (HD / 2) + lane; c < (half + 1) * (HD / 2); c += 32) {
          for (int row = begin; row < last; ++row) {
            uint16_t* e = reinterpret_cast<uint16_t*>(tile + Lay::kv_offset(row, c >> 3)) + (c & 7);
            const uint16_t x = *e;
            if ((x & 0x7f80) != 0x7f80) continue;
            const int kind = (x & 0x7f) ? 0 : x & 0x8000 ? 2 : 1;
            const int rel = min(kt * kTile + row - un.pos0, 0xfffe);
            if (rel < notes[kind * HD + c]) notes[kind * HD + c] = (uint16_t)rel;
            *e = 0;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.full[st]);
    }
    tiles += un.kt1 - un.kt0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.uempty[slot]);
  }
}

// -------------------------------------------------------------- the CTA's share
struct Share {
  long long unit_at;  // line position where the first unit begins (perhaps before the share)
  long long x1;       // end of the share on the line
  long long share;    // its length
  int b, h, rt, kt0;
  int q0, n, len;     // the first unit's sequence
};

__device__ __forceinline__ int row_tiles(int n, int tu) {
  return (int)(((unsigned)n + (unsigned)tu - 1u) / (unsigned)tu);
}

// Length on the line of one KV head of the 32 sequences b0 .. b0 + 31, one per
// lane of a warp; seq = their first row, tokens and length.
__device__ __forceinline__ long long sequence_lengths(const ChunkParams& p, int b0, int tu, int lane,
                                                      int4& seq) {
  const int b = b0 + lane;
  int q0 = 0, n = 0, len = 0;
  if (b < p.batch && !sequence_of(p, b, q0, n, len) && blockIdx.x == 0)
    flag_error(p.error_flag, VG_DEVERR_LENGTH);
  seq = make_int4(q0, n, len, 0);
  const int nrt = row_tiles(n, tu);
  long long c = 0;
  if (nrt <= 4)
    for (int rt = 0; rt < nrt; ++rt) c += unit_length(n, len, tu, rt);
  uint32_t todo = __ballot_sync(0xffffffffu, nrt > 4);
  while (todo) {  // long sequences: a lane per row tile
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    const int sn = __shfl_sync(0xffffffffu, n, src), sl = __shfl_sync(0xffffffffu, len, src);
    const int sr = __shfl_sync(0xffffffffu, nrt, src);
    long long s = 0;
    for (int rt = lane; rt < sr; rt += 32) s += unit_length(sn, sl, tu, rt);
    // 64 bits in two reductions of 32
    const long long lo = __reduce_add_sync(0xffffffffu, (uint32_t)s & 0x3ffffffu);
    const long long hi = __reduce_add_sync(0xffffffffu, (uint32_t)(s >> 26));
    if (lane == src) c = (hi << 26) + lo;
  }
  return c;
}

// Batches of more than 32 sequences: the CTA's warps put every sequence's
// length into shared memory first.
struct SequenceTable {
  long long* length;
  int4* seq;
};

__device__ __forceinline__ void fill_sequence_table(const ChunkParams& p, const SequenceTable& tab) {
  const int lane = threadIdx.x & 31, tu = 2 * (kTile / p.group);
  for (int b0 = threadIdx.x - lane; b0 < p.batch; b0 += kChunkThreads) {
    int4 seq;
    const long long c = sequence_lengths(p, b0, tu, lane, seq);
    if (b0 + lane < p.batch) {
      tab.length[b0 + lane] = c;
      tab.seq[b0 + lane] = seq;
    }
  }
}

// Where the CTA's share of the line begins; found by one warp.  b < 0: no work.
__device__ __forceinline__ Share find_share(const ChunkParams& p, const SequenceTable& tab, int lane) {
  const int tu = 2 * (kTile / p.group);
  const bool small = p.batch <= 32;
  int4 seq = make_int4(0, 0, 0, 0);
  long long sum = 0, total = 0;  // running sum over the line, this lane's sequence included
  if (small) {
    sum = warp_inclusive_sum(sequence_lengths(p, 0, tu, lane, seq) * p.num_kv_heads, lane);
    total = __shfl_sync(0xffffffffu, sum, 31);
  } else {
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const bool in = b0 + lane < p.batch;
      sum = total + warp_inclusive_sum(in ? tab.length[b0 + lane] * p.num_kv_heads : 0, lane);
      if (in) tab.length[b0 + lane] = sum;
      total = __shfl_sync(0xffffffffu, sum, 31);
    }
    __syncwarp();
  }
  // at least one tile, so that every CTA inside a divided unit has a part of it
  const long long share = max(quotient(total + gridDim.x - 1, gridDim.x),
                              (long long)(p.rows == kTile ? kOneCost : kTwoCost));
  const long long x0 = share * blockIdx.x;
  Share s = {};
  s.share = share;
  s.x1 = min(total, x0 + share);
  s.b = -1;
  if (x0 >= total) return s;
  long long base = 0, end = 0;  // the sequence's part of the line
  if (small) {
    s.b = __ffs(__ballot_sync(0xffffffffu, sum > x0)) - 1;
    end = __shfl_sync(0xffffffffu, sum, s.b);
    base = __shfl_sync(0xffffffffu, sum, max(s.b - 1, 0));
    if (s.b == 0) base = 0;
    s.q0 = __shfl_sync(0xffffffffu, seq.x, s.b);
    s.n = __shfl_sync(0xffffffffu, seq.y, s.b);
    s.len = __shfl_sync(0xffffffffu, seq.z, s.b);
  } else {
    for (int b0 = 0; b0 < p.batch && s.b < 0; b0 += 32) {
      const uint32_t past = __ballot_sync(0xffffffffu, b0 + lane < p.batch && tab.length[b0 + lane] > x0);
      if (past) s.b = b0 + __ffs(past) - 1;
    }
    end = tab.length[s.b];
    base = s.b > 0 ? tab.length[s.b - 1] : 0;
    s.q0 = tab.seq[s.b].x;
    s.n = tab.seq[s.b].y;
    s.len = tab.seq[s.b].z;
  }
  const long long per_head = quotient(end - base, p.num_kv_heads);
  s.h = (int)quotient(x0 - base, per_head);
  const long long y = x0 - base - s.h * per_head;
  const int nrt = row_tiles(s.n, tu);
  long long before = 0;  // length of the row tiles before rt
  for (int rt0 = 0; rt0 < nrt; rt0 += 32) {
    const long long own = rt0 + lane < nrt ? unit_length(s.n, s.len, tu, rt0 + lane) : 0;
    const long long v = warp_inclusive_sum(own, lane);
    const uint32_t past = __ballot_sync(0xffffffffu, before + v > y);
    if (past) {
      const int l = __ffs(past) - 1;
      s.rt = rt0 + l;
      before += __shfl_sync(0xffffffffu, v - own, l);
      break;
    }
    before += __shfl_sync(0xffffffffu, v, 31);
  }
  s.kt0 = tiles_before(y - before, tile_cost(min(tu, s.n - s.rt * tu), tu));
  s.unit_at = x0 - (y - before);
  return s;
}

// ----------------------------------------------------------------- producer
// Walks the CTA's units, publishes them and streams their Q, K and V.  On a
// wait that was given up it stops, then waits (bounded) for its own copies.
template <int HD>
__device__ __forceinline__ void producer_role(const ChunkParams& p, const ChunkBars& bars,
                                              const Share& s, const CUtensorMap& tmq,
                                              const CUtensorMap& tmk, const CUtensorMap& tmv,
                                              Unit* units, int* note_flags, uint8_t* smem, int lane) {
  using Lay = ChunkLayout<HD>;
  constexpr int NST = Lay::kStages;
  const int g = p.group, tt = kTile / g, tu = 2 * tt;
  uint8_t* ring = smem + Lay::kRing;
  const int pi = lane & 7;
  int b = s.b, h = s.h, rt = s.rt, kt0 = s.kt0;
  long long at = s.unit_at;  // line position of the current unit's first tile
  int q0 = s.q0, n = s.n, len = s.len;
  uint32_t ri = 0, u = 0, on_landed = 0, landed = 0;  // bits: last load of a stage, its parity
  bool live = true, q_armed = false;
  MergeUnit cut = {};
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    int go = 1;
    if (lane == 0) go = wait_phase(bar, parity, p);
    return __shfl_sync(0xffffffffu, go, 0) != 0;
  };
  while (live) {
    const int ntok = min(tu, n - rt * tu), cost = tile_cost(ntok, tu);
    // its next position tile ends in the share
    const bool more = b >= 0 && at + kUnitCost + (long long)cost * (kt0 + 1) <= s.x1;
    const int slot = u & 1;
    if (u >= 2 && !wait(&bars.uempty[slot], ((u >> 1) - 1) & 1)) {
      live = false;
      break;
    }
    Unit un = {};
    if (more) {
      un.tok0 = q0 + rt * tu;
      un.ntok = ntok;
      un.pos0 = len - n + rt * tu;
      un.len = len;
      un.h = h;
      un.two = un.ntok > tt;
      un.n0 = tiles_to(un.pos0 + min(tt, un.ntok) - 1);
      const int tiles = tiles_to(un.pos0 + un.ntok - 1);
      un.kt0 = kt0;
      un.kt1 = min(tiles, tiles_before(s.x1 - at, cost));
      un.part = kt0 > 0 ? 2 * (int)blockIdx.x : un.kt1 < tiles ? 2 * (int)blockIdx.x + 1 : -1;
      at += kUnitCost + (long long)cost * tiles;  // the next unit's
      if (kt0 == 0 && un.kt1 < tiles) {
        cut.parts = (int)quotient(at - 1, s.share) - (int)blockIdx.x + 1;
        cut.tok0 = un.tok0;
        cut.ntok = un.ntok;
        cut.h = h;
      }
    }
    // page ids of four tiles at a time, one per lane (read here, looked at
    // where they are used)
    const int npages = (len + kPageSize - 1) / kPageSize;
    auto fetch = [&](int kt) -> int {
      const int lp = kt * kPagesPerTile + lane;
      return lp < npages && kt + (lane >> 3) < un.kt1 ? p.page_table[(size_t)b * p.width + lp] : INT_MIN;
    };
    auto page = [&](int id) -> int {
      if (id >= 0 && id < p.num_pages) return id;
      if (id != INT_MIN) flag_error(p.error_flag, VG_DEVERR_PAGE);
      return p.num_pages;  // past the pool: zeros
    };
    int ids_next = more ? fetch(kt0) : 0, ids = 0;
    q_armed = false;
    if (lane == 0) {
      units[slot] = un;
      note_flags[slot * 2] = note_flags[slot * 2 + 1] = 0;
      mbar_arrive(&bars.ufull[slot]);
    }
    __syncwarp();
    if (!more) break;
    for (int kt = un.kt0; kt < un.kt1 && live; ++kt) {
      const int w = (kt - un.kt0) & 3;
      if (w == 0) {
        ids = page(ids_next);
        ids_next = fetch(kt + 4);
      }
      const int id = __shfl_sync(0xffffffffu, ids, w * 8 + pi);
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        if (v == 1 && kt == un.kt0) {  // Q, once the unit before has made its scores
          if (u >= 1 && !wait(bars.qempty, (u - 1) & 1)) {
            live = false;
            break;
          }
          q_armed = true;
          if (lane == 0) {
            mbar_arrive_expect_tx(bars.qfull, (un.two ? 2 : 1) * Lay::kBlocks * tt * g * 128);
            for (int t = 0; t < (un.two ? 2 : 1); ++t)
              for (int x = 0; x < Lay::kBlocks; ++x)
                tma_load_3d(smem + t * Lay::kQBytes + x * Lay::kQBlockBytes, &tmq, bars.qfull, x * 64,
                            h * g, un.tok0 + t * tt);
          }
          __syncwarp();
        }
        const uint32_t st = ri % NST;
        if (ri >= NST && !wait(&bars.empty[st], ((ri / NST) - 1) & 1)) {
          live = false;
          break;
        }
        uint64_t* bar = &(v && checked_tile(un.pos0, kt) ? bars.landed : bars.full)[st];
        if (lane == 0) {
          if (bar == &bars.full[st]) mbar_arrive(bar);  // for the second checker
          mbar_arrive_expect_tx(bar, Lay::kStageBytes);
        }
        __syncwarp();
        if (lane < kPagesPerTile)
          tma_load_4d(ring + st * Lay::kStageBytes + pi * Lay::kPageBytes, v ? &tmv : &tmk, bar, 0, 0,
                      0, (id * p.num_kv_heads + h) * 2);
        __syncwarp();
        on_landed &= ~(1u << st);
        if (bar == &bars.landed[st]) {
          on_landed |= 1u << st;
          landed ^= 1u << st;
        }
        ++ri;
      }
    }
    ++u;
    kt0 = 0;
    if (++rt * tu >= n) {
      rt = 0;
      if (++h == p.num_kv_heads) {
        h = 0;
        do {
          if (++b >= p.batch) break;
          sequence_of(p, b, q0, n, len);
        } while (n == 0);
      }
    }
  }
  if (lane == 0) {
    p.merge[blockIdx.x] = cut;
    if (!live) {
      for (uint32_t i = ri > NST ? ri - NST : 0; i < ri; ++i) {
        const uint32_t st = i % NST;
        if ((on_landed >> st) & 1)
          mbar_wait(&bars.landed[st], ((landed >> st) & 1) ^ 1);
        else
          mbar_wait(&bars.full[st], (i / NST) & 1);
      }
      if (u > 0 && q_armed) mbar_wait(bars.qfull, (u - 1) & 1);
    }
  }
  __syncwarp();
}

template <int HD>
__global__ void __launch_bounds__(kChunkThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                 const __grid_constant__ CUtensorMap tmv, const ChunkParams p) {
  using Lay = ChunkLayout<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const ChunkBars bars = chunk_bars(reinterpret_cast<uint64_t*>(smem + Lay::kBars), Lay::kStages);
  Unit* units = reinterpret_cast<Unit*>(smem + Lay::kUnits);
  int* note_flags = reinterpret_cast<int*>(smem + Lay::kFlags);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + Lay::kFlags + 16);
  uint16_t* notes = reinterpret_cast<uint16_t*>(smem + Lay::kNotes);
  float2* ml = reinterpret_cast<float2*>(smem + Lay::kMl);
  // what needs no input comes before the wait for the previous kernel
  if (warp == kProducer && lane == 0) {
    tma_prefetch_desc(&tmq);
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
    for (int i = 0; i < Lay::kStages; ++i) {
      mbar_init(&bars.full[i], 2);
      mbar_init(&bars.empty[i], 1);
      mbar_init(&bars.landed[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.sfull[i], 1);
      mbar_init(&bars.pfull[i], 4);
      mbar_init(&bars.ofull[i], 1);
      mbar_init(&bars.ufull[i], 1);
      mbar_init(&bars.uempty[i], 8 + 1 + 2);
    }
    mbar_init(bars.qfull, 1);
    mbar_init(bars.qempty, 1);
    mbar_init(bars.drain, 1);
    mbar_init(bars.xfull, 4);
    mbar_init(bars.xdone, 4);
    fence_barrier_init();
  }
  if (warp == kMma) tmem_alloc(tmem_at, 512);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  // in memory that the ring takes over afterwards
  const SequenceTable tab = {reinterpret_cast<long long*>(smem),
                             reinterpret_cast<int4*>(smem + kMaxBatch * sizeof(long long))};
  if (p.batch > 32) fill_sequence_table(p, tab);
  fence_proxy_async_smem();  // the table was written by ordinary stores, the ring is not
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  // The softmax warpgroups hold a row of S in registers: 208 for their threads,
  // 80 for the others (256 * 208 + 128 * 80 of the launch's 384 * 168).
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  }
  if (warp < 8) {
    softmax_role<HD>(p, bars, units, note_flags, notes, ml, tmem, warp >> 2, warp, lane);
  } else if (warp == kProducer) {
    const Share share = find_share(p, tab, lane);
    fence_proxy_async_smem();
    __syncwarp();
    producer_role<HD>(p, bars, share, tmq, tmk, tmv, units, note_flags, smem, lane);
  } else if (warp == kMma) {
    const uint32_t base = smem_u32(smem);
    if (!mma_role<HD>(p, bars, units, tmem, base + Lay::kRing, base, lane)) {
      // abandoned: wait (bounded) for every tensor-core operation issued
      umma_commit_elect(bars.drain);
      if (lane == 0) mbar_wait(bars.drain, 0);
    }
  } else {
    check_role<HD>(p, bars, units, note_flags, notes, smem + Lay::kRing, warp - kChecker, lane);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();  // every access to tensor memory of this CTA is done
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct ChunkPlan {
  int grid, rows;
  size_t off_ml, off_merge, bytes;
};

ChunkPlan make_chunk_plan(int num_tokens, int group, int head_dim) {
  ChunkPlan pl;
  pl.grid = device_sm_count();
  pl.rows = num_tokens > kTile / group ? kRowsMax : kTile;  // one row tile holds every unit
  const size_t rows = (size_t)pl.grid * 2 * pl.rows;
  pl.off_ml = align_up(rows * head_dim * sizeof(float), 256);
  pl.off_merge = align_up(pl.off_ml + rows * 2 * sizeof(float), 256);
  pl.bytes = pl.off_merge + align_up(pl.grid * sizeof(MergeUnit), 256);
  return pl;
}

template <int HD>
cudaError_t launch_chunk(const ChunkPlan& pl, const CUtensorMap& tq, const CUtensorMap& tk,
                         const CUtensorMap& tv, const ChunkParams& p, cudaStream_t stream) {
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        chunk_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkLayout<HD>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev] = true;
  }
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.grid);
  cfg.blockDim = dim3(kChunkThreads);
  cfg.dynamicSmemBytes = ChunkLayout<HD>::kBytes;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_kernel<HD>, tq, tk, tv, p);
  if (e != cudaSuccess) return e;
  const MergeParams m = {reinterpret_cast<uint16_t*>(p.out), p.lse,          p.part_o,  p.part_ml, p.merge,
                         p.out_stride,                       p.num_q_heads, p.group,   p.rows};
  const long long rows = (long long)p.num_tokens * p.group;
  const long long usual = rows <= 32 ? 2 * (rows / p.batch) + 1 : rows;
  return launch_unit_merge<HD, false>(cfg, pl.grid, rows, usual, m);
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" size_t vg_chunk_workspace_bytes(int batch, int num_tokens, int num_q_heads,
                                           int num_kv_heads, int head_dim) {
  if (batch <= 0 || num_tokens <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > 16 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return make_chunk_plan(num_tokens, num_q_heads / num_kv_heads, head_dim).bytes;
}

extern "C" vg_status vg_chunk_attention(const vg_paged_kv* kv, const void* q, int64_t q_stride,
                                        const int32_t* cu_q, const int32_t* kv_lens, int batch,
                                        int num_tokens, int num_q_heads, float softmax_scale,
                                        void* out, int64_t out_stride, float* lse, void* workspace,
                                        size_t workspace_bytes, int32_t* error_flag,
                                        cudaStream_t stream) {
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
  const int g = num_q_heads / kv->num_kv_heads;
  if (g > 16 || batch > kMaxBatch || kv->max_pages_per_seq > (1 << 26) ||
      (int64_t)kv->num_pages * kv->num_kv_heads >= (1 << 29))
    return VG_ERR_UNSUPPORTED;
  const ChunkPlan pl = make_chunk_plan(num_tokens, g, kv->head_dim);
  if (!workspace || workspace_bytes < pl.bytes) return VG_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return VG_ERR_INVALID_ARGUMENT;
  CUtensorMap tq, tk, tv;
  if (!page_chunk_tensor_map(kv->k_pages, kv->num_pages, kv->num_kv_heads, kv->head_dim, &tk) ||
      !page_chunk_tensor_map(kv->v_pages, kv->num_pages, kv->num_kv_heads, kv->head_dim, &tv) ||
      !token_rows_tensor_map(q, num_tokens, num_q_heads, kv->head_dim, q_stride, g, kTile / g, &tq))
    return VG_ERR_LAUNCH;
  ChunkParams p = {};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.page_table = kv->page_table;
  p.cu_q = cu_q;
  p.kv_lens = kv_lens;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + pl.off_ml);
  p.merge = reinterpret_cast<MergeUnit*>(ws + pl.off_merge);
  p.error_flag = error_flag;
  p.out_stride = out_stride;
  p.wait_ns = wait_report_ns();
  p.polls = p.wait_ns < kWaitLimitNs ? 1 : 64;
  p.scale_log2 = softmax_scale * kLog2e;
  p.batch = batch;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = kv->num_kv_heads;
  p.group = g;
  p.num_pages = kv->num_pages;
  p.width = kv->max_pages_per_seq;
  p.rows = pl.rows;
  const cudaError_t e = kv->head_dim == 128 ? launch_chunk<128>(pl, tq, tk, tv, p, stream)
                                             : launch_chunk<64>(pl, tq, tk, tv, p, stream);
  return e == cudaSuccess ? VG_OK : VG_ERR_LAUNCH;
}
