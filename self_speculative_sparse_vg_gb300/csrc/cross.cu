// Cross attention: rows of new tokens to the states of an encoder, whose length
// is its own (sm_103a).
//
// Row t of sequence e computes softmax(scale q_t . k_j) v over the states j of
// [start_e, start_e + len_e) that the mask, if there is one, leaves: no causal
// order.  The beams of one request are rows of one sequence.
//
// Design (one persistent CTA per SM), as in chunk.cu:
//  * A unit is one or two 128-row tiles of one KV head of one sequence, the
//    floor(128 / g) tokens of a tile times their g query heads, so K and V are
//    read once for all heads of the group and all beams of the request.  Its
//    work is the ceil(len / 128) state tiles, the same for all its rows.
//  * All units' tiles form one line (sequence, KV head, rows; weighted by what
//    they cost), cut into equal shares, one per CTA, found from the lengths on
//    the device.  A unit that a cut divides leaves fp32 partials (m, l, O) that
//    a chained kernel merges.
//  * Two softmax warpgroups, one row per thread, each with its own S (128 fp32
//    columns of tensor memory, P written back over it in 16 bits) and O.  A unit
//    of one row tile gives both the same rows and alternate state tiles.
//  * Units of at most 32 rows (single tokens, beams, verify rows) would leave a
//    tile's 128 columns to the one warp that holds their lanes.  Their Q is
//    laid four times into the row tile, so that each warp of a warpgroup finds
//    the rows' scores in its own lanes and takes 32 columns; the warps exchange
//    the rows' maxima and write P to shared memory, whence the product with V
//    reads it.
//  * Where most sequences have one row tile and heads are 64 wide, a unit is a pair
//    of neighbouring KV heads, one for each warpgroup: a state's 128 bytes of one
//    head come from HBM at 4.5 TB/s, 256 bytes of two at 6.5 (16 heads, 6144
//    states of 64 requests).
//  * States lie in rows of a projection, so a tile of K or V of one head is one
//    TMA box of 128 rows (128-byte swizzle) into a ring of stages.
//  * All rows of a unit attend the same states.  Tiles with states that are not
//    attended (masked, or past the end, where another sequence's lie) pass
//    through two warps that zero those rows of V: a weight of zero times a NaN
//    or an infinity would still spoil the row.  Their scores become -inf.
//
// Measured, calls in a row, merge included.  One token to 1500 states, 16 heads of
// 64: 10 us, latency (share, first loads, partials, merge).  Five beams of 24
// requests to 200 - 1500 states of them: 28 us for 105 MB; six verify rows of 8
// requests to up to 6404 masked states, 32/8 heads of 128: 30 us for 121 MB, both
// HBM between a start of 4 us and a merge of 4 (64 requests of 6144 states stream at
// 6.5 - 6.8 TB/s).  4777 tokens of five prompts to 129 - 6404 states, 32/8 heads of
// 128: 272 us, 1250 TFLOP/s (262 in a graph); the tensor pipe is active 62 % of the
// time, since S, P and O fill tensor memory and a warpgroup's softmax and products
// alternate.
#include <limits.h>
#include <math.h>

#include "units.cuh"
#include "vg_host.h"

namespace vg {
namespace {

constexpr int kTile = kUnitTile;       // states of a K or V tile, rows of a row tile
constexpr int kCrossThreads = 384;
constexpr int kProducer = 8, kMma = 9, kChecker = 10;  // warps (0..7: softmax; two checkers)
constexpr int kMaxBatch = 4096;
constexpr int kRowsMax = 2 * kTile;    // rows of a unit
// Costs on the line that the CTAs share: a state tile of a unit with two row
// tiles or with one, and what a unit costs beside its tiles.
constexpr int kTwoCost = 5, kOneCost = 4, kUnitCost = 15;

// The reference m of a row's weights 2^(score - m), in powers of two: it is set kBelow
// below the row's maximum, and again when that outgrows it by kLimit.  fp16 weights
// reach 2^15 so (of 2^16), and what a weight loses below fp16's normal range is at
// most 2^-32 of the row's largest: with the reference at the maximum it was 2^-25, and
// thousands of states of 2^-26 each were lost whole while the row's sum kept them.
// bf16 has float32's exponents.
template <bool F16>
struct Reference {
  static constexpr float kBelow = F16 ? 7.f : 0.f, kLimit = F16 ? 15.f : 8.f;
};

struct CrossParams {
  const int32_t* cu_q;
  const int32_t* starts;
  const int32_t* lens;
  const uint8_t* mask;
  uint16_t* out;
  float* lse;
  float* part_o;      // [grid][2][HD / 4][rows][4]
  float* part_ml;     // [grid][2][rows][2]
  MergeUnit* merge;   // [grid]
  int32_t* error_flag;
  int64_t out_stride;
  uint64_t wait_ns;    // a longer wait is reported
  int polls;           // polls of a wait between two looks at the timer
  float scale_log2;
  int batch, num_tokens, num_states, num_q_heads, num_kv_heads, group, rows;
  int heads;          // of the line: KV heads, or pairs of them
  int tile_tokens, few_tokens, unit_tokens;  // tokens of a row tile, of 32 rows, and of a unit
  uint32_t by_unit_tokens;       // ceil(2^32 / unit_tokens), 0 for 1
};

// A unit of work as the CTA's roles see it.
struct Unit {
  int tok0, ntok;     // first token row, tokens (at most 2 * tile_tokens)
  int start, len;     // states of the sequence
  int h;
  int kt0, kt1;       // state tiles of this CTA; kt0 == kt1: no more units
  int two;            // two row tiles (else one, state tiles alternate)
  int narrow;         // at most 32 rows, four times in the row tile
  int part;           // partial slot of the workspace, -1: writes its rows
};

template <int HD, bool PAIR>
struct CrossLayout {
  static constexpr int kBlocks = PAIR ? 2 : HD / 64;   // 64-dim blocks of a row (of a pair: its heads)
  // Q, K and V tiles: [block][row][128 bytes], as one TMA box brings them
  static constexpr int kBlockBytes = kTile * 128;
  static constexpr int kStageBytes = kBlocks * kBlockBytes;
  static constexpr int kStages = kBlocks == 2 ? 5 : 10;
  // P of units of few rows, [warpgroup][64-column block][32 rows][128 bytes], and the
  // warps' exchange: in the place of the second row tile of Q, if that has room
  static constexpr int kPBlockBytes = 32 * 128;
  static constexpr int kPBytes = 2 * kPBlockBytes;
  static constexpr int kP = kBlocks == 2 ? kStageBytes : 2 * kStageBytes;
  static constexpr int kExchange = kP + 2 * kPBytes;
  // behind two row tiles of Q.  (The product reads 128 rows of P, of which 32 are
  // there: what follows is the other P and the ring, and goes to unused lanes.)
  static constexpr int kRing = kBlocks == 2 ? 2 * kStageBytes : kExchange + 2048;
  static constexpr int kBars = kRing + kStages * kStageBytes;
  static constexpr int kBarCount = 3 * kStages + 17;
  static constexpr int kUnits = kBars + (kBarCount + 1) / 2 * 16;
  static constexpr int kTmemAt = kUnits + 2 * 48;
  static constexpr int kMl = kTmemAt + 16;
  static constexpr int kBytes = kMl + kTile * 8;
  static constexpr int kSCol = 0, kOCol = 2 * kTile;

  // Byte offset of 16-byte piece `ch` of state `row` in a K or V tile.
  static __device__ __forceinline__ uint32_t kv_offset(int row, int ch) {
    return (ch >> 3) * kBlockBytes + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
  }
};
static_assert(CrossLayout<128, false>::kBytes <= 227 * 1024 && CrossLayout<64, false>::kBytes <= 227 * 1024 &&
                  CrossLayout<64, true>::kBytes <= 227 * 1024,
              "");
static_assert(sizeof(Unit) <= 48, "");

struct CrossBars {
  // Ring stages.  `landed`: a V tile with states that are not attended has
  // landed; `full`: a tile may be read (it has landed, or was gone through);
  // `empty`: its products are done.
  uint64_t *full, *landed, *empty;         // [stages]
  uint64_t *sfull, *pfull, *ofull;         // [2]: S, P, all of O of a warpgroup
  uint64_t *xmax;                          // [2]: the warps' maxima of a unit of few rows
  uint64_t *qfull, *qempty, *ufull, *uempty, *xfull, *xdone, *drain;
};

__device__ __forceinline__ CrossBars cross_bars(uint64_t* b, int stages) {
  CrossBars r;
  r.full = b;
  r.landed = b + stages;
  r.empty = b + 2 * stages;
  b += 3 * stages;
  r.sfull = b;
  r.pfull = b + 2;
  r.ofull = b + 4;
  r.ufull = b + 6;
  r.uempty = b + 8;
  r.xmax = b + 10;
  r.qfull = b + 12;
  r.qempty = b + 13;
  r.xfull = b + 14;
  r.xdone = b + 15;
  r.drain = b + 16;
  return r;
}

// State tiles of a unit, at least one (rows without states are still written).
__device__ __forceinline__ int state_tiles(int len) { return len > 0 ? (len - 1) / kTile + 1 : 1; }

// Rows and states of sequence e; n = 0 when it has no rows or makes no sense.
struct Sequence {
  int q0, n, start, len;
};
__device__ __forceinline__ bool sequence_of(const CrossParams& p, int e, Sequence& s) {
  s.q0 = p.cu_q[e];
  const int q1 = p.cu_q[e + 1];
  s.start = p.starts[e];
  s.len = p.lens[e];
  const bool ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= p.num_tokens && s.start >= 0 && s.len >= 0 &&
                  s.len <= p.num_states - s.start;
  s.n = ok ? q1 - s.q0 : 0;
  return ok;
}

__device__ __forceinline__ int tile_cost(const CrossParams& p, int ntok) {
  return ntok > p.tile_tokens ? kTwoCost : kOneCost;
}

// Length on the line of a unit of ntok tokens: its overhead, then its tiles.
__device__ __forceinline__ long long unit_length(const CrossParams& p, int ntok, int len) {
  return kUnitCost + (long long)tile_cost(p, ntok) * state_tiles(len);
}

// A unit's state tiles that end before offset y of its length; a CTA whose
// share holds [y0, y1) of it takes tiles [tiles_before(y0), tiles_before(y1)).
__device__ __forceinline__ int tiles_before(long long y, int cost) {
  if (y <= kUnitCost) return 0;
  const long long z = y - kUnitCost;
  if (z >> 32) return (int)(z / cost);
  return cost == kTwoCost ? (int)((uint32_t)z / kTwoCost) : (int)((uint32_t)z / kOneCost);
}

// Whether tile kt may hold states that are not attended.
__device__ __forceinline__ bool checked_tile(const CrossParams& p, int len, int kt) {
  return p.mask != nullptr || (kt + 1) * kTile > len;
}

// The mask bytes of tile kt that this lane looks at, state 32 w + lane in
// byte w (1: attended), and the tile's words from those of all lanes.
__device__ __forceinline__ uint32_t mask_bytes(const CrossParams& p, int start, int len, int kt, int lane) {
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int j = kt * kTile + 32 * w + lane;
    bool in = j < len;
    if (in && p.mask) in = p.mask[(int64_t)start + j] != 0;
    m |= (uint32_t)in << (8 * w);
  }
  return m;
}
__device__ __forceinline__ uint32_t mask_word(uint32_t bytes, int w) {
  return __ballot_sync(0xffffffffu, (bytes >> (8 * w)) & 1u);
}

// ---------------------------------------------------------------- softmax
// One warp of a warpgroup through all units of the CTA.
template <int HD, bool F16, bool PAIR>
__device__ __forceinline__ void softmax_role(const CrossParams& p, const CrossBars& bars, const Unit* units,
                                             float2* ml_s, uint8_t* smem, uint32_t tmem, int wg, int warp, int lane) {
  using Lay = CrossLayout<HD, PAIR>;
  const int g = p.group, tt = p.tile_tokens;
  const int r = (warp & 3) * 32 + lane;  // row within the tile
  const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  const uint32_t scol = trow + Lay::kSCol + wg * kTile;
  const uint32_t ocol = trow + Lay::kOCol + wg * HD;
  const int tok_r = r / g, head_r = r - tok_r * g;
  uint32_t sc = 0, oc = 0, xc = 0, mc = 0;
  const int quarter = warp & 3;  // of a tile's columns, for few rows
  float* maxima = reinterpret_cast<float*>(smem + Lay::kExchange) + wg * 256 + lane;  // [2][4][32]
  uint8_t* p_row = smem + Lay::kP + wg * Lay::kPBytes + (quarter >> 1) * Lay::kPBlockBytes + lane * 128;
  for (uint32_t u = 0;; ++u) {
    const int slot = u & 1;
    if (!wait_phase_warp(&bars.ufull[slot], (u >> 1) & 1, p)) return;
    const Unit un = units[slot];
    if (un.kt0 == un.kt1) return;
    const int tok = un.two && !PAIR ? wg * tt + tok_r : tok_r;  // token within the unit
    const bool valid = tok_r < tt && tok < un.ntok;
    const bool rows = __any_sync(0xffffffffu, valid);       // a warp without rows only keeps step
    const int first = un.two ? un.kt0 : un.kt0 + wg;
    const int step = un.two ? 1 : 2;
    const int end = un.kt1;
    float m_used = -INFINITY, lsum = 0.f;
    // the four warps' values of this lane's row, joined
    auto exchange = [&](float v, auto join, float& all) {
      float* at = maxima + (mc & 1) * 128;
      at[quarter * 32] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.xmax[wg]);
      if (!wait_phase_warp(&bars.xmax[wg], mc & 1, p)) return false;
      ++mc;
      all = join(join(at[0], at[32]), join(at[64], at[96]));
      return true;
    };
    for (int kt = first; un.narrow && kt < end; kt += step) {
      const bool partly = checked_tile(p, un.len, kt);
      const uint32_t attended = partly ? mask_bytes(p, un.start, un.len, kt, lane) : 0x01010101u;
      if (!wait_phase_warp(&bars.sfull[wg], sc & 1, p)) return;
      ++sc;
      tc_fence_after();
      float s[32];
      tmem_ld32(scol + quarter * 32, s);
      if (partly) {
        const uint32_t keep = mask_word(attended, quarter);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (!((keep >> j) & 1u)) s[j] = -INFINITY;
      }
      float mx[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) mx[j] = fmaxf(s[j], s[j + 4]);
#pragma unroll
      for (int j = 8; j < 32; j += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], s[j + k], s[j + k + 4]);
      float m_tile;
      if (!exchange(fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * p.scale_log2,
                    [](float a, float b) { return fmaxf(a, b); }, m_tile))
        return;
      const bool need = m_tile > m_used + Reference<F16>::kLimit;
      if (__any_sync(0xffffffffu, need)) {
        const float mn = need ? m_tile - Reference<F16>::kBelow : m_used;
        if (kt != first) {  // P(t - 1) V is done: S(t) was issued after it
          const float corr = mn == -INFINITY ? 1.f : ex2(m_used - mn);
          lsum *= corr;
          if (quarter == 0) {  // O is in the first warp's lanes
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
        }
        m_used = mn;
      }
      const float nref = -safe_ref(m_used);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float a = ex2(fmaf(s[8 * i + 2 * j], p.scale_log2, nref));
          const float b = ex2(fmaf(s[8 * i + 2 * j + 1], p.scale_log2, nref));
          w[j] = pack2<F16>(a, b);
          sum += a + b;
        }
        const int ch = (4 * quarter + i) & 7;
        *reinterpret_cast<uint4*>(p_row + ((ch ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.pfull[wg]);
      lsum += sum;
    }
    if (un.narrow && end > first &&
        !exchange(lsum, [](float a, float b) { return a + b; }, lsum))
      return;
    for (int kt = un.narrow ? end : first; kt < end; kt += step) {
      // read before the wait, so that the mask is there with the scores
      const bool partly = checked_tile(p, un.len, kt);
      const uint32_t attended = rows && partly ? mask_bytes(p, un.start, un.len, kt, lane) : 0x01010101u;
      if (!wait_phase_warp(&bars.sfull[wg], sc & 1, p)) return;
      ++sc;
      tc_fence_after();
      if (rows) {
        uint32_t s[2][64];
        tmem_ld64(scol, s[0]);
        tmem_ld64(scol + 64, s[1]);
        if (partly) {
#pragma unroll
          for (int w = 0; w < kTile / 32; ++w) {
            const uint32_t keep = mask_word(attended, w);
            if (keep == 0xffffffffu) continue;
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
        const bool need = m_tile > m_used + Reference<F16>::kLimit;
        if (__any_sync(0xffffffffu, need)) {
          const float mn = need ? m_tile - Reference<F16>::kBelow : m_used;
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
        // P = 2^(s scale - m), at most 2^8 (fp16: 2^15), rounded to 16 bits for the tensor
        // cores (half a step of each weight, fp16: or 2^-25); the row sum takes it unrounded
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
            pk[j] = pack2<F16>(x.x, x.y);
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
      const bool direct = un.part < 0;
      const int t = un.tok0 + tok, qh = (PAIR ? 2 * un.h + wg : un.h) * g + head_r;
      // row of the partial
      const int half = tt / 2;  // (of a pair: as many tokens have 128 rows of both heads)
      const int prow = PAIR ? tok_r / half * kTile + (tok_r % half * 2 + wg) * g + head_r : (un.two ? wg * kTile : 0) + r;
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
          uint16_t* dst = p.out + t * p.out_stride + (int64_t)qh * HD + c;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = pack2<F16>(__uint_as_float(o[16 * j + 2 * i]), __uint_as_float(o[16 * j + 2 * i + 1]));
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
template <int HD, bool F16, bool PAIR>
struct MmaIssuer {
  using Lay = CrossLayout<HD, PAIR>;
  const CrossBars& bars;
  uint32_t tmem, ring_lo, q_lo, v_lo, p_lo;  // low descriptor words of stage 0, Q and P
  static constexpr uint32_t kTypes = F16 ? (1u << 7) | (1u << 10) : 0u;  // fp16 operands: the bf16 bits off
  static constexpr uint32_t kIdQk = umma_idesc_bf16(kTile, kTile, 0, 0) ^ kTypes;
  static constexpr uint32_t kIdPv = umma_idesc_bf16(kTile, HD, 0, 1) ^ kTypes;
  static constexpr uint32_t kHi = umma_desc_hi(1024);

  // S of warpgroup `wg` = Q (row tile qt) K^T of the stage
  __device__ __forceinline__ void qk(int wg, int qt, uint32_t stage) {
    const uint32_t k = ring_lo + stage * (Lay::kStageBytes >> 4);
    const uint32_t q = q_lo + (PAIR ? 0 : qt) * (Lay::kStageBytes >> 4);
#pragma unroll
    for (int ks = 0; ks < HD / 16; ++ks) {
      const uint32_t at = ((PAIR ? wg : ks >> 2) * Lay::kBlockBytes + (ks & 3) * 32) >> 4;
      umma_bf16_elect(tmem + Lay::kSCol + wg * kTile, q + at, kHi, k + at, kHi, kIdQk, ks > 0);
    }
    umma_commit_elect(&bars.sfull[wg]);
  }
  // O of warpgroup `wg` (+)= P V of the stage
  __device__ __forceinline__ void pv(int wg, uint32_t stage, bool accumulate) {
    const uint32_t v = v_lo + (stage * Lay::kStageBytes + (PAIR ? wg * Lay::kBlockBytes : 0) >> 4);
#pragma unroll
    for (int ks = 0; ks < kTile / 16; ++ks)
      umma_bf16_ts_elect(tmem + Lay::kOCol + wg * HD, tmem + Lay::kSCol + wg * kTile + ks * 8,
                         v + ks * (16 * 128 >> 4), kHi, kIdPv, accumulate || ks > 0);
  }
  // the same with P in shared memory
  __device__ __forceinline__ void pv_few(int wg, uint32_t stage, bool accumulate) {
    const uint32_t v = v_lo + (stage * Lay::kStageBytes + (PAIR ? wg * Lay::kBlockBytes : 0) >> 4);
    const uint32_t a = p_lo + wg * (Lay::kPBytes >> 4);
#pragma unroll
    for (int ks = 0; ks < kTile / 16; ++ks)
      umma_bf16_elect(tmem + Lay::kOCol + wg * HD, a + (((ks >> 2) * Lay::kPBlockBytes + (ks & 3) * 32) >> 4), kHi,
                      v + ks * (16 * 128 >> 4), kHi, kIdPv, accumulate || ks > 0);
  }
};

template <int HD, bool F16, bool PAIR>
__device__ __forceinline__ bool mma_role(const CrossParams& p, const CrossBars& bars, const Unit* units,
                                         uint32_t tmem, uint32_t ring, uint32_t q, int lane) {
  using Lay = CrossLayout<HD, PAIR>;
  constexpr uint32_t NST = Lay::kStages;
  MmaIssuer<HD, F16, PAIR> mma{bars, tmem, umma_desc_lo(ring, 16), umma_desc_lo(q, 16),
                         umma_desc_lo(ring, Lay::kBlockBytes), umma_desc_lo(q + Lay::kP, 16)};
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
  auto pv_product = [&](int wg, uint32_t st, bool accumulate, bool few = false) {
    const uint32_t par = (pc >> wg) & 1;
    pc ^= 1u << wg;
    if (!wait_phase_warp(&bars.pfull[wg], par, p)) return false;
    tc_fence_after();
    if (few)
      mma.pv_few(wg, st, accumulate);
    else
      mma.pv(wg, st, accumulate);
    return true;
  };
  for (uint32_t u = 0;; ++u) {
    const int slot = u & 1;
    if (!wait_phase_warp(&bars.ufull[slot], (u >> 1) & 1, p)) return false;
    const int kt0 = same(units[slot].kt0), kt1 = same(units[slot].kt1), two = same(units[slot].two);
    const bool few = same(units[slot].narrow) != 0;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.uempty[slot]);
    if (kt0 == kt1) return true;
    if (!wait_phase_warp(bars.qfull, u & 1, p)) return false;
    const int n = kt1 - kt0;
    if (two) {
      if (!wait(&bars.full[sk], pk)) return false;
      tc_fence_after();
      mma.qk(0, 0, sk);
      mma.qk(1, 1, sk);
      umma_commit_elect(&bars.empty[sk]);
      if (n == 1) umma_commit_elect(bars.qempty);
      next(sk, pk);
      for (int j = 0; j < n; ++j) {
        const bool more = j + 1 < n;
        // the tiles are waited for first, while the warpgroups are at P(j)
        if (!wait(&bars.full[sv], pv) || (more && !wait(&bars.full[sk], pk))) return false;
        // (one copy of this code for both warpgroups: the roles share the
        // instruction cache)
#pragma unroll 1
        for (int wg = 0; wg < 2; ++wg) {
          if (!pv_product(wg, sv, j > 0, few)) return false;
          if (more)
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
        if (!wait(&bars.full[sv], pv) || !pv_product(wg, sv, j > 1, few)) return false;
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

// ------------------------------------------------- V rows that nobody attends
// Warp `half` of two owns half of the dimensions of every such V tile.
template <int HD, bool PAIR>
__device__ __forceinline__ void check_role(const CrossParams& p, const CrossBars& bars, const Unit* units,
                                           uint8_t* ring, int half, int lane) {
  using Lay = CrossLayout<HD, PAIR>;
  constexpr int NST = Lay::kStages;
  constexpr int CPW = Lay::kBlocks * 4;  // 16-byte pieces of a row per warp
  constexpr int RPI = 32 / CPW;          // rows per pass
  uint32_t tiles = 0, landed = 0;
  const int ch = half * CPW + lane % CPW, r = lane / CPW;  // piece of the row, row of the pass
  for (uint32_t u = 0;; ++u) {
    const int slot = u & 1;
    if (!wait_phase_warp(&bars.ufull[slot], (u >> 1) & 1, p)) return;
    const Unit un = units[slot];
    if (un.kt0 == un.kt1) return;
    // without a mask only the last tile of a sequence
    for (int kt = p.mask ? un.kt0 : max(un.kt0, un.len / kTile); kt < un.kt1; ++kt) {
      if (!checked_tile(p, un.len, kt)) continue;
      const uint32_t st = (2 * (tiles + kt - un.kt0) + 1) % NST;
      const uint32_t attended = mask_bytes(p, un.start, un.len, kt, lane);
      if (!wait_phase_warp(&bars.landed[st], (landed >> st) & 1, p)) return;
      landed ^= 1u << st;
      uint8_t* tile = ring + st * Lay::kStageBytes;
#pragma unroll
      for (int w = 0; w < kTile / 32; ++w) {
        const uint32_t keep = mask_word(attended, w);
        if (keep == 0xffffffffu) continue;
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += RPI)
          if (!((keep >> (r0 + r)) & 1u))
            *reinterpret_cast<uint4*>(tile + Lay::kv_offset(32 * w + r0 + r, ch)) = make_uint4(0u, 0u, 0u, 0u);
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
  int e, h, rt, kt0;
  Sequence seq;       // the first unit's
};

// Units of n tokens (a product's upper half for the quotient, put right by one).
__device__ __forceinline__ int row_units(const CrossParams& p, int n) {
  const uint32_t a = (uint32_t)n + (uint32_t)p.unit_tokens - 1u;
  if (p.by_unit_tokens == 0) return (int)a;
  uint32_t q = __umulhi(a, p.by_unit_tokens);
  if (q * (uint32_t)p.unit_tokens > a) --q;
  return (int)q;
}

// Length on the line of one head of a sequence: full units, then the last.
__device__ __forceinline__ long long head_length(const CrossParams& p, const Sequence& s) {
  const int units = row_units(p, s.n);
  if (units == 0) return 0;
  return (units - 1) * unit_length(p, p.unit_tokens, s.len) +
         unit_length(p, s.n - (units - 1) * p.unit_tokens, s.len);
}

// The sequence of this lane among the 32 from e0 on, and its length on the line.
__device__ __forceinline__ long long sequence_length(const CrossParams& p, int e, Sequence& s) {
  s = {};
  if (e < p.batch && !sequence_of(p, e, s) && blockIdx.x == 0) flag_error(p.error_flag, VG_DEVERR_LENGTH);
  return head_length(p, s) * p.heads;
}

// Batches of more than 32 sequences: the CTA's warps put every sequence's
// length into shared memory first.
struct SequenceTable {
  long long* length;
  Sequence* seq;
};

__device__ __forceinline__ void fill_sequence_table(const CrossParams& p, const SequenceTable& tab) {
  for (int e = threadIdx.x; e < p.batch; e += kCrossThreads) {
    Sequence s;
    tab.length[e] = sequence_length(p, e, s);
    tab.seq[e] = s;
  }
}

// Where the CTA's share of a line of `total` begins, in the numbers that it needs (one
// division of 64 bits is a call of its own on the way to the first load).  sum: the
// line up to and with this lane's sequence, where they are at most 32.
template <typename N>
__device__ __forceinline__ Share locate_share(const CrossParams& p, const SequenceTable& tab, const Sequence& seq,
                                              long long sum, long long total, int lane) {
  // at least one tile, so that every CTA inside a divided unit has a part of it
  const N share = max((N)((N)(total + gridDim.x - 1) / (N)gridDim.x), (N)(p.rows == kTile ? kOneCost : kTwoCost));
  const long long x0 = (long long)share * blockIdx.x;
  Share s = {};
  s.share = share;
  s.x1 = min(total, x0 + (long long)share);
  s.e = -1;
  if (x0 >= total) return s;
  long long base = 0;  // where the sequence's part of the line begins
  if (p.batch <= 32) {
    s.e = __ffs(__ballot_sync(0xffffffffu, sum > x0)) - 1;
    base = __shfl_sync(0xffffffffu, sum, max(s.e - 1, 0));
    if (s.e == 0) base = 0;
    s.seq.q0 = __shfl_sync(0xffffffffu, seq.q0, s.e);
    s.seq.n = __shfl_sync(0xffffffffu, seq.n, s.e);
    s.seq.start = __shfl_sync(0xffffffffu, seq.start, s.e);
    s.seq.len = __shfl_sync(0xffffffffu, seq.len, s.e);
  } else {
    for (int e0 = 0; e0 < p.batch && s.e < 0; e0 += 32) {
      const uint32_t past = __ballot_sync(0xffffffffu, e0 + lane < p.batch && tab.length[e0 + lane] > x0);
      if (past) s.e = e0 + __ffs(past) - 1;
    }
    base = s.e > 0 ? tab.length[s.e - 1] : 0;
    s.seq = tab.seq[s.e];
  }
  const N per_head = (N)head_length(p, s.seq), full = (N)unit_length(p, p.unit_tokens, s.seq.len);
  const N in_seq = (N)(x0 - base);
  s.h = in_seq < per_head ? 0 : (int)(in_seq / per_head);
  const N y = in_seq - (N)s.h * per_head;
  s.rt = y < full ? 0 : min((int)(y / full), row_units(p, s.seq.n) - 1);
  const N in = y - (N)s.rt * full;
  s.kt0 = tiles_before((long long)in, tile_cost(p, min(p.unit_tokens, s.seq.n - s.rt * p.unit_tokens)));
  s.unit_at = x0 - (long long)in;
  return s;
}

// Where the CTA's share of the line begins; found by one warp.  e < 0: no work.
__device__ __forceinline__ Share find_share(const CrossParams& p, const SequenceTable& tab, int lane) {
  const bool small = p.batch <= 32;
  Sequence seq = {};
  long long sum = 0, total = 0;  // running sum over the line, this lane's sequence included
  if (small) {
    sum = warp_inclusive_sum(sequence_length(p, lane, seq), lane);
    total = __shfl_sync(0xffffffffu, sum, 31);
  } else {
    for (int e0 = 0; e0 < p.batch; e0 += 32) {
      const bool in = e0 + lane < p.batch;
      sum = total + warp_inclusive_sum(in ? tab.length[e0 + lane] : 0, lane);
      if (in) tab.length[e0 + lane] = sum;
      total = __shfl_sync(0xffffffffu, sum, 31);
    }
    __syncwarp();
  }
  if (total >> 31 == 0) return locate_share<uint32_t>(p, tab, seq, sum, total, lane);
  return locate_share<long long>(p, tab, seq, sum, total, lane);
}

// ----------------------------------------------------------------- producer
// Walks the CTA's units, publishes them and streams their Q, K and V; one lane.
// K and V do not wait for room for Q: it is looked for before each of them and
// while they wait for a stage.  On a wait that was given up the lane stops, then
// waits (bounded) for its own copies.
template <int HD, bool PAIR>
struct Producer {
  using Lay = CrossLayout<HD, PAIR>;
  const CrossParams& p;
  const CrossBars& bars;
  const CUtensorMap &tmq, &tmf, &tmk, &tmv;
  uint8_t* smem;
  Unit q_unit = {};       // whose Q is to come, if
  bool q_wanted = false;
  bool q_all = false;     // once the unit before is done with, P too (else with its Q)
  uint32_t q_sent = 0;    // units whose Q was sent

  __device__ __forceinline__ bool q_has_room() const {
    if (q_sent == 0) return true;
    const uint32_t before = q_sent - 1;
    return q_all ? mbar_test_wait(&bars.uempty[before & 1], (before >> 1) & 1) : mbar_test_wait(bars.qempty, before & 1);
  }
  __device__ __forceinline__ void send_q() {
    const int g = p.group, tt = p.tile_tokens;
    const bool narrow = q_unit.narrow;
    const int copies = narrow ? 4 : q_unit.two && !PAIR ? 2 : 1, tokens = narrow ? p.few_tokens : tt;
    mbar_arrive_expect_tx(bars.qfull, copies * Lay::kBlocks * tokens * g * 128);
    for (int t = 0; t < copies; ++t)
      for (int x = 0; x < Lay::kBlocks; ++x) {
        uint8_t* dst = smem + x * Lay::kBlockBytes + t * (narrow ? 32 * 128 : Lay::kStageBytes);
        tma_load_3d(dst, narrow ? &tmf : &tmq, bars.qfull, PAIR ? 0 : x * 64,
                    (PAIR ? 2 * q_unit.h + x : q_unit.h) * g, q_unit.tok0 + (narrow ? 0 : t * tt));
      }
    q_wanted = false;
    ++q_sent;
  }
  // Waits for the phase of `bar` (a stage, or null), or for Q's room if that is
  // wanted and `q_too`; sends Q when there is room.  Bounded as wait_phase.
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, bool q_too) {
    uint64_t t0 = 0;
    while (true) {
#pragma unroll 1
      for (int i = 0; i < p.polls; ++i) {
        if (q_wanted && q_has_room()) send_q();
        const bool there = bar == nullptr || (q_wanted || p.polls == 1 ? mbar_test_wait(bar, parity)
                                                                       : mbar_try_wait(bar, parity));
        if (there && !(q_too && q_wanted)) return true;
      }
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > p.wait_ns) flag_error(p.error_flag, VG_DEVERR_TIMEOUT);
      if (now - t0 > kWaitLimitNs) return false;
    }
  }

  __device__ __forceinline__ void run(const Share& s, Unit* units) {
    constexpr int NST = Lay::kStages;
    const int tt = p.tile_tokens, tu = p.unit_tokens;
    uint8_t* ring = smem + Lay::kRing;
    int e = s.e, h = s.h, rt = s.rt, kt0 = s.kt0;
    long long at = s.unit_at;  // line position of the current unit's first tile
    Sequence seq = s.seq;
    uint32_t ri = 0, u = 0, on_landed = 0, landed = 0;  // bits: last load of a stage, its parity
    bool live = true, last_narrow = false;
    const uint64_t once = l2_policy_evict_first();
    MergeUnit cut = {};
    while (true) {
      const int ntok = min(tu, seq.n - rt * tu), cost = tile_cost(p, ntok);
      // its next state tile ends in the share
      const bool more = e >= 0 && at + kUnitCost + (long long)cost * (kt0 + 1) <= s.x1;
      const int slot = u & 1;
      if (u >= 2 && !wait(&bars.uempty[slot], ((u >> 1) - 1) & 1, false)) {
        live = false;
        break;
      }
      Unit un = {};
      if (more) {
        un.tok0 = seq.q0 + rt * tu;
        un.ntok = ntok;
        un.start = seq.start;
        un.len = seq.len;
        un.h = h;
        un.two = PAIR || un.ntok > tt;
        un.narrow = un.ntok <= p.few_tokens;
        const int tiles = state_tiles(seq.len);
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
      units[slot] = un;
      mbar_arrive(&bars.ufull[slot]);
      if (!more) break;
      q_wanted = true;
      q_unit = un;
      q_all = !PAIR && un.two && last_narrow && Lay::kP < 2 * Lay::kStageBytes;
      last_narrow = un.narrow;
      for (int kt = un.kt0; kt < un.kt1 && live; ++kt) {
#pragma unroll 1
        for (int v = 0; v < 2; ++v) {
          const uint32_t st = ri % NST;
          if (!wait(ri >= NST ? &bars.empty[st] : nullptr, ((ri / NST) - 1) & 1, false)) {
            live = false;
            break;
          }
          uint64_t* bar = &(v && checked_tile(p, un.len, kt) ? bars.landed : bars.full)[st];
          if (bar == &bars.full[st]) mbar_arrive(bar);  // for the second checker
          mbar_arrive_expect_tx(bar, Lay::kStageBytes);
          // (states that no other unit reads leave L2 first: verify rows 31.0 us, 32.1
          // without; prompts, whose units share them, 273 with and 262 without)
          if (seq.n <= tu)
            tma_load_4d(ring + st * Lay::kStageBytes, v ? &tmv : &tmk, bar, 0, un.start + kt * kTile, 0, h, once);
          else
            tma_load_4d(ring + st * Lay::kStageBytes, v ? &tmv : &tmk, bar, 0, un.start + kt * kTile, 0, h);
          on_landed &= ~(1u << st);
          if (bar == &bars.landed[st]) {
            on_landed |= 1u << st;
            landed ^= 1u << st;
          }
          ++ri;
        }
      }
      if (live && !wait(nullptr, 0, true)) live = false;
      if (!live) break;
      ++u;
      kt0 = 0;
      if (++rt * tu >= seq.n) {
        rt = 0;
        if (++h == p.heads) {
          h = 0;
          do {
            if (++e >= p.batch) break;
            sequence_of(p, e, seq);
          } while (seq.n == 0);
        }
      }
    }
    p.merge[blockIdx.x] = cut;
    if (!live) {
      for (uint32_t i = ri > NST ? ri - NST : 0; i < ri; ++i) {
        const uint32_t st = i % NST;
        if ((on_landed >> st) & 1)
          mbar_wait(&bars.landed[st], ((landed >> st) & 1) ^ 1);
        else
          mbar_wait(&bars.full[st], (i / NST) & 1);
      }
      if (q_sent > 0) mbar_wait(bars.qfull, (q_sent - 1) & 1);
    }
  }
};

template <int HD, bool F16, bool PAIR>
__global__ void __launch_bounds__(kCrossThreads, 1)
    cross_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmf,
                 const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                 const CrossParams p) {
  using Lay = CrossLayout<HD, PAIR>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const CrossBars bars = cross_bars(reinterpret_cast<uint64_t*>(smem + Lay::kBars), Lay::kStages);
  Unit* units = reinterpret_cast<Unit*>(smem + Lay::kUnits);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + Lay::kTmemAt);
  float2* ml = reinterpret_cast<float2*>(smem + Lay::kMl);
  // what needs no input comes before the wait for the previous kernel
  if (warp == kProducer && lane == 0) {
    tma_prefetch_desc(&tmq);
    tma_prefetch_desc(&tmf);
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
      mbar_init(&bars.xmax[i], 4);
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
                             reinterpret_cast<Sequence*>(smem + kMaxBatch * sizeof(long long))};
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
    softmax_role<HD, F16, PAIR>(p, bars, units, ml, smem, tmem, warp >> 2, warp, lane);
  } else if (warp == kProducer) {
    const Share share = find_share(p, tab, lane);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      Producer<HD, PAIR> producer{p, bars, tmq, tmf, tmk, tmv, smem};
      producer.run(share, units);
    }
  } else if (warp == kMma) {
    const uint32_t base = smem_u32(smem);
    if (!mma_role<HD, F16, PAIR>(p, bars, units, tmem, base + Lay::kRing, base, lane)) {
      // abandoned: wait (bounded) for every tensor-core operation issued
      umma_commit_elect(bars.drain);
      if (lane == 0) mbar_wait(bars.drain, 0);
    }
  } else {
    check_role<HD, PAIR>(p, bars, units, smem + Lay::kRing, warp - kChecker, lane);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();  // every access to tensor memory of this CTA is done
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct CrossPlan {
  int grid, rows;
  size_t off_ml, off_merge, bytes;
};

// Whether heads may be taken in pairs: then a token has 2 group rows, of which the
// merge finds kTile / (2 group) tokens' in a tile.
bool may_pair(int group, int num_kv_heads, int head_dim) {
  return head_dim == 64 && num_kv_heads % 2 == 0 && 2 * group <= kTile;
}

CrossPlan make_cross_plan(int num_tokens, int group, int num_kv_heads, int head_dim) {
  CrossPlan pl;
  pl.grid = device_sm_count();
  // one row tile holds every unit
  const bool one = num_tokens <= kTile / (may_pair(group, num_kv_heads, head_dim) ? 2 * group : group);
  pl.rows = one ? kTile : kRowsMax;
  const size_t rows = (size_t)pl.grid * 2 * pl.rows;
  pl.off_ml = align_up(rows * head_dim * sizeof(float), 256);
  pl.off_merge = align_up(pl.off_ml + rows * 2 * sizeof(float), 256);
  pl.bytes = pl.off_merge + align_up(pl.grid * sizeof(MergeUnit), 256);
  return pl;
}

template <int HD, bool F16, bool PAIR>
cudaError_t launch_cross(const CrossPlan& pl, const CUtensorMap& tq, const CUtensorMap& tf, const CUtensorMap& tk,
                         const CUtensorMap& tv, const CrossParams& p, cudaStream_t stream) {
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        cross_kernel<HD, F16, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, CrossLayout<HD, PAIR>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev] = true;
  }
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.grid);
  cfg.blockDim = dim3(kCrossThreads);
  cfg.dynamicSmemBytes = CrossLayout<HD, PAIR>::kBytes;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, cross_kernel<HD, F16, PAIR>, tq, tf, tk, tv, p);
  if (e != cudaSuccess) return e;
  const int group = PAIR ? 2 * p.group : p.group;  // (as the rows of a partial lie)
  const MergeParams m = {p.out,        p.lse,         p.part_o, p.part_ml, p.merge,
                         p.out_stride, p.num_q_heads, group,    p.rows};
  const long long rows = (long long)(PAIR ? min(p.num_tokens, p.unit_tokens) : p.num_tokens) * group;
  const long long usual = 2 * ((long long)p.num_tokens * group / p.batch) + 1;
  return launch_unit_merge<HD, F16>(cfg, pl.grid, rows, usual, m);
}

bool known_shape(int num_q_heads, int num_kv_heads, int head_dim) {
  return num_q_heads / num_kv_heads <= kTile && (head_dim == 64 || head_dim == 128);
}

}  // namespace
}  // namespace vg

using namespace vg;

extern "C" size_t vg_cross_workspace_bytes(int batch, int num_tokens, int num_q_heads, int num_kv_heads,
                                           int head_dim) {
  if (batch <= 0 || num_tokens <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads || !known_shape(num_q_heads, num_kv_heads, head_dim))
    return 0;
  return make_cross_plan(num_tokens, num_q_heads / num_kv_heads, num_kv_heads, head_dim).bytes;
}

extern "C" vg_status vg_cross_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                        const void* v, int64_t v_stride, int type, const int32_t* cu_q,
                                        const int32_t* state_starts, const int32_t* state_lens,
                                        const uint8_t* mask, int batch, int num_tokens, int num_states,
                                        int num_q_heads, int num_kv_heads, int head_dim,
                                        float softmax_scale, void* out, int64_t out_stride, float* lse,
                                        void* workspace, size_t workspace_bytes, int32_t* error_flag,
                                        cudaStream_t stream) {
  if (!cu_q || !state_starts || !state_lens || batch <= 0 || num_tokens < 0 || num_states < 0 ||
      num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || !(softmax_scale > 0.f) ||
      softmax_scale == INFINITY || num_q_heads % num_kv_heads)
    return VG_ERR_INVALID_ARGUMENT;
  if (type != VG_TYPE_BF16 && type != VG_TYPE_FP16) return VG_ERR_UNSUPPORTED;
  if (!known_shape(num_q_heads, num_kv_heads, head_dim) || batch > kMaxBatch || num_states > (1 << 30))
    return VG_ERR_UNSUPPORTED;
  if (num_tokens == 0) return VG_OK;
  const int64_t row = (int64_t)num_q_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
  auto bad = [](const void* x, int64_t stride, int64_t least) {
    return !x || (reinterpret_cast<uintptr_t>(x) & 15) || stride < least || stride % 8 ||
           stride >= ((int64_t)1 << 38);
  };
  if (bad(q, q_stride, row) || bad(out, out_stride, row) ||
      (num_states > 0 && (bad(k, k_stride, kv_row) || bad(v, v_stride, kv_row))))
    return VG_ERR_INVALID_ARGUMENT;
  const int g = num_q_heads / num_kv_heads;
  const CrossPlan pl = make_cross_plan(num_tokens, g, num_kv_heads, head_dim);
  if (!workspace || workspace_bytes < pl.bytes) return VG_ERR_WORKSPACE_TOO_SMALL;
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return VG_ERR_INVALID_ARGUMENT;
  // without states there is nothing to map: Q stands in (a tile that is loaded
  // for rows without states is never used)
  const bool none = num_states == 0;
  // (Q of few rows: as many tokens as have 32)
  CUtensorMap tq, tf, tk, tv;
  // Pairs of heads: where sequences have at most 128 rows of a head on average (a
  // pair's unit has one row tile of each, so longer ones load K and V twice as
  // often), and past 32 only where a CTA has several tiles (a pair's divided units have
  // twice the rows to merge; the buffer's states decide, as lengths are on the device).
  // us in pairs and one by one, 16 heads, 1500 states: 64 sequences of 4 rows 72 and
  // 101, 32 rows 75 and 100, 33 rows 78 and 107, 128 rows 83 and 106, 160 rows 154 and
  // 133; 6 sequences of 64 rows 19.6 and 20.6, of 128 rows 20.7 both; 2 of 128 rows 16.7
  // and 14.3; 1, 2 and 6 of 1 row 10.0, 11.6 and 16.6 against 10.3, 12.0 and 18.0.
  const int64_t rows = (int64_t)num_tokens * g;
  const bool many = (int64_t)num_states * num_kv_heads >= (int64_t)7 * kTile * pl.grid;
  const bool pairs = may_pair(g, num_kv_heads, head_dim) && rows <= (int64_t)(many ? kTile : 32) * batch;
  const int few = g > 32 ? 0 : 32 / g, wide = pairs ? 128 : head_dim;
  const int tile_tokens = pairs ? 2 * (kTile / (2 * g)) : kTile / g;
  const int heads = pairs ? num_kv_heads / 2 : num_kv_heads;
  const int there = none ? num_tokens : num_states, mapped = none ? (pairs ? num_q_heads / 2 : num_q_heads) : heads;
  if (!head_tile_tensor_map(none ? q : k, there, mapped, wide, none ? q_stride : k_stride, kTile, &tk) ||
      !head_tile_tensor_map(none ? q : v, there, mapped, wide, none ? q_stride : v_stride, kTile, &tv) ||
      !token_rows_tensor_map(q, num_tokens, num_q_heads, head_dim, q_stride, g, tile_tokens, &tq) ||
      !token_rows_tensor_map(q, num_tokens, num_q_heads, head_dim, q_stride, g, few ? few : 1, &tf))
    return VG_ERR_LAUNCH;
  CrossParams p = {};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.cu_q = cu_q;
  p.starts = state_starts;
  p.lens = state_lens;
  p.mask = mask;
  p.out = static_cast<uint16_t*>(out);
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
  p.num_states = num_states;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = g;
  p.rows = pl.rows;
  p.heads = heads;
  p.tile_tokens = tile_tokens;
  p.few_tokens = few;
  p.unit_tokens = pairs ? tile_tokens : 2 * tile_tokens;
  p.by_unit_tokens = p.unit_tokens == 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + p.unit_tokens - 1) / p.unit_tokens);
  const bool f16 = type == VG_TYPE_FP16;
  auto launch = [&](auto kernel_of_type) { return kernel_of_type(pl, tq, tf, tk, tv, p, stream); };
  const cudaError_t e = head_dim == 128 ? launch(f16 ? launch_cross<128, true, false> : launch_cross<128, false, false>)
                        : pairs         ? launch(f16 ? launch_cross<64, true, true> : launch_cross<64, false, true>)
                                        : launch(f16 ? launch_cross<64, true, false> : launch_cross<64, false, false>);
  return e == cudaSuccess ? VG_OK : VG_ERR_LAUNCH;
}
