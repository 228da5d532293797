// fh_kv_decode.cu -- attention over the paged NVFP4 cache for few query rows a
// request: single tokens, drafts, and whatever else does not fill a tile.
//
//   out[t, h] = sum_j p_j v[j, h / G],  p = softmax_j(sm_scale q[t, h] . k[j, h / G])
//
// with k, v = code * S * s_g read straight from the cache.  What a call cannot do
// without is reading it: at d = 128 a cached token of one KV head is 144 bytes,
// shared by the G query heads of its group.  64 requests of up to 8192 tokens, 8
// KV heads: 88.4 us, 59 % of the HBM rate.  No one unit is full (issue slots 57 %,
// ALU 49 %, tensor pipe 21 %): three warps a scheduler wait for their own
// conversions and products.
//
// Work split.  A tile is eight query rows (row = token * G + head in group)
// of one request and one KV head; its keys are cut into units of 128 tokens.
// All units of all tiles form one line, which the CTAs cut into equal pieces,
// so ragged requests load the GPU evenly.  A tile that lies within one CTA's
// piece is finished there.  One that spans several leaves a partial result per
// CTA in the workspace, and the CTA that finishes last (an atomic count; nobody
// waits) joins them in the order of the pieces, so results do not depend on
// who was last.
//
// Inside a CTA each of four warps takes 32 tokens of a unit, with a running
// maximum, sum and output of its own, and feeds itself through a private ring
// of cp.async stages; there is no block barrier in the loop.  The products run
// on mma.m16n8k16 (FP16 operands, FP32 sums) with the cached tokens as the
// 16-row operand: queries are the 8-wide one, so eight rows a KV head waste
// nothing, where a 128-row tcgen05 tile would be idle to 94%.  Orders of d and
// of tokens inside the products are free, and chosen so that
//   - a lane's K operand is 16 consecutive code bytes (32 for the pair of rows)
//     and the block scale multiplies in registers: code * S has 6 significant
//     bits, exact in FP16;
//   - a lane's V operand interleaves the nibbles of two tokens before the
//     conversion, so V needs no transposition;
//   - the probabilities go from the accumulator layout to the operand layout
//     with one movmatrix per 8 x 8.
// Query rows go to FP16 scaled by a power of two (query_exponent), which loses
// nothing that a BF16 row has.  Probabilities are rounded to FP16 (2^-11,
// against 2^-8 of the BF16 output); they are kept below 2^(6 + 8): a warp's
// maximum is only raised when a score exceeds it by more than 8 (in log2), and
// P is 2^(s - m + 6), so that small weights down to 2^-30 of the largest count.
// Maxima, sums and outputs are FP32.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fh_internal.h"
#include "fh_kv.cuh"
#include "fh_kv_attn.h"

namespace fh {

namespace {

using namespace kv;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTileRows = 8;                // query rows of a tile
constexpr int kUnit = 128;                  // tokens of a unit
constexpr int kWarpTokens = kUnit / kWarps; // 32
constexpr int kStages = 3;
constexpr int kMaxCtas = kCounters;         // workspace bound: a counter and two partial tiles per CTA
constexpr float kRaise = 8.0f;              // log2: how far a score may exceed the running maximum
constexpr float kHead = 6.0f;               // log2: head room of P above 1

template <int D>
struct Stage {  // bytes of one warp's stage
  static constexpr int kCodes = kWarpTokens * D / 2;
  static constexpr int kScales = kWarpTokens * D / 16;
  static constexpr int kBytes = 2 * (kCodes + kScales);
  static constexpr int kOffKs = kCodes, kOffV = kCodes + kScales, kOffVs = 2 * kCodes + kScales;
};

template <int D>
struct Smem {
  static constexpr int kRing = kWarps * kStages * Stage<D>::kBytes;
  static constexpr int kRowFloats = D + 4;
  static constexpr int kO = kWarps * kTileRows * kRowFloats * 4;
  static constexpr int kMl = kWarps * kTileRows * 8;
  static constexpr int kBytes = kRing + kO + kMl;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes global -> shared; zeros when !live (src is not read then).
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// a / b for a, b >= 0; 32-bit wherever that does (a 64-bit division is some 150 instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// The line of units.  A request's tiles all run over its units [u_lo, u_hi).
struct Walk {
  int b, tile, head, unit;  // the current unit
  Request rq;
  int u_lo, n_units, n_tiles;
};

__device__ __forceinline__ void load_walk(const AttnParams& p, int R, Walk& w) {
  w.rq = load_request(p, w.b);
  w.u_lo = w.rq.lo / kUnit;
  w.n_units = max(1, (w.rq.hi + kUnit - 1) / kUnit - w.u_lo);  // a row that sees nothing is written all the same
  w.n_tiles = (int)(((int64_t)w.rq.n_q * p.group + R - 1) / R);
}

__device__ __forceinline__ int64_t walk_weight(const AttnParams& p, const Walk& w) {
  return (int64_t)w.n_tiles * p.kv_heads * w.n_units;
}

// One unit on; the requests behind an exhausted one that have no rows are skipped.
__device__ __forceinline__ void advance(const AttnParams& p, int R, Walk& w) {
  if (++w.unit < w.n_units) return;
  w.unit = 0;
  if (++w.head < p.kv_heads) return;
  w.head = 0;
  if (++w.tile < w.n_tiles) return;
  w.tile = 0;
  while (++w.b < p.batch) {
    load_walk(p, R, w);
    if (w.n_tiles > 0) return;
  }
}

// The 16 values of one MMA operand pair from two tokens' words of eight
// nibbles: E holds the even nibbles (token x in the low half of each byte), O the odd ones.
__device__ __forceinline__ void interleave(uint32_t x, uint32_t y, uint32_t& even, uint32_t& odd) {
  even = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
  odd = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 3) kv_decode_kernel(const __grid_constant__ AttnParams p) {
  constexpr int R = kTileRows;
  constexpr int kMt = D / 16;            // 16-row tiles of the output's d
  using St = Stage<D>;
  using Sm = Smem<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long scan_s[kWarps];
  __shared__ int start_s[4];
  __shared__ int last_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  float* o_s = reinterpret_cast<float*>(smem + Sm::kRing);                  // [warp][R][D + 4]
  float2* ml_s = reinterpret_cast<float2*>(smem + Sm::kRing + Sm::kO);      // [warp][R]
  const uint32_t ring = smem_addr(smem) + warp * (kStages * St::kBytes);
  const uint8_t* ring_p = smem + warp * (kStages * St::kBytes);
  wait_for_preceding();

  // --- this CTA's piece of the line ------------------------------------------------
  Walk w;
  const int2 share = share_of_requests(p, tid, kThreads);
  const int rb0 = share.x, rb1 = share.y;
  long long mine = 0;
  for (int b = rb0; b < rb1; ++b) {
    w.b = b;
    load_walk(p, R, w);
    mine += walk_weight(p, w);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan_s[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += scan_s[i];
    total += scan_s[i];
  }
  // No piece is empty, so a tile's pieces are those of consecutive CTAs.
  const long long ctas = min((long long)gridDim.x, total);
  if (blockIdx.x >= ctas) return;
  const long long u0 = quotient(blockIdx.x * total, ctas), u1 = quotient((blockIdx.x + 1) * total, ctas);
  if (u0 >= before && u0 < before + mine) {  // exactly one thread
    long long rest = u0 - before;
    for (int b = rb0; b < rb1; ++b) {
      w.b = b;
      load_walk(p, R, w);
      const long long weight = walk_weight(p, w);
      if (rest < weight) {
        start_s[0] = b;
        const long long per_tile = (long long)p.kv_heads * w.n_units, tile = quotient(rest, per_tile);
        const long long in_tile = rest - tile * per_tile, head = quotient(in_tile, w.n_units);
        start_s[1] = (int)tile;
        start_s[2] = (int)head;
        start_s[3] = (int)(in_tile - head * w.n_units);
        break;
      }
      rest -= weight;
    }
  }
  __syncthreads();
  Walk f;  // the unit to fetch next
  f.b = start_s[0];
  load_walk(p, R, f);
  f.tile = start_s[1];
  f.head = start_s[2];
  f.unit = start_s[3];
  int n_left = (int)(u1 - u0), n_fetch = n_left;  // (2^31 units would take a CTA a quarter of an hour)
  long long at = u0;  // the line's index of the current unit

  // --- fetching: this warp's 32 tokens of a unit into a stage ---------------------
  // The pages of the unit to fetch are looked up one unit ahead.
  int next_page[2];
  auto look_up = [&]() {
    const int tok0 = (f.u_lo + f.unit) * kUnit + warp * kWarpTokens;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // A group of 16 tokens lies in one page (page sizes are multiples of 16).
      const int tok = tok0 + 16 * h;
      next_page[h] = -1;
      if (tok < f.rq.hi && tok + 16 > f.rq.lo) next_page[h] = p.table[(int64_t)f.b * p.max_pages + (tok >> p.page_shift)];
    }
  };
  // A lane's 16 bytes of eight rows of codes (d = 128; of sixteen at d = 64) lie at
  // 16 * lane behind the first row.  K goes to the operands' row order, V's
  // pieces are turned within a row so that reading them meets no bank twice.
  constexpr int kCpr = D / 32;                             // 16-byte pieces of a row of codes
  constexpr int kCopies = kWarpTokens * kCpr / 32;         // of K, and of V: 4 or 2
  constexpr int kCopyRows = 32 / kCpr;
  const int copy_row = lane / kCpr, copy_part = lane % kCpr;
  const uint32_t k_dst = ((copy_row & ~7) | (2 * (copy_row & 3) + ((copy_row >> 2) & 1))) * (D / 2) + 16 * copy_part;
  const uint32_t v_dst = St::kOffV + copy_row * (D / 2) + 16 * (D == 128 ? copy_part ^ (copy_row & 2) : copy_part);
  // Scales: lanes 0 .. kScaleCopies - 1 K's, as many behind them V's.
  constexpr int kScaleCopies = St::kScales / 16;
  const bool scale_v = lane >= kScaleCopies, scale_second = (lane % kScaleCopies) >= kScaleCopies / 2;
  const uint8_t* scale_src = (scale_v ? p.v_scales : p.k_scales) + 16 * (lane % (kScaleCopies / 2));
  const uint32_t scale_dst = (scale_v ? St::kOffVs : St::kOffKs) + 16 * (lane % kScaleCopies);
  const uint32_t page_tokens = (uint32_t)p.kv_heads << p.page_shift;  // at most 2^22
  auto fetch = [&](int stage) {
    const uint32_t base = ring + stage * St::kBytes;
    const uint32_t tok0 = (f.u_lo + f.unit) * kUnit + warp * kWarpTokens, mask = (1u << p.page_shift) - 1;
    bool live[2];
    uint64_t scale_at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      live[h] = next_page[h] >= 0 && next_page[h] < p.num_pages;
      const uint32_t page = live[h] ? next_page[h] : 0;
      const uint32_t in_page = ((uint32_t)f.head << p.page_shift) + ((tok0 + 16 * h) & mask);
      const uint64_t at = (uint64_t)page * (page_tokens * (D / 2)) + (in_page * (D / 2) + 16 * lane);
      scale_at[h] = (uint64_t)page * (page_tokens * (D / 16)) + in_page * (D / 16);
#pragma unroll
      for (int i = 0; i < kCopies / 2; ++i) {
        const int k = h * (kCopies / 2) + i;
        copy16(base + k_dst + k * (kCopyRows * D / 2), p.k_codes + at + i * 512, live[h]);
        copy16(base + v_dst + k * (kCopyRows * D / 2), p.v_codes + at + i * 512, live[h]);
      }
    }
    if (lane < 2 * kScaleCopies)
      copy16(base + scale_dst, scale_src + (scale_second ? scale_at[1] : scale_at[0]), scale_second ? live[1] : live[0]);
    return (live[0] ? 1 : 0) | (live[1] ? 2 : 0);
  };
  // Which groups of the stages in flight are there: two bits a stage.
  uint32_t live_bits = 0;
  int fetch_stage = 0;
  auto fetch_next = [&]() {
    if (n_fetch > 0) {
      const uint32_t lv = fetch(fetch_stage);
      live_bits = (live_bits & ~(3u << (2 * fetch_stage))) | (lv << (2 * fetch_stage));
      if (--n_fetch > 0) {
        advance(p, R, f);
        look_up();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fetch_stage = fetch_stage + 1 == kStages ? 0 : fetch_stage + 1;
  };
  // Query rows of a segment: this lane's quarter of row g.
  uint4 raws[D / 32];
  auto load_query = [&]() {
    const int n_rows = (int)min((int64_t)R, (int64_t)w.rq.n_q * p.group - (int64_t)w.tile * R);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) raws[i] = make_uint4(0, 0, 0, 0);
    if (g < n_rows) {
      const uint32_t row = (uint32_t)w.tile * R + g, ti = query_of_row(p, row), hd = row - ti * p.group;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(w.rq.row0 + ti) * p.ldq +
                                                        (int64_t)(w.head * p.group + hd) * D + t * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raws[i] = src[i];
    }
  };
  w = f;  // (before it is advanced any further)
  look_up();
  load_query();
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) fetch_next();
  int stage = 0;

  bool first_segment = true;
  while (n_left > 0) {
    // --- a segment: consecutive units of one tile ---------------------------------
    const int seg_tile = w.tile, seg_head = w.head, seg_unit0 = w.unit, n_units = w.n_units;
    const Request rq = w.rq;
    const int seg_tok0 = (w.u_lo + seg_unit0) * kUnit + warp * kWarpTokens;
    const int seg_n = min(n_left, n_units - seg_unit0);
    const int n_rows = (int)min((int64_t)R, (int64_t)rq.n_q * p.group - (int64_t)seg_tile * R);

    // The query as FP16, scaled by a power of two; and what the lane's accumulator
    // columns need.
    uint32_t qf[D / 8];
    float factor[2];
    int lo_q[2], hi_q[2];
    int lo_max = 0, hi_min = rq.hi;
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t v[4] = {raws[i].x, raws[i].y, raws[i].z, raws[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) amax = max(amax, max(v[k] & 0x7FFFu, (v[k] >> 16) & 0x7FFFu));
    }
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
    const int e = query_exponent(amax);
    // A negative scale goes to the query, so that larger scores are larger sums.
    const float up = p.qk_scale < 0.0f ? -pow2(e) : pow2(e);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t v[4] = {raws[i].x, raws[i].y, raws[i].z, raws[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) qf[4 * i + k] = pack_f16x2(bf16_lo(v[k]) * up, bf16_hi(v[k]) * up);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = 2 * t + c;
      factor[c] = score_factor(p, __shfl_sync(0xFFFFFFFFu, e, 4 * col));
      const int2 s = col < n_rows ? seen_by(p, rq, (int)query_of_row(p, (uint32_t)seg_tile * R + col)) : make_int2(0, rq.hi);
      lo_q[c] = s.x;
      hi_q[c] = s.y;
      lo_max = max(lo_max, s.x);
      hi_min = min(hi_min, s.y);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lo_max = max(lo_max, __shfl_xor_sync(0xFFFFFFFFu, lo_max, o));
      hi_min = min(hi_min, __shfl_xor_sync(0xFFFFFFFFu, hi_min, o));
    }

    float acc[kMt][4];
    float m[2], l[2];
#pragma unroll
    for (int i = 0; i < kMt; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0.0f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;

    for (int u = 0; u < seg_n; ++u) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();
      const uint8_t* sb = ring_p + stage * St::kBytes;
      const int tok0 = seg_tok0 + u * kUnit;
      const uint32_t lv = (live_bits >> (2 * stage)) & 3u;
      const bool edge = lv != 3u || tok0 < lo_max || tok0 + kWarpTokens > hi_min;
      if (lv != 0u && tok0 < rq.hi) {
        if (tok0 < rq.lo || tok0 + kWarpTokens > rq.hi) {
          // Scales in front of the first token seen and behind the last are whatever
          // the page holds: as zeros they cannot bring a NaN into sums that weigh
          // them with zero.
          uint8_t* vs = const_cast<uint8_t*>(sb) + St::kOffVs + lane * (D / 16);
          if (tok0 + lane < rq.lo || tok0 + lane >= rq.hi) {
            if constexpr (D == 128)
              *reinterpret_cast<uint2*>(vs) = make_uint2(0, 0);
            else
              *reinterpret_cast<uint32_t*>(vs) = 0;
          }
          __syncwarp();
        }
        // --- scores: s[i][c] for the tokens of the 16-row tile i -----------------
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int c = 0; c < 4; ++c) s[i][c] = 0.0f;
          uint32_t ka[D / 32], kb[D / 32];  // rows g and g + 8: D / 4 nibbles each
          uint32_t sa, sb2;
          const int tok_g = (g >> 1) + 4 * (g & 1);  // the token that operand row g holds
          if constexpr (D == 128) {
            const uint4 a = *reinterpret_cast<const uint4*>(sb + (16 * i + g) * 64 + 16 * t);
            const uint4 b = *reinterpret_cast<const uint4*>(sb + (16 * i + g + 8) * 64 + 16 * t);
            ka[0] = a.x, ka[1] = a.y, ka[2] = a.z, ka[3] = a.w;
            kb[0] = b.x, kb[1] = b.y, kb[2] = b.z, kb[3] = b.w;
            sa = *reinterpret_cast<const uint16_t*>(sb + St::kOffKs + (16 * i + tok_g) * 8 + 2 * t);
            sb2 = *reinterpret_cast<const uint16_t*>(sb + St::kOffKs + (16 * i + 8 + tok_g) * 8 + 2 * t);
          } else {
            const uint2 a = *reinterpret_cast<const uint2*>(sb + (16 * i + g) * 32 + 8 * t);
            const uint2 b = *reinterpret_cast<const uint2*>(sb + (16 * i + g + 8) * 32 + 8 * t);
            ka[0] = a.x, ka[1] = a.y;
            kb[0] = b.x, kb[1] = b.y;
            sa = sb[St::kOffKs + (16 * i + tok_g) * 4 + t];
            sb2 = sb[St::kOffKs + (16 * i + 8 + tok_g) * 4 + t];
          }
          const uint32_t ha = e4m3x2_to_f16x2(sa), hb = e4m3x2_to_f16x2(sb2);
#pragma unroll
          for (int wd = 0; wd < D / 32; ++wd) {  // a word is eight nibbles: two k steps
            // A lane's nibbles are 32 (two blocks) at d = 128, 16 (one block) at d = 64.
            const uint32_t xa = __byte_perm(ha, ha, (D == 128 && wd >= 2) ? 0x3232 : 0x1010);
            const uint32_t xb = __byte_perm(hb, hb, (D == 128 && wd >= 2) ? 0x3232 : 0x1010);
            const uint32_t a0 = hmul2(e2m1x2_to_f16x2<0>(ka[wd]), xa), a2 = hmul2(e2m1x2_to_f16x2<1>(ka[wd]), xa);
            const uint32_t a1 = hmul2(e2m1x2_to_f16x2<0>(kb[wd]), xb), a3 = hmul2(e2m1x2_to_f16x2<1>(kb[wd]), xb);
            mma_16816(s[i], a0, a1, a2, a3, qf[4 * wd], qf[4 * wd + 1]);
            const uint32_t c0 = hmul2(e2m1x2_to_f16x2<2>(ka[wd]), xa), c2 = hmul2(e2m1x2_to_f16x2<3>(ka[wd]), xa);
            const uint32_t c1 = hmul2(e2m1x2_to_f16x2<2>(kb[wd]), xb), c3 = hmul2(e2m1x2_to_f16x2<3>(kb[wd]), xb);
            mma_16816(s[i], c0, c1, c2, c3, qf[4 * wd + 2], qf[4 * wd + 3]);
          }
        }
        // --- scores of tokens not seen ---------------------------------------------------
        if (edge) {
          const int tok_g = (g >> 1) + 4 * (g & 1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const bool there = (lv >> i) & 1u;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int tok = tok0 + 16 * i + 8 * (c >> 1) + tok_g;
              if (!there || tok < lo_q[c & 1] || tok >= hi_q[c & 1]) s[i][c] = -INFINITY;
            }
          }
        }
        // --- running maximum: raised only when a score is well above it ------------------
        bool raise = false;
        float top[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          // In log2 units (the factor is > 0).
          top[c] = fmaxf(fmaxf(s[0][c], s[0][c + 2]), fmaxf(s[1][c], s[1][c + 2])) * factor[c];
          raise = raise || top[c] > m[c] + kRaise;
        }
        if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = top[c];
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
            const float mn = fmaxf(m[c], v);
            const float keep = m[c] == mn ? 1.0f : exp2_fast(m[c] - mn);  // 0 from -inf
            m[c] = mn;
            l[c] *= keep;
#pragma unroll
            for (int k = 0; k < kMt; ++k) {
              acc[k][c] *= keep;
              acc[k][c + 2] *= keep;
            }
          }
        }
        // --- P = 2^(s - m + 6), its sum, and its operand layout ----------------------------
        uint32_t pb[2][2];
        const float off0 = m[0] == -INFINITY ? 0.0f : kHead - m[0];
        const float off1 = m[1] == -INFINITY ? 0.0f : kHead - m[1];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float p0 = exp2_fast(fmaf(s[i][0], factor[0], off0)), p1 = exp2_fast(fmaf(s[i][1], factor[1], off1));
          const float p2 = exp2_fast(fmaf(s[i][2], factor[0], off0)), p3 = exp2_fast(fmaf(s[i][3], factor[1], off1));
          l[0] += p0 + p2;
          l[1] += p1 + p3;
          pb[i][0] = transpose8x8(pack_f16x2(p0, p1));
          pb[i][1] = transpose8x8(pack_f16x2(p2, p3));
        }
        // --- O^T += V^T P^T ------------------------------------------------------------------
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* vb = sb + St::kOffV;
          const uint8_t* vs = sb + St::kOffVs + 16 * i * (D / 16);
          const int blk = D == 128 ? g : g >> 1;
          const uint32_t h01 = e4m3x2_to_f16x2((uint32_t)vs[t * (D / 16) + blk] | ((uint32_t)vs[(t + 4) * (D / 16) + blk] << 8));
          const uint32_t h23 =
              e4m3x2_to_f16x2((uint32_t)vs[(t + 8) * (D / 16) + blk] | ((uint32_t)vs[(t + 12) * (D / 16) + blk] << 8));
          constexpr int kW = D / 64;  // words of a lane's d range: 2 (16 values) or 1 (8 values)
          uint32_t v[4][kW];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 16 * i + t + 4 * k;
            if constexpr (D == 128) {
              const uint2 x = *reinterpret_cast<const uint2*>(vb + row * 64 + 16 * ((g >> 1) ^ (row & 2)) + 8 * (g & 1));
              v[k][0] = x.x;
              v[k][1] = x.y;
            } else {
              v[k][0] = *reinterpret_cast<const uint32_t*>(vb + row * 32 + 4 * g);
            }
          }
          // The output's 16-row tile mt has the lane's d value mt in row g and
          // value mt + D / 16 in row g + 8.
          if constexpr (D == 128) {
            uint32_t e0, o0, e1, o1, e2, o2, e3, o3;
            interleave(v[0][0], v[1][0], e0, o0);  // values 0..7, tokens t, t + 4
            interleave(v[0][1], v[1][1], e1, o1);  // values 8..15
            interleave(v[2][0], v[3][0], e2, o2);  // tokens t + 8, t + 12
            interleave(v[2][1], v[3][1], e3, o3);
            auto out = [&](uint32_t a, uint32_t b, uint32_t c, uint32_t d, int mt) {
              mma_16816(acc[mt], a, b, c, d, pb[i][0], pb[i][1]);
            };
#define FH_KV_MT(byte)                                                                                              \
  out(hmul2(e2m1x2_to_f16x2<byte>(e0), h01), hmul2(e2m1x2_to_f16x2<byte>(e1), h01),                                 \
      hmul2(e2m1x2_to_f16x2<byte>(e2), h23), hmul2(e2m1x2_to_f16x2<byte>(e3), h23), 2 * byte);                      \
  out(hmul2(e2m1x2_to_f16x2<byte>(o0), h01), hmul2(e2m1x2_to_f16x2<byte>(o1), h01),                                 \
      hmul2(e2m1x2_to_f16x2<byte>(o2), h23), hmul2(e2m1x2_to_f16x2<byte>(o3), h23), 2 * byte + 1);
            FH_KV_MT(0)
            FH_KV_MT(1)
            FH_KV_MT(2)
            FH_KV_MT(3)
#undef FH_KV_MT
          } else {
            uint32_t e0, o0, e2, o2;
            interleave(v[0][0], v[1][0], e0, o0);
            interleave(v[2][0], v[3][0], e2, o2);
            auto out = [&](uint32_t a, uint32_t b, uint32_t c, uint32_t d, int mt) {
              mma_16816(acc[mt], a, b, c, d, pb[i][0], pb[i][1]);
            };
            // Values 0..3 are bytes 0 and 1, values 4..7 bytes 2 and 3.
            out(hmul2(e2m1x2_to_f16x2<0>(e0), h01), hmul2(e2m1x2_to_f16x2<2>(e0), h01),
                hmul2(e2m1x2_to_f16x2<0>(e2), h23), hmul2(e2m1x2_to_f16x2<2>(e2), h23), 0);
            out(hmul2(e2m1x2_to_f16x2<0>(o0), h01), hmul2(e2m1x2_to_f16x2<2>(o0), h01),
                hmul2(e2m1x2_to_f16x2<0>(o2), h23), hmul2(e2m1x2_to_f16x2<2>(o2), h23), 1);
            out(hmul2(e2m1x2_to_f16x2<1>(e0), h01), hmul2(e2m1x2_to_f16x2<3>(e0), h01),
                hmul2(e2m1x2_to_f16x2<1>(e2), h23), hmul2(e2m1x2_to_f16x2<3>(e2), h23), 2);
            out(hmul2(e2m1x2_to_f16x2<1>(o0), h01), hmul2(e2m1x2_to_f16x2<3>(o0), h01),
                hmul2(e2m1x2_to_f16x2<1>(o2), h23), hmul2(e2m1x2_to_f16x2<3>(o2), h23), 3);
          }
        }
      }
      __syncwarp();  // every lane has read the stage before it is fetched into again
      fetch_next();
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }

    // --- the next segment's query is on its way while this one is finished ------------
    if (n_left > seg_n) {
      w.unit += seg_n - 1;
      advance(p, R, w);
      load_query();
    }
    // --- join the four warps -----------------------------------------------------------
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float v = l[c];
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
      const int row = 2 * t + c;
      if (g == 0) ml_s[warp * R + row] = make_float2(m[c], v);
      // The lane's d values are contiguous: D / 8 from g * D / 8.
      float* dst = o_s + (warp * R + row) * Sm::kRowFloats + g * (D / 8);
#pragma unroll
      for (int k = 0; k < kMt; k += 4) {
        *reinterpret_cast<float4*>(dst + k) =
            make_float4(acc[k][c], acc[k + 1][c], acc[k + 2][c], acc[k + 3][c]);
        *reinterpret_cast<float4*>(dst + kMt + k) =
            make_float4(acc[k][c + 2], acc[k + 1][c + 2], acc[k + 2][c + 2], acc[k + 3][c + 2]);
      }
    }
    __syncthreads();
    const bool whole = seg_n == n_units;
    const int part = 2 * (int)blockIdx.x + (first_segment ? 0 : 1);
    auto store_row = [&](int row, int d, float4 o, float mm, float ll) {
      const uint32_t rr = (uint32_t)seg_tile * R + row, ti = query_of_row(p, rr);
      const int64_t tok = rq.row0 + (int64_t)ti;
      const int head = seg_head * p.group + (int)(rr - ti * p.group);
      const float inv = ll > 0.0f ? p.v_scale / ll : (ll == 0.0f ? 0.0f : ll);  // a NaN stays one
      const float unit = p.v_unit;
      uint2 v = make_uint2(pack_bf16x2(o.x * inv * unit, o.y * inv * unit), pack_bf16x2(o.z * inv * unit, o.w * inv * unit));
      *reinterpret_cast<uint2*>(p.out + tok * p.ldo + (int64_t)head * D + d) = v;
      if (d == 0 && p.lse != nullptr)
        p.lse[tok * p.q_heads + head] = ll == 0.0f ? -INFINITY : (mm - kHead + log2f(ll)) * 0.6931471805599453f;
    };
    // What the warps have left in o_s and ml_s, as one: emit(row, d, output, maximum, sum).
    auto join_warps = [&](auto emit) {
      for (int i = tid; i < n_rows * (D / 4); i += kThreads) {
        const int row = i / (D / 4), d = 4 * (i % (D / 4));
        float mm = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, ml_s[k * R + row].x);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float ll = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float2 ml = ml_s[k * R + row];
          const float c = ml.x == mm ? 1.0f : exp2_fast(ml.x - mm);
          const float4 x = *reinterpret_cast<const float4*>(o_s + (k * R + row) * Sm::kRowFloats + d);
          o.x += c * x.x;
          o.y += c * x.y;
          o.z += c * x.z;
          o.w += c * x.w;
          ll += c * ml.y;
        }
        emit(row, d, o, mm, ll);
      }
    };
    if (whole) {
      join_warps(store_row);
    } else {
      join_warps([&](int row, int d, float4 o, float mm, float ll) {
        *reinterpret_cast<float4*>(p.part_o + ((int64_t)part * R + row) * D + d) = o;
        if (d == 0) p.part_ml[(int64_t)part * R + row] = make_float2(mm, ll);
      });
    }
    if (!whole) {
      // The pieces of this tile: CTA i has the line's units from i * total / ctas on.
      const long long a = at - seg_unit0, z = a + n_units - 1;
      const int i0 = (int)quotient((a + 1) * ctas - 1, total), i1 = (int)quotient((z + 1) * ctas - 1, total);
      __threadfence();
      __syncthreads();
      // A CTA is the first of at most one tile that goes on behind it, so the
      // count at its index is this tile's alone.
      if (tid == 0) last_s = atomicAdd(p.count + i0, 1u) == (unsigned)(i1 - i0);
      __syncthreads();
      if (last_s) {
        __threadfence();
        const int slot0 = 2 * i0 + (quotient(i0 * total, ctas) == a ? 0 : 1);
        // Few pieces: a thread an output.  Many: each warp joins every fourth piece of
        // all outputs and leaves what it has where the warps' own results were.
        const bool many = i1 - i0 >= 16;
        const int by = many ? kWarps : 1;
        for (int i = many ? lane : tid; i < n_rows * (D / 4); i += many ? 32 : kThreads) {
          const int row = i / (D / 4), d = 4 * (i % (D / 4));
          float mm = -INFINITY, ll = 0.0f;
          float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          for (int c0 = i0 + (many ? warp : 0); c0 <= i1; c0 += 8 * by) {  // eight pieces' loads at a time
            float2 ml[8];
            float4 x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int c = c0 + k * by;
              ml[k] = make_float2(-INFINITY, 0.0f);
              x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              if (c <= i1) {
                const int64_t slot = (int64_t)(c == i0 ? slot0 : 2 * c) * R + row;
                ml[k] = __ldcg(p.part_ml + slot);
                x[k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + slot * D + d));
              }
            }
            float mn = mm;
#pragma unroll
            for (int k = 0; k < 8; ++k) mn = fmaxf(mn, ml[k].x);
            const float keep = mm == mn ? 1.0f : exp2_fast(mm - mn);
            o.x *= keep, o.y *= keep, o.z *= keep, o.w *= keep;
            ll *= keep;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float add = ml[k].x == mn ? 1.0f : exp2_fast(ml[k].x - mn);
              o.x += add * x[k].x;
              o.y += add * x[k].y;
              o.z += add * x[k].z;
              o.w += add * x[k].w;
              ll += add * ml[k].y;
            }
            mm = mn;
          }
          if (!many) {
            store_row(row, d, o, mm, ll);
          } else {
            *reinterpret_cast<float4*>(o_s + (warp * R + row) * Sm::kRowFloats + d) = o;
            if (d == 0) ml_s[warp * R + row] = make_float2(mm, ll);
          }
        }
        if (many) {
          __syncthreads();
          join_warps(store_row);
        }
        if (tid == 0) p.count[i0] = 0;  // as the next call needs it
      }
    }
    first_segment = false;
    at += seg_n;
    n_left -= seg_n;
    __syncthreads();  // o_s and ml_s are written again by the next segment
  }
}

template <int D>
cudaError_t launch_decode(const AttnParams& p, int64_t ctas, cudaStream_t s) {
  using Sm = Smem<D>;
  static DeviceTable resident;  // CTAs an SM holds
  int dev = 0;
  cudaGetDevice(&dev);
  const int per_sm = per_device(resident, dev, [](int) {
    cudaError_t e =
        cudaFuncSetAttribute(kv_decode_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::kBytes);
    int n = 0;
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kv_decode_kernel<D>, kThreads, Sm::kBytes);
    return e != cudaSuccess ? -(int)e : (n < 1 ? 1 : n);
  });
  if (per_sm <= 0) return (cudaError_t)(-per_sm);
  int64_t grid = (int64_t)sm_count() * per_sm;
  if (grid > kMaxCtas) grid = kMaxCtas;
  if (grid > ctas) grid = ctas;
  return launch_overlapping(kv_decode_kernel<D>, dim3((unsigned)grid), dim3(kThreads), Sm::kBytes, s, p);
}

}  // namespace

size_t kv_attn_split_workspace(const KvAttnShape& s) {
  // The counters, then two partial tiles per CTA.
  return kMaxCtas * sizeof(unsigned) + (size_t)2 * kMaxCtas * kTileRows * (size_t)(s.head_dim + 2) * sizeof(float);
}

// Tiles of all KV heads, at most.
int64_t split_tiles(const KvAttnShape& s) {
  const int64_t rows = s.total_q * (s.q_heads / s.kv_heads), most = rows < s.batch ? rows : s.batch;
  return (rows / kTileRows + most) * s.kv_heads;
}

double kv_attn_split_cost(const KvAttnShape& s, int64_t max_kv) {
  // Every 32 tokens of a tile take about 0.8 ns (0.5 at d = 64) on the whole GPU,
  // a tile 5 ns beside, and many requests of up to max_kv tokens have fewer.
  const double part = s.batch >= 8 ? 0.6 : 1.0, tiles = (double)split_tiles(s);
  return 9.0 + tiles * (0.005 + (s.head_dim == 64 ? 0.0005 : 0.0008) * part * (double)max_kv / kWarpTokens);
}

cudaError_t launch_kv_attn_split(const AttnParams& params, const KvAttnShape& shape, void* workspace, cudaStream_t s) {
  AttnParams p = params;
  p.count = static_cast<unsigned*>(workspace);
  p.part_o = reinterpret_cast<float*>(p.count + kMaxCtas);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)2 * kMaxCtas * kTileRows * shape.head_dim);
  // No more CTAs than there can be units; nor so many that joining a lone tile's
  // pieces takes longer than they save.
  const int64_t tiles = split_tiles(shape), per_tile = (shape.max_kv + kUnit - 1) / kUnit + 1;
  const int64_t ctas = tiles * (per_tile < 64 ? per_tile : 64);
  return shape.head_dim == 128 ? launch_decode<128>(p, ctas, s) : launch_decode<64>(p, ctas, s);
}

}  // namespace fh
