// fh_kv_attn.h -- what the two attention kernels over the NVFP4 cache share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fh_internal.h"
#include "fh_kv.cuh"

namespace fh {
namespace kv {

struct AttnParams {
  const uint16_t* q;  // BF16 [total_q, q_heads, d], tokens ldq elements apart
  uint16_t* out;      // BF16 [total_q, q_heads, d], tokens ldo elements apart
  float* lse;         // FP32 [total_q, q_heads] or null
  const uint8_t* k_codes;
  const uint8_t* k_scales;
  const uint8_t* v_codes;
  const uint8_t* v_scales;
  const int32_t* table;     // [batch, max_pages]
  const int32_t* lens;      // [batch]
  const int32_t* q_starts;  // [batch + 1]
  int64_t ldq, ldo, max_pages;
  int total_q, batch, q_heads, kv_heads, group;  // group = q_heads / kv_heads
  uint32_t group_magic;  // of the division by it, with group_shift (set_group)
  int group_shift;
  int page_shift, num_pages;
  int causal, window;
  int stall;        // test hook: the tile kernel's first CTA stops its products after two key tiles
  // sm_scale * log2(e) * k_gscale = qk_scale * 2^qk_exp, for scores in units of log2;
  // 0.5 <= |qk_scale| <= 1, or both are 0: the product may be outside FP32 where the
  // scores are not.
  float qk_scale;
  int qk_exp;
  // v_gscale = v_scale * v_unit, 1 <= v_scale < 2 and v_unit a power of two: outputs are
  // divided by the softmax's denominator in units of v_unit, since v_gscale / it may be
  // below FP32's normal range where the outputs are not.
  float v_scale, v_unit;
  // Workspace: partial results of key ranges split over CTAs, and their counters.
  float* part_o;        // [slots][rows][d], not normalised
  float2* part_ml;      // [slots][rows]: running maximum (log2 units) and sum
  unsigned int* count;  // zero between calls
};

// row / group for 0 <= row < 2^31: with s = ceil(log2 group) and m =
// floor(2^(31 + s) / group) + 1, m group exceeds 2^(31 + s) by at most 2^s, so
// that row m / 2^(31 + s) is above row / group by less than 1 / group.
inline void set_group(AttnParams* p, int group) {
  int s = 0;
  while (((int64_t)1 << s) < group) ++s;
  p->group = group;
  p->group_shift = s - 1;
  p->group_magic = group == 1 ? 0u : (uint32_t)(((uint64_t)1 << (31 + s)) / (uint64_t)group + 1);
}

__device__ __forceinline__ uint32_t query_of_row(const AttnParams& p, uint32_t row) {
  return p.group == 1 ? row : __umulhi(row, p.group_magic) >> p.group_shift;
}

// One request as every kernel reads it, with the lengths brought into range so
// that no index built from them leaves a buffer.
struct Request {
  int row0, n_q;  // first row of q, and how many
  int len;        // cached tokens
  int lo, hi;     // cached tokens that any of its queries may see: [lo, hi)
};

__device__ __forceinline__ Request load_request(const AttnParams& p, int b) {
  Request r;
  const int s = min(max(p.q_starts[b], 0), p.total_q), e = min(max(p.q_starts[b + 1], s), p.total_q);
  r.row0 = s;
  r.n_q = e - s;
  r.len = (int)min((int64_t)max(p.lens[b], 0), p.max_pages << p.page_shift);
  r.hi = r.len;
  r.lo = 0;
  if (p.window > 0) r.lo = (int)min((int64_t)r.hi, max((int64_t)0, (int64_t)r.len - r.n_q - p.window + 1));
  return r;
}

// What turns a row's sums into scores in units of log2, its query having been scaled
// by 2^e.  Never 0: a hidden score of -inf stays -inf times it.
__device__ __forceinline__ float score_factor(const AttnParams& p, int e) {
  return fmaxf(fabsf(p.qk_scale) * pow2(min(max(p.qk_exp - e, -126), 127)), 1.17549435e-38f);
}

// Thread i's share of the requests where `threads` share them: [x, y).  (Unsigned:
// with batch < 2^31 - 1, i per < 2^31 and i per + per < 2^32.)
__device__ __forceinline__ int2 share_of_requests(const AttnParams& p, uint32_t i, uint32_t threads) {
  const uint32_t n = (uint32_t)p.batch, per = (n - 1) / threads + 1, from = min(n, i * per);
  return make_int2((int)from, (int)min(n, from + per));
}

// The cached tokens [lo, hi) that query i of a request sees.
__device__ __forceinline__ int2 seen_by(const AttnParams& p, const Request& r, int i) {
  const int64_t pos = (int64_t)r.len - r.n_q + i;
  int2 s = make_int2(0, r.len);
  if (p.causal) s.y = (int)min((int64_t)r.len, max((int64_t)0, pos + 1));
  if (p.window > 0) s.x = (int)min((int64_t)s.y, max((int64_t)0, pos - p.window + 1));
  return s;
}

}  // namespace kv

// Both kernels' workspace begins with this many counters, zero between calls;
// nothing else is ever kept there.
constexpr int kCounters = 1024;

// Up to this many rows (queries x heads of a group) a request always go to the
// kernel for few rows.
constexpr int64_t kFewRows = 32;

// Few rows a request (fh_kv_decode.cu), and tiles of many on the tcgen05 tensor
// cores (fh_kv_prefill.cu).  The costs are estimates in microseconds, by which a
// call's kernel is chosen; max_kv: cached tokens that a query may see, at most.
size_t kv_attn_split_workspace(const KvAttnShape& s);
double kv_attn_split_cost(const KvAttnShape& s, int64_t max_kv);
cudaError_t launch_kv_attn_split(const kv::AttnParams& p, const KvAttnShape& shape, void* workspace, cudaStream_t s);

size_t kv_attn_tiles_workspace(const KvAttnShape& s);
double kv_attn_tiles_cost(const KvAttnShape& s, int64_t max_kv);
cudaError_t launch_kv_attn_tiles(const kv::AttnParams& p, const KvAttnShape& shape, int64_t max_kv, void* workspace,
                                 cudaStream_t s);

}  // namespace fh
