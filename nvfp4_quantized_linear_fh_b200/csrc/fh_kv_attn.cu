// fh_kv_attn.cu -- attention over the paged NVFP4 cache: which kernel takes a call.
#include <math.h>
#include <stdlib.h>

#include "fh_internal.h"
#include "fh_kv_attn.h"

namespace fh {

size_t kv_attention_workspace(const KvAttnShape& s) {
  const size_t a = kv_attn_split_workspace(s), b = kv_attn_tiles_workspace(s);
  return a > b ? a : b;
}

cudaError_t launch_kv_attention(const fh_kv_cache& c, const KvAttnCall& call, const KvAttnShape& shape,
                                void* workspace, cudaStream_t s) {
  kv::AttnParams p;
  p.q = call.q;
  p.out = call.out;
  p.lse = call.lse;
  p.k_codes = c.k_codes;
  p.k_scales = c.k_scales;
  p.v_codes = c.v_codes;
  p.v_scales = c.v_scales;
  p.table = call.table;
  p.lens = call.lens;
  p.q_starts = call.q_starts;
  p.ldq = call.ldq;
  p.ldo = call.ldo;
  p.max_pages = call.max_pages;
  p.total_q = (int)shape.total_q;
  p.batch = (int)shape.batch;
  p.q_heads = (int)shape.q_heads;
  p.kv_heads = (int)shape.kv_heads;
  kv::set_group(&p, (int)(shape.q_heads / shape.kv_heads));
  p.page_shift = 0;
  while (((int64_t)1 << p.page_shift) < c.page_size) ++p.page_shift;
  p.num_pages = (int)c.num_pages;
  p.causal = call.causal ? 1 : 0;
  p.window = call.window;
  const char* stall = getenv("FH_KV_TEST_STALL");  // read at each launch
  p.stall = stall != nullptr && stall[0] == '1' ? 1 : 0;
  p.qk_scale = (float)frexp((double)call.sm_scale * 1.4426950408889634 * (double)c.k_gscale, &p.qk_exp);
  int v_exp;
  p.v_scale = 2.0f * frexpf(c.v_gscale, &v_exp);
  p.v_unit = ldexpf(1.0f, v_exp - 1);
  p.part_o = nullptr;
  p.part_ml = nullptr;
  p.count = nullptr;
  // Which kernel: the one for few rows reads the cache once per eight rows and
  // spreads over the GPU however few they are; the one for tiles reads it once per
  // 256.  Measured with both, in us (few / tiles): 32 rows of 16 requests of up to
  // 4000 tokens, 8 KV heads, 52 / 72; 64 rows of them 67 / 72; 64 rows of 64
  // requests of up to 1000, 92 / 78; 48 rows of one of 30000, 21 KV heads,
  // 124 / 91; 64 rows of one of 30000, one KV head, 30 / 78.  The choice is the whole
  // call's, and max_q is all that it knows of the requests' rows: 63 single tokens and
  // a prompt's 512 over up to 8192 tokens, 32 heads over 8, take 602 / 317 as one call
  // (here the estimate is wrong) and 87 + 81 as two.
  int64_t max_kv = shape.max_kv;
  if (p.window > 0 && max_kv > (int64_t)p.window + shape.max_q) max_kv = (int64_t)p.window + shape.max_q;
  bool few = shape.max_q * p.group <= kFewRows || kv_attn_split_cost(shape, max_kv) < kv_attn_tiles_cost(shape, max_kv);
  const char* kernel = getenv("FH_KV_KERNEL");  // read at each launch
  if (kernel != nullptr && kernel[0] == 'f') few = true;
  if (kernel != nullptr && kernel[0] == 't') few = false;
  if (few)
    return launch_kv_attn_split(p, shape, workspace, s);
  return launch_kv_attn_tiles(p, shape, max_kv, workspace, s);
}

}  // namespace fh
