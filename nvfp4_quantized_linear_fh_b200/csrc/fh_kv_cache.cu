// fh_kv_cache.cu -- writing keys and values into the paged NVFP4 cache, and
// reading them back as BF16.
//
// Write: per 16 elements of a head S = E4M3(amax / (6 s_g)) and code =
// E2M1(x / (S s_g)), to nearest with ties to the even code on the exact
// quotients: the block quantization that fh_quantize_act makes of a row's
// blocks (fh_nvfp4.cuh), so a cached token's codes are those of its rows.  Read:
// bf16(fp32(code * S) * s_g), where code * S (2 + 4 significant bits) is exact.
//
// Both are HBM-bound: a token's element costs 2 bytes on one side and 0.5625
// on the other.  A thread has one 16-element block (32 bytes of BF16, 8 of
// codes, one scale); the blocks of a token follow one another in the rows of
// x, and the 64 code bytes of one head (d = 128) in the page, so both sides
// move whole sectors.  Four blocks per thread are in flight at once.  Keys and
// values go in one launch (blockIdx.y), each with its own decision table.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "fh_internal.h"
#include "fh_kv.cuh"
#include "fh_nvfp4.cuh"

namespace fh {

namespace {

using namespace nvfp4;

constexpr int kKvThreads = 256;
constexpr int kKvBlocksPerThread = 4;

// One of keys and values.
struct KvSide {
  const uint16_t* x;  // write: input rows
  uint16_t* y;        // read: output rows
  int64_t ld;         // elements between tokens of x or y
  uint8_t* codes;
  uint8_t* scales;
  float gscale, inv6sg;
  uint32_t clip_thr;
};

struct KvParams {
  KvSide side[2];
  const int64_t* slots;
  int64_t tokens, n_slots;  // n_slots: num_pages * page_size
  int64_t groups;           // of `group` tokens each
  int group;
  uint32_t row_blocks;      // kv_heads * d / 16
  int head_shift;           // log2(d / 16)
  int page_shift, kv_heads;
  unsigned long long* clip;
};

struct KvWriteParams {
  QuantTable tab[2];
  KvParams k;
};

// Where the block `j` of a token's row lies: its index among the cache's blocks.
__device__ __forceinline__ int64_t cache_block(const KvParams& p, int64_t slot, uint32_t j) {
  const uint32_t head = j >> p.head_shift, in_head = j & ((1u << p.head_shift) - 1);
  const int64_t page = slot >> p.page_shift, at = slot & (((int64_t)1 << p.page_shift) - 1);
  return (((page * p.kv_heads + head) << p.page_shift) + at) * ((int64_t)1 << p.head_shift) + in_head;
}

__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const __grid_constant__ KvWriteParams wp) {
  __shared__ QuantTable tab;
  const KvParams& p = wp.k;
  const KvSide& s = p.side[blockIdx.y];
  {
    const uint4* src = reinterpret_cast<const uint4*>(&wp.tab[blockIdx.y]);
    uint4* dst = reinterpret_cast<uint4*>(&tab);
    for (int i = threadIdx.x; i < (int)(sizeof(QuantTable) / 16); i += kKvThreads) dst[i] = src[i];
  }
  __syncthreads();
  uint32_t clips = 0;
  for (int64_t g = blockIdx.x; g < p.groups; g += gridDim.x) {
    const int64_t t0 = g * p.group;
    const uint32_t n = (uint32_t)min((int64_t)p.group, p.tokens - t0) * p.row_blocks;
    for (uint32_t i0 = threadIdx.x; i0 < n; i0 += kKvThreads * kKvBlocksPerThread) {
      uint4 q[kKvBlocksPerThread][2];
      int64_t at[kKvBlocksPerThread];
#pragma unroll
      for (int u = 0; u < kKvBlocksPerThread; ++u) {
        const uint32_t i = i0 + u * kKvThreads;
        at[u] = -1;
        if (i < n) {
          const uint32_t t = i / p.row_blocks, j = i - t * p.row_blocks;
          const int64_t slot = p.slots[t0 + t];
          if (slot >= 0 && slot < p.n_slots) {
            at[u] = cache_block(p, slot, j);
            const uint4* src = reinterpret_cast<const uint4*>(s.x + (t0 + t) * s.ld + 16 * (int64_t)j);
            q[u][0] = __ldcs(src);
            q[u][1] = __ldcs(src + 1);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kKvBlocksPerThread; ++u) {
        if (at[u] < 0) continue;
        const uint32_t w[8] = {q[u][0].x, q[u][0].y, q[u][0].z, q[u][0].w, q[u][1].x, q[u][1].y, q[u][1].z, q[u][1].w};
        uint32_t amax;
        uint2 codes;
        const uint32_t c = quantize_block_codes(tab, s.inv6sg, w, amax, codes);
        *reinterpret_cast<uint2*>(s.codes + 8 * at[u]) = codes;
        s.scales[at[u]] = (uint8_t)c;
        clips += block_clips(w, amax, s.clip_thr);
      }
    }
  }
  if (p.clip != nullptr) {
    clips = __reduce_add_sync(0xFFFFFFFFu, clips);
    if ((threadIdx.x & 31) == 0 && clips != 0) atomicAdd(p.clip, (unsigned long long)clips);
  }
}

__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const __grid_constant__ KvParams p) {
  const KvSide& s = p.side[blockIdx.y];
  for (int64_t g = blockIdx.x; g < p.groups; g += gridDim.x) {
    const int64_t t0 = g * p.group;
    const uint32_t n = (uint32_t)min((int64_t)p.group, p.tokens - t0) * p.row_blocks;
    for (uint32_t i0 = threadIdx.x; i0 < n; i0 += kKvThreads * kKvBlocksPerThread) {
      uint2 codes[kKvBlocksPerThread];
      uint32_t scale[kKvBlocksPerThread];
      uint16_t* out[kKvBlocksPerThread];
#pragma unroll
      for (int u = 0; u < kKvBlocksPerThread; ++u) {
        const uint32_t i = i0 + u * kKvThreads;
        out[u] = nullptr;
        if (i < n) {
          const uint32_t t = i / p.row_blocks, j = i - t * p.row_blocks;
          const int64_t slot = p.slots[t0 + t];
          if (slot >= 0 && slot < p.n_slots) {
            const int64_t at = cache_block(p, slot, j);
            codes[u] = *reinterpret_cast<const uint2*>(s.codes + 8 * at);
            scale[u] = s.scales[at];
            out[u] = s.y + (t0 + t) * s.ld + 16 * (int64_t)j;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kKvBlocksPerThread; ++u) {
        if (out[u] == nullptr) continue;
        const float sc = kv::f16x2_to_float2(kv::e4m3x2_to_f16x2(scale[u])).x;
        uint32_t w[8];
        auto word = [&](uint32_t f16x2) {
          const float2 v = kv::f16x2_to_float2(f16x2);
          return kv::pack_bf16x2((v.x * sc) * s.gscale, (v.y * sc) * s.gscale);
        };
        w[0] = word(kv::e2m1x2_to_f16x2<0>(codes[u].x));
        w[1] = word(kv::e2m1x2_to_f16x2<1>(codes[u].x));
        w[2] = word(kv::e2m1x2_to_f16x2<2>(codes[u].x));
        w[3] = word(kv::e2m1x2_to_f16x2<3>(codes[u].x));
        w[4] = word(kv::e2m1x2_to_f16x2<0>(codes[u].y));
        w[5] = word(kv::e2m1x2_to_f16x2<1>(codes[u].y));
        w[6] = word(kv::e2m1x2_to_f16x2<2>(codes[u].y));
        w[7] = word(kv::e2m1x2_to_f16x2<3>(codes[u].y));
        reinterpret_cast<uint4*>(out[u])[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(out[u])[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
}

int log2_of(int64_t v) {
  int s = 0;
  while (((int64_t)1 << s) < v) ++s;
  return s;
}

void fill_params(KvParams* p, const fh_kv_cache& c, const int64_t* slots, int64_t tokens) {
  p->slots = slots;
  p->tokens = tokens;
  p->n_slots = c.num_pages * c.page_size;
  p->row_blocks = (uint32_t)(c.kv_heads * c.head_dim / 16);
  p->head_shift = log2_of(c.head_dim / 16);
  p->page_shift = log2_of(c.page_size);
  p->kv_heads = (int)c.kv_heads;
  p->clip = nullptr;
  uint8_t* codes[2] = {c.k_codes, c.v_codes};
  uint8_t* scales[2] = {c.k_scales, c.v_scales};
  const float gs[2] = {c.k_gscale, c.v_gscale};
  for (int i = 0; i < 2; ++i) {
    p->side[i].codes = codes[i];
    p->side[i].scales = scales[i];
    p->side[i].gscale = gs[i];
  }
  // A group is what a CTA takes at a time: about a thousand blocks, so that
  // each thread has four, and at least one token.
  const int64_t blocks = (int64_t)kKvThreads * kKvBlocksPerThread;
  p->group = (int)(blocks / p->row_blocks > 0 ? blocks / p->row_blocks : 1);
  p->groups = (tokens + p->group - 1) / p->group;
}

dim3 kv_grid(const KvParams& p) {
  const int64_t cap = (int64_t)sm_count() * 4;
  return dim3((unsigned)(p.groups < cap ? p.groups : cap), 2);
}

}  // namespace

cudaError_t launch_kv_write(const fh_kv_cache& c, const uint16_t* k, const uint16_t* v, int64_t tokens, int64_t ldk,
                            int64_t ldv, const int64_t* slots, unsigned long long* clip, cudaStream_t s) {
  KvWriteParams p;
  memcpy(&p.tab[0], &quant_table_for(c.k_gscale), sizeof(QuantTable));
  memcpy(&p.tab[1], &quant_table_for(c.v_gscale), sizeof(QuantTable));
  fill_params(&p.k, c, slots, tokens);
  p.k.clip = clip;
  const uint16_t* x[2] = {k, v};
  const int64_t ld[2] = {ldk, ldv};
  for (int i = 0; i < 2; ++i) {
    KvSide& e = p.k.side[i];
    e.x = x[i];
    e.y = nullptr;
    e.ld = ld[i];
    e.inv6sg = (float)(1.0 / (6.0 * (double)e.gscale));
    e.clip_thr = clip_threshold_bits(e.gscale);
  }
  kv_write_kernel<<<kv_grid(p.k), kKvThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv_read(const fh_kv_cache& c, const int64_t* slots, int64_t tokens, uint16_t* k, uint16_t* v,
                           int64_t ldk, int64_t ldv, cudaStream_t s) {
  KvParams p;
  fill_params(&p, c, slots, tokens);
  uint16_t* y[2] = {k, v};
  const int64_t ld[2] = {ldk, ldv};
  for (int i = 0; i < 2; ++i) {
    p.side[i].x = nullptr;
    p.side[i].y = y[i];
    p.side[i].ld = ld[i];
    p.side[i].inv6sg = 0.0f;
    p.side[i].clip_thr = 0;
  }
  kv_read_kernel<<<kv_grid(p), kKvThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fh
