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
// move whole sectors: a block's BF16 in one 256-bit access where rows are
// 32-byte aligned, else in two of 128.  A thread has several blocks in flight,
// their rows read beside the slots, not behind them.  Keys and values go
// in one launch (blockIdx.y), each with its own decision table.
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
// Blocks of a thread in flight.  32768 tokens x 21 heads x 128: write 87 us
// with four in 64 registers (four CTAs an SM; 100 bytes a thread are spilled),
// 100 in 80 registers, 91 with two; read 73 with two, 79 with four.
constexpr int kWriteBlocks = 4, kReadBlocks = 2;

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
  uint32_t step_tokens, step_blocks;  // kKvThreads blocks on, as whole rows and a rest
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
  const int64_t page = slot >> p.page_shift;
  const uint32_t at = (uint32_t)slot & ((1u << p.page_shift) - 1);
  return ((page * p.kv_heads + head) << (p.page_shift + p.head_shift)) + ((at << p.head_shift) + in_head);
}

// A block's 32 bytes.  kWide: one access of 256 bits (32-byte aligned).
template <bool kWide>
__device__ __forceinline__ void load_block(const uint16_t* x, uint32_t (&w)[8]) {
  if constexpr (kWide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(x));
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(x)[0], b = reinterpret_cast<const uint4*>(x)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

template <bool kWide>
__device__ __forceinline__ void store_block(uint16_t* y, const uint32_t (&w)[8]) {
  if constexpr (kWide) {
    asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(y)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(y)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(y)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// A thread's blocks within a CTA's group of tokens: block i0 = its index, then
// every kKvThreads-th, as (token, block of the row) without a division each.
struct BlockWalk {
  uint32_t t, j;
  __device__ __forceinline__ BlockWalk(const KvParams& p) {
    t = threadIdx.x / p.row_blocks;
    j = threadIdx.x - t * p.row_blocks;
  }
  __device__ __forceinline__ void next(const KvParams& p) {
    t += p.step_tokens;
    j += p.step_blocks;
    if (j >= p.row_blocks) {
      j -= p.row_blocks;
      ++t;
    }
  }
};

template <bool kWide>
__global__ void __launch_bounds__(kKvThreads, 4) kv_write_kernel(const __grid_constant__ KvWriteParams wp) {
  __shared__ QuantTable tab;
  const KvParams& p = wp.k;
  const KvSide& s = p.side[blockIdx.y];
  {
    const uint4* src = reinterpret_cast<const uint4*>(&wp.tab[blockIdx.y]);
    uint4* dst = reinterpret_cast<uint4*>(&tab);
    for (int i = threadIdx.x; i < (int)(sizeof(QuantTable) / 16); i += kKvThreads) dst[i] = src[i];
  }
  __syncthreads();
  kv::wait_for_preceding();
  uint32_t clips = 0;
  for (int64_t g = blockIdx.x; g < p.groups; g += gridDim.x) {
    const int64_t t0 = g * p.group;
    const uint32_t n = (uint32_t)min((int64_t)p.group, p.tokens - t0);  // tokens
    BlockWalk at(p);
    while (at.t < n) {
      uint32_t w[kWriteBlocks][8], j[kWriteBlocks];
      int64_t slot[kWriteBlocks];
#pragma unroll
      for (int u = 0; u < kWriteBlocks; ++u) {
        slot[u] = -1;
        j[u] = at.j;
        if (at.t < n) {
          slot[u] = p.slots[t0 + at.t];
          load_block<kWide>(s.x + (t0 + at.t) * s.ld + 16 * at.j, w[u]);
        }
        at.next(p);
      }
#pragma unroll
      for (int u = 0; u < kWriteBlocks; ++u) {
        if (slot[u] < 0 || slot[u] >= p.n_slots) continue;
        uint32_t amax;
        uint2 codes;
        const uint32_t c = quantize_block_codes(tab, s.inv6sg, w[u], amax, codes);
        const int64_t b = cache_block(p, slot[u], j[u]);
        *reinterpret_cast<uint2*>(s.codes + 8 * b) = codes;
        s.scales[b] = (uint8_t)c;
        clips += block_clips(w[u], amax, s.clip_thr);
      }
    }
  }
  if (p.clip != nullptr) {
    clips = __reduce_add_sync(0xFFFFFFFFu, clips);
    if ((threadIdx.x & 31) == 0 && clips != 0) atomicAdd(p.clip, (unsigned long long)clips);
  }
}

template <bool kWide>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const __grid_constant__ KvParams p) {
  const KvSide& s = p.side[blockIdx.y];
  const float2 gs = make_float2(s.gscale, s.gscale);
  kv::wait_for_preceding();
  for (int64_t g = blockIdx.x; g < p.groups; g += gridDim.x) {
    const int64_t t0 = g * p.group;
    const uint32_t n = (uint32_t)min((int64_t)p.group, p.tokens - t0);  // tokens
    BlockWalk at(p);
    while (at.t < n) {
      int64_t slot[kReadBlocks];
      uint32_t t[kReadBlocks], j[kReadBlocks], scale[kReadBlocks];
      uint2 codes[kReadBlocks];
#pragma unroll
      for (int u = 0; u < kReadBlocks; ++u) {
        slot[u] = at.t < n ? p.slots[t0 + at.t] : -1;
        t[u] = at.t;
        j[u] = at.j;
        at.next(p);
      }
#pragma unroll
      for (int u = 0; u < kReadBlocks; ++u) {
        if (slot[u] < 0 || slot[u] >= p.n_slots) continue;
        const int64_t b = cache_block(p, slot[u], j[u]);
        codes[u] = *reinterpret_cast<const uint2*>(s.codes + 8 * b);
        scale[u] = s.scales[b];
      }
#pragma unroll
      for (int u = 0; u < kReadBlocks; ++u) {
        if (slot[u] < 0 || slot[u] >= p.n_slots) continue;
        const uint32_t h = kv::e4m3x2_to_f16x2(scale[u]);
        const uint32_t sc = __byte_perm(h, h, 0x1010);
        auto word = [&](uint32_t pair) {  // code * scale is exact in FP16
          const float2 v = __fmul2_rn(kv::f16x2_to_float2(kv::hmul2(pair, sc)), gs);
          return kv::pack_bf16x2(v.x, v.y);
        };
        uint32_t w[8];
        w[0] = word(kv::e2m1x2_to_f16x2<0>(codes[u].x));
        w[1] = word(kv::e2m1x2_to_f16x2<1>(codes[u].x));
        w[2] = word(kv::e2m1x2_to_f16x2<2>(codes[u].x));
        w[3] = word(kv::e2m1x2_to_f16x2<3>(codes[u].x));
        w[4] = word(kv::e2m1x2_to_f16x2<0>(codes[u].y));
        w[5] = word(kv::e2m1x2_to_f16x2<1>(codes[u].y));
        w[6] = word(kv::e2m1x2_to_f16x2<2>(codes[u].y));
        w[7] = word(kv::e2m1x2_to_f16x2<3>(codes[u].y));
        store_block<kWide>(s.y + (t0 + t[u]) * s.ld + 16 * j[u], w);
      }
    }
  }
}

int log2_of(int64_t v) {
  int s = 0;
  while (((int64_t)1 << s) < v) ++s;
  return s;
}

void fill_params(KvParams* p, const fh_kv_cache& c, const int64_t* slots, int64_t tokens, int per_thread) {
  p->slots = slots;
  p->tokens = tokens;
  p->n_slots = c.num_pages * c.page_size;
  p->row_blocks = (uint32_t)(c.kv_heads * c.head_dim / 16);
  p->step_tokens = kKvThreads / p->row_blocks;
  p->step_blocks = kKvThreads % p->row_blocks;
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
  // A group is what a CTA takes at a time: per_thread blocks a thread or a few
  // less, and at least one token; fewer a thread where SMs would be idle (64 tokens
  // x 8 heads x 128 in a graph: write 2.5 us with one, 5.8 with four).
  while (per_thread > 1 && tokens * p->row_blocks < (int64_t)kKvThreads * per_thread * sm_count()) per_thread >>= 1;
  const int64_t blocks = (int64_t)kKvThreads * per_thread;
  p->group = (int)(blocks / p->row_blocks > 0 ? blocks / p->row_blocks : 1);
  p->groups = (tokens + p->group - 1) / p->group;
}

dim3 kv_grid(const KvParams& p, int per_sm) {
  const int64_t cap = (int64_t)sm_count() * per_sm;
  return dim3((unsigned)(p.groups < cap ? p.groups : cap), 2);
}

// Whether every block of 16 elements of these rows is 32-byte aligned.
bool wide_rows(const uint16_t* x, int64_t ld) { return (reinterpret_cast<uintptr_t>(x) & 31) == 0 && ld % 16 == 0; }

}  // namespace

cudaError_t launch_kv_write(const fh_kv_cache& c, const uint16_t* k, const uint16_t* v, int64_t tokens, int64_t ldk,
                            int64_t ldv, const int64_t* slots, unsigned long long* clip, cudaStream_t s) {
  KvWriteParams p;
  memcpy(&p.tab[0], &quant_table_for(c.k_gscale), sizeof(QuantTable));
  memcpy(&p.tab[1], &quant_table_for(c.v_gscale), sizeof(QuantTable));
  fill_params(&p.k, c, slots, tokens, kWriteBlocks);
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
  const bool wide = wide_rows(k, ldk) && wide_rows(v, ldv);
  return launch_overlapping(wide ? kv_write_kernel<true> : kv_write_kernel<false>, kv_grid(p.k, 2), dim3(kKvThreads), 0, s, p);
}

cudaError_t launch_kv_read(const fh_kv_cache& c, const int64_t* slots, int64_t tokens, uint16_t* k, uint16_t* v,
                           int64_t ldk, int64_t ldv, cudaStream_t s) {
  KvParams p;
  fill_params(&p, c, slots, tokens, kReadBlocks);
  uint16_t* y[2] = {k, v};
  const int64_t ld[2] = {ldk, ldv};
  for (int i = 0; i < 2; ++i) {
    p.side[i].x = nullptr;
    p.side[i].y = y[i];
    p.side[i].ld = ld[i];
    p.side[i].inv6sg = 0.0f;
    p.side[i].clip_thr = 0;
  }
  const bool wide = wide_rows(k, ldk) && wide_rows(v, ldv);
  return launch_overlapping(wide ? kv_read_kernel<true> : kv_read_kernel<false>, kv_grid(p, 16), dim3(kKvThreads), 0, s, p);
}

}  // namespace fh
