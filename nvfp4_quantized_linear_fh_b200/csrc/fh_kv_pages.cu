// fh_kv_pages.cu -- bookkeeping of the paged key/value cache: block tables, the
// stack of free pages and the slots of new tokens, from request lengths.
//
// With P = page_size, request b holds ceil(held / P) pages and is to hold
// ceil(target / P).  Requests that need fewer give back the entries behind;
// those pages go onto the free stack in the order of the requests and of their
// tables.  Then requests that need more take pages from the stack's top in the
// same order.  Three exclusive prefix sums over the requests (pages given back,
// pages taken, new tokens) place every entry and every slot independently of
// the others, so each output is written once, by whichever thread has it.
//
// One cluster of eight CTAs, whose hardware barrier separates reading the
// lengths and the stack's count from overwriting them: the outputs may be the
// inputs' own buffers, and no workspace, counter or second launch is needed.
// Every CTA forms the prefix sums of all requests for itself in shared memory
// (that is cheaper than exchanging them); a warp then takes 128 consecutive
// slots, finds the requests of the first and the last by binary search, and its
// lanes search only between those.  The call is latency-bound: it moves a few
// bytes a request and eight a slot.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fh_internal.h"

namespace fh {

namespace {

constexpr int kPagesCtas = 8;
constexpr int kPagesThreads = 1024;

struct PagesParams {
  const int32_t* held;
  const int32_t* target;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* lens;
  int32_t* q_starts;
  int64_t* slots;
  int32_t* status;
  int64_t max_pages, free_capacity, slot_capacity;
  int batch, shift;
};

// First index in [lo, hi) whose successor prefix a[index + 1] is above x; hi - 1 if none is.
__device__ __forceinline__ int owner_of(const int32_t* a, int lo, int hi, int x) {
  while (lo + 1 < hi) {
    const int mid = (lo + hi) >> 1;  // invariant: the answer is in [lo, hi)
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __cluster_dims__(kPagesCtas, 1, 1) __launch_bounds__(kPagesThreads, 1)
    kv_pages_kernel(const PagesParams p) {
  extern __shared__ int32_t pages_smem[];
  const int n = p.batch;
  int32_t* held_s = pages_smem;          // [n]
  int32_t* target_s = held_s + n;        // [n]
  int32_t* taken = target_s + n;         // [n + 1] prefix sums, exclusive; [n] the total
  int32_t* given = taken + n + 1;        // [n + 1]
  int32_t* starts = given + n + 1;       // [n + 1]
  __shared__ long long warp_sums[3][kPagesThreads / 32];
  __shared__ int bad_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto cluster = cooperative_groups::this_cluster();
  const int count = *p.free_count;
  if (tid == 0) bad_s = 0;
  __syncthreads();

  // A thread takes `per` neighbouring requests.
  const int per = (n + kPagesThreads - 1) / kPagesThreads;
  const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
  const int mask = (1 << p.shift) - 1;
  auto pages_of = [&](int len) { return (int)(((int64_t)len + mask) >> p.shift); };
  long long sum[3] = {0, 0, 0};
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int h = p.held[b], t = p.target[b];
    if (h < 0 || t < 0)
      bad |= FH_KV_BAD_LENGTH;
    else if (max(pages_of(h), pages_of(t)) > p.max_pages)
      bad |= FH_KV_TABLE_FULL;
    held_s[b] = h;
    target_s[b] = t;
    if (h >= 0 && t >= 0) {
      sum[0] += max(0, pages_of(t) - pages_of(h));
      sum[1] += max(0, pages_of(h) - pages_of(t));
      sum[2] += max(0, t - h);
    }
  }
  if (bad) atomicOr(&bad_s, bad);
  // Block-wide exclusive prefix of the threads' sums.
  long long pre[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long v = sum[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    pre[k] = v - sum[k];
    if (lane == 31) warp_sums[k][warp] = v;
  }
  __syncthreads();
  long long total[3] = {0, 0, 0};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    for (int w = 0; w < kPagesThreads / 32; ++w) {
      if (w < warp) pre[k] += warp_sums[k][w];
      total[k] += warp_sums[k][w];
    }
  }
  int status = bad_s;
  if (count < 0 || count + total[1] > p.free_capacity) status |= FH_KV_STACK_OVERFLOW;
  if (total[0] > count + total[1]) status |= FH_KV_NO_PAGES;
  if (total[2] > p.slot_capacity) status |= FH_KV_SLOTS_FULL;
  if (status == 0) {  // the totals fit 32 bits
    for (int b = b0; b < b1; ++b) {
      const int h = held_s[b], t = target_s[b];
      taken[b] = (int)pre[0];
      given[b] = (int)pre[1];
      starts[b] = (int)pre[2];
      pre[0] += max(0, pages_of(t) - pages_of(h));
      pre[1] += max(0, pages_of(h) - pages_of(t));
      pre[2] += max(0, t - h);
    }
    if (tid == 0) {
      taken[n] = (int)total[0];
      given[n] = (int)total[1];
      starts[n] = (int)total[2];
    }
  }
  __syncthreads();
  cluster.sync();  // every CTA has read the lengths and the count: they may be overwritten

  const int gt = (int)cluster.block_rank() * kPagesThreads + tid;
  constexpr int kAll = kPagesCtas * kPagesThreads;
  const bool ok = status == 0;
  for (int b = gt; b <= n; b += kAll) {
    if (b < n) p.lens[b] = ok ? target_s[b] : held_s[b];
    p.q_starts[b] = ok ? starts[b] : 0;
  }
  if (gt == 0) {
    *p.free_count_out = ok ? (int)(count + total[1] - total[0]) : count;
    *p.status = status;
  }
  if (!ok) {
    for (int64_t r = gt; r < p.slot_capacity; r += kAll) p.slots[r] = -1;
    return;
  }
  // The f-th page given back, from the entries behind its request's new end.
  auto given_page = [&](int f) {
    const int b = owner_of(given, 0, n, f);
    return p.table[(int64_t)b * p.max_pages + pages_of(target_s[b]) + (f - given[b])];
  };
  // The i-th page taken: from the stack as it stands once the pages given back are on it.
  const int n_taken = (int)total[0], n_given = (int)total[1], n_rows = (int)total[2];
  auto taken_page = [&](int i) {
    const int at = count + n_given - 1 - i;
    return at >= count ? given_page(at - count) : p.free_pages[at];
  };
  for (int i = gt; i < n_taken; i += kAll) {
    const int b = owner_of(taken, 0, n, i);
    p.table[(int64_t)b * p.max_pages + pages_of(held_s[b]) + (i - taken[b])] = taken_page(i);
  }
  for (int f = gt; f < n_given; f += kAll) p.free_pages[(int64_t)count + f] = given_page(f);

  constexpr int kRun = 128;  // slots a warp takes at a time
  for (int64_t r0 = (int64_t)(gt >> 5) * kRun; r0 < p.slot_capacity; r0 += (int64_t)(kAll / 32) * kRun) {
    int first = 0, last = 0;
    if (r0 < n_rows) {
      const int x = lane == 0 ? (int)r0 : min((int)r0 + kRun - 1, n_rows - 1);
      const int b = owner_of(starts, 0, n, x);
      first = __shfl_sync(0xFFFFFFFFu, b, 0);
      last = __shfl_sync(0xFFFFFFFFu, b, 1);
    }
#pragma unroll
    for (int k = 0; k < kRun / 32; ++k) {
      const int64_t r = r0 + k * 32 + lane;
      if (r >= p.slot_capacity) break;
      int64_t slot = -1;
      if (r < n_rows) {
        const int b = owner_of(starts, first, last + 1, (int)r);
        const int token = held_s[b] + ((int)r - starts[b]);
        const int at = token >> p.shift, have = pages_of(held_s[b]);
        const int page = at < have ? p.table[(int64_t)b * p.max_pages + at] : taken_page(taken[b] + at - have);
        if (page >= 0) slot = ((int64_t)page << p.shift) + (token & mask);
      }
      p.slots[r] = slot;
    }
  }
}

}  // namespace

cudaError_t launch_kv_pages(const int32_t* held, const int32_t* target, int64_t batch, int64_t page_size,
                            int32_t* table, int64_t max_pages, int32_t* free_pages, int64_t free_capacity,
                            const int32_t* free_count, int32_t* free_count_out, int32_t* lens, int32_t* q_starts,
                            int64_t* slots, int64_t slot_capacity, int32_t* status, cudaStream_t s) {
  PagesParams p;
  p.held = held;
  p.target = target;
  p.table = table;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.free_count_out = free_count_out;
  p.lens = lens;
  p.q_starts = q_starts;
  p.slots = slots;
  p.status = status;
  p.max_pages = max_pages;
  p.free_capacity = free_capacity;
  p.slot_capacity = slot_capacity;
  p.batch = (int)batch;
  p.shift = 0;
  while (((int64_t)1 << p.shift) < page_size) ++p.shift;
  const int smem = (int)(5 * batch + 3) * 4;
  static DeviceTable configured;
  int dev = 0;
  cudaGetDevice(&dev);
  const int cfg = per_device(configured, dev, [](int) {
    const cudaError_t e = cudaFuncSetAttribute(kv_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (5 * FH_KV_MAX_BATCH + 3) * 4);
    return e == cudaSuccess ? 1 : -(int)e;
  });
  if (cfg <= 0) return (cudaError_t)(-cfg);
  kv_pages_kernel<<<kPagesCtas, kPagesThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace fh
