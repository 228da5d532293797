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
// The tables are one cluster's work (one CTA for small calls, eight for large
// ones), whose hardware barrier separates reading the lengths and the stack's
// count from overwriting them: the outputs may be the inputs' own buffers, and
// no workspace or counter is needed.  Every CTA forms the prefix sums of all
// requests for itself in shared memory (that is cheaper than exchanging them).
// Few slots are written by the same launch.  Many go to a second one over the
// whole GPU, which needs only the first one's outputs: a growing request held
// lens - (q_starts[b + 1] - q_starts[b]) tokens.  A warp takes 128 consecutive
// slots, finds the requests of the first and the last by binary search, and its
// lanes search only between those.  Bound by latency: a call moves a few bytes
// a request and eight a slot.  (All in one cluster of eight, 300,000 slots
// took 45 us.)
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fh_internal.h"
#include "fh_kv.cuh"

namespace fh {

namespace {

constexpr int kPagesCtas = 8;      // of a large call's cluster
constexpr int kPagesThreads = 1024;
constexpr int kFewSlots = 8192;    // written by the first launch
constexpr int kRun = 128;          // slots a warp takes at a time

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

// The slots of this thread's share of [0, capacity): page_of(b, at) names the
// page of request b's table entry `at`, start(b) where its new tokens begin.
template <class Held, class PageOf>
__device__ __forceinline__ void write_slots(const PagesParams& p, const int32_t* starts, int n_rows, int64_t warp,
                                            int64_t warps, Held held, PageOf page_of) {
  const int lane = threadIdx.x & 31, n = p.batch;
  for (int64_t r0 = warp * kRun; r0 < p.slot_capacity; r0 += warps * kRun) {
    int first = 0, last = 0;
    if (r0 < n_rows) {
      const int x = lane == 0 ? (int)r0 : (int)min(r0 + kRun - 1, (int64_t)n_rows - 1);
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
        const int token = held(b) + ((int)r - starts[b]);
        const int page = page_of(b, token >> p.shift);
        if (page >= 0) slot = ((int64_t)page << p.shift) + (token & ((1 << p.shift) - 1));
      }
      p.slots[r] = slot;
    }
  }
}

__global__ void __launch_bounds__(kPagesThreads, 1) kv_pages_kernel(const PagesParams p, bool with_slots) {
  extern __shared__ int32_t pages_smem[];
  const int n = p.batch;
  int32_t* held_s = pages_smem;          // [n]
  int32_t* target_s = held_s + n;        // [n]
  int32_t* taken = target_s + n;         // [n + 1] prefix sums, exclusive; [n] the total
  int32_t* given = taken + n + 1;        // [n + 1]
  int32_t* starts = given + n + 1;       // [n + 1]
  __shared__ long long warp_sums[3][kPagesThreads / 32 + 1];  // then their exclusive prefix, and the total
  __shared__ int bad_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto cluster = cooperative_groups::this_cluster();
  kv::wait_for_preceding();
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
  if (warp < 3) {  // a warp a sum
    const long long own = warp_sums[warp][lane];
    long long v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    warp_sums[warp][lane] = v - own;
    if (lane == 31) warp_sums[warp][32] = v;
  }
  __syncthreads();
  long long total[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    pre[k] += warp_sums[k][warp];
    total[k] = warp_sums[k][32];
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
  const int all = (int)cluster.num_blocks() * kPagesThreads;
  const bool ok = status == 0;
  for (int b = gt; b <= n; b += all) {
    if (b < n) p.lens[b] = ok ? target_s[b] : held_s[b];
    p.q_starts[b] = ok ? starts[b] : 0;
  }
  if (gt == 0) {
    *p.free_count_out = ok ? (int)(count + total[1] - total[0]) : count;
    *p.status = status;
  }
  if (!ok) {
    if (with_slots)
      for (int64_t r = gt; r < p.slot_capacity; r += all) p.slots[r] = -1;
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
  // (64-bit: the totals may be 2^31 - 1, and the last step goes past them.)
  for (int64_t i = gt; i < n_taken; i += all) {
    const int b = owner_of(taken, 0, n, (int)i);
    p.table[(int64_t)b * p.max_pages + pages_of(held_s[b]) + ((int)i - taken[b])] = taken_page((int)i);
  }
  for (int64_t f = gt; f < n_given; f += all) p.free_pages[count + f] = given_page((int)f);

  if (with_slots)
    write_slots(p, starts, n_rows, gt >> 5, all / 32, [&](int b) { return held_s[b]; },
                [&](int b, int at) {
                  const int have = pages_of(held_s[b]);
                  return at < have ? p.table[(int64_t)b * p.max_pages + at] : taken_page(taken[b] + at - have);
                });
}

constexpr int kSlotThreads = 512;

// The slots alone, from what kv_pages_kernel has written.
__global__ void __launch_bounds__(kSlotThreads) kv_slots_kernel(const PagesParams p) {
  extern __shared__ int32_t pages_smem[];  // [batch + 1]
  kv::wait_for_preceding();
  for (int b = threadIdx.x; b <= p.batch; b += kSlotThreads) pages_smem[b] = p.q_starts[b];
  __syncthreads();
  const int32_t* starts = pages_smem;
  write_slots(p, starts, starts[p.batch], ((int64_t)blockIdx.x * kSlotThreads + threadIdx.x) >> 5,
              (int64_t)gridDim.x * (kSlotThreads / 32), [&](int b) { return p.lens[b] - (starts[b + 1] - starts[b]); },
              [&](int b, int at) { return p.table[(int64_t)b * p.max_pages + at]; });
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
  const bool few = slot_capacity <= kFewSlots;
  // Table entries to write: at most one a request and one a page of new tokens.
  const bool large = batch + slot_capacity / page_size > 1024;
  cudaLaunchConfig_t cfg_a = {};
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = large ? kPagesCtas : 1;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg_a.gridDim = dim3(large ? kPagesCtas : 1);
  cfg_a.blockDim = dim3(kPagesThreads);
  cfg_a.dynamicSmemBytes = smem;
  cfg_a.stream = s;
  cfg_a.attrs = attr;
  cfg_a.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg_a, kv_pages_kernel, p, few);
  if (e != cudaSuccess || few) return e;
  const int64_t runs = (slot_capacity + kRun - 1) / kRun, per_cta = kSlotThreads / 32;
  const int64_t want = (runs + per_cta - 1) / per_cta, cap = (int64_t)sm_count() * 4;
  return launch_overlapping(kv_slots_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(kSlotThreads),
                            (size_t)(batch + 1) * 4, s, p);
}

}  // namespace fh
