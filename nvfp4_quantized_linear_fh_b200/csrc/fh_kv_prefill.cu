// fh_kv_prefill.cu -- attention over the paged NVFP4 cache for many query rows a
// request (prompts, whole clips), on the tcgen05 tensor cores.
//
// The same attention as fh_kv_decode.cu; here the two products bound it, and
// beside them the exponentials.  At d = 128, 256 rows x 128 keys are 2048
// cycles of an SM's nominal FP16 tensor rate; as issued, 2868 (measured alone:
// a 128 x 128 x 16 MMA takes 105 cycles with A in shared memory, 74 with A in
// TMEM), and 2048 of its 16 exponentials a cycle.
//
// A CTA has 256 packed query rows (row = token * G + head in group) of one
// request and KV head, as two 128-row tiles, and walks 128-token key tiles:
//   warps 0..3, 4..7   one row a thread, a tile each: scores from TMEM, running
//                      maximum and sum, P back to TMEM over the scores' columns,
//                      where the second product takes it as its A operand.
//   warps 8..11        codes from shared memory, converted to code * scale in
//                      FP16 (exact) and laid out in 128-byte swizzled rows; the
//                      same layout serves K as a K-major operand and V as an
//                      MN-major one, so V is not transposed.
//   warp 12            issues the products: S = Q K^T of one tile while the other
//                      tile's softmax runs, O += P V.
//   warp 13            brings the pages' codes and scales to shared memory with
//                      cp.async.bulk, three half steps ahead.  (Loads by the
//                      converting threads would be waited for by the proxy fence
//                      that hands their stores to the tensor cores: 265 us at
//                      21 x 4096 x 4096 x 128, where softmax and products alone
//                      take 232.)
// The output stays in TMEM.  It is rescaled only when a row's maximum grows by
// more than 8 (in log2), by the row's own thread: the commit that announces
// S(j) also covers O += P(j-1) V, so nothing else is writing O then.
//
// Too few row tiles for the GPU, or too few in its last wave: their keys are cut
// into up to eight pieces, a CTA each, which leave their partial results in the
// workspace; the one that finishes last (an atomic count; nobody waits) joins
// them in the pieces' order.  (At 21 x 4096 x 4096 x 128, 336 tiles on 148 SMs,
// the last 40 as 120 thirds.)
//
// Queries, probabilities, sums and roundings are as in fh_kv_decode.cu.  Every
// mbarrier wait is bounded; on expiry the kernel sets its error word, drains
// what it issued, frees its TMEM and returns.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fh_internal.h"
#include "fh_kv.cuh"
#include "fh_kv_attn.h"
#include "fh_nvfp4.cuh"

namespace fh {

namespace {

using namespace kv;

__device__ unsigned int g_kv_error = 0;

constexpr int kRows = 128;     // query rows of a tile (threads of a softmax group)
constexpr int kTiles = 2;      // tiles of a CTA
constexpr int kKeys = 128;     // tokens of a key tile
constexpr int kStages = 2;     // of K and of V
constexpr int kSoftWarps = 4 * kTiles;
constexpr int kFeedWarps = 4;
constexpr int kMmaWarp = kSoftWarps + kFeedWarps, kCopyWarp = kMmaWarp + 1;
constexpr int kRaw = 3;        // ring of tiles' codes and scales, K and V in turns
constexpr int kThreads = 32 * (kMmaWarp + 4);  // whole warpgroups: two warps of the last one have no work
// Registers: launched with 128 a thread (512 threads, the whole file); the
// eight softmax warps take 176, the others keep 80: 256 * 176 + 256 * 80 = 65536.
constexpr int kSoftRegs = 176, kOtherRegs = 80;
constexpr int kLive = 4;       // ring of the key tiles' page masks
constexpr int kMaxPieces = 8;  // of a row tile's keys
// Requests that are put in order, each by a thread that looks at all others.  More
// take the batch's order, last to first; put in order as well (128 here), in us: 66 of
// 64 .. 4000 tokens, 8 heads over 2, 222, and 233 in the batch's order (219 .. 238 by
// that order); 100 of up to 2000, d = 64, 141 and 149 (137 .. 156); 128 of 200 .. 1500,
// 118.5 and 122 (114.5 .. 125).
constexpr int kSorted = 64;
constexpr int kMaxPieceCtas = 320;  // workspace bound: a partial result each
constexpr float kRaise = 8.0f;
constexpr float kHead = 6.0f;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;                 // 64-element (128-byte) column blocks of an operand
  static constexpr int kHalfBytes = 128 * 128;           // 128 rows of 128 bytes
  static constexpr int kOperand = kHalves * kHalfBytes;  // Q tile, K tile, V tile
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kTiles * kOperand;
  static constexpr int kOffV = kOffK + kStages * kOperand;
  static constexpr int kRawCodes = kKeys * D / 2, kRawScales = kKeys * D / 16;
  static constexpr int kRawBytes = kRawCodes + kRawScales;
  static constexpr int kOffRaw = kOffV + kStages * kOperand;
  static constexpr int kOffBar = kOffRaw + kRaw * kRawBytes;
  // Columns for scores: 128 of a tile each; where there is room a third 128 that the
  // tiles take in turns, so that a tile's next scores are there when its softmax is
  // done with the last ones.
  static constexpr int kBufs = kTiles * (kKeys + D) + kKeys <= 512 ? 3 : 2;
  static constexpr int kBars = 4 * kStages + 8 * kTiles + 4 + 2 * kRaw;
  static constexpr int kOffLive = kOffBar + 8 * kBars;
  static constexpr int kOffRawLive = kOffLive + 8 * kLive;
  static constexpr int kOffMisc = kOffRawLive + 8 * kRaw;
  // At least half of an SM's shared memory, so that no two CTAs of an SM wait for each other's TMEM.
  static constexpr int kNeed = kOffMisc + 64 + 1024;
  static constexpr int kSmem = kNeed > 120 * 1024 ? kNeed : 120 * 1024;
  static constexpr int kTmemS = 0, kTmemO = kBufs * kKeys;  // column offsets
  static_assert(kTmemO + kTiles * D <= 512, "TMEM");
  static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ uint32_t s_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}

__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One arrival for the warp (128 threads arriving one by one queue up on the barrier's word).
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) bar_arrive(bar);
}

__device__ __forceinline__ bool bar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Bounded wait (~4 s, or until another role gave up): sets the error word and
// the CTA's abort flag on expiry.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; i < (1u << 30); ++i) {
    if (bar_try_wait(bar, parity)) return true;
    // The clock is looked at late and seldom: reading it takes about 900
    // cycles, in which the barrier is not seen to complete.
    if ((i & 1023u) == 0u) {
      if (*abort) return false;
      const uint64_t now = now_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > 4000000000ull) break;
    }
  }
  atomicOr(&g_kv_error, (unsigned)kDevErrTimeout);
  *abort = 1;
  return false;
}

// The wait of a whole warp: false for all lanes if any gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, abort));
}

// Drain wait: bounded by time only (~1 s), ignores the abort flag.
__device__ __forceinline__ void bar_drain(uint32_t bar, uint32_t parity) {
  if (bar_try_wait(bar, parity)) return;
  const uint64_t t0 = now_ns();
  for (uint32_t i = 1; i < (1u << 30); ++i) {
    if (bar_try_wait(bar, parity)) return;
    if ((i & 255u) == 0u && now_ns() - t0 > 1000000000ull) break;
  }
  atomicOr(&g_kv_error, (unsigned)kDevErrTimeout);
}

__device__ __forceinline__ bool elect() {
  uint32_t pred = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Operand descriptors of 128-byte swizzled rows in 1024-byte atoms of eight
// rows (the stride between atoms down the rows).  lead: for an MN-major
// operand, the bytes between 64-element column blocks.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lead) {
  uint64_t dsc = (uint64_t)((addr >> 4) & 0x3FFFu);
  dsc |= (uint64_t)(lead >> 4) << 16;
  dsc |= (uint64_t)(1024u >> 4) << 32;
  dsc |= (uint64_t)1u << 46;
  dsc |= (uint64_t)2u << 61;
  return dsc;
}

// A descriptor `bytes` on: the address is in the low word, and stays there.
__device__ __forceinline__ uint64_t desc_add(uint64_t d, uint32_t bytes) {
  return (d & 0xFFFFFFFF00000000ull) | (uint32_t)((uint32_t)d + (bytes >> 4));
}

// tcgen05.mma kind::f16: FP16 operands, FP32 accumulator; M = 128.
__host__ __device__ constexpr uint32_t idesc(int n, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ void tmem_load_32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}

// Completes the tcgen05.ld that wrote v; the registers are tied to the wait so
// that no use of them can be scheduled before it.
__device__ __forceinline__ void tmem_wait_32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                 "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                 "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_store_16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16],"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}

// 16 columns, complete on return.
__device__ __forceinline__ void tmem_load_16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// What a CTA works on.
struct Job {
  Request rq;
  int b, head, row0, n_rows;  // packed rows row0 .. row0 + n_rows - 1 of the request
  int key0, n_keys;           // first key tile, and how many
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    kv_prefill_kernel(const __grid_constant__ AttnParams p, int whole, int cut) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = s_u32(smem);
  const uint32_t bar0 = sbase + C::kOffBar;
  constexpr bool kAhead = C::kBufs > kTiles;  // scores run ahead of the softmax
  auto kempty = [&](int s) { return bar0 + 8u * s; };
  auto vempty = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto kfull = [&](int s) { return bar0 + 8u * (2 * kStages + s); };  // kAhead
  auto vfull = [&](int s) { return bar0 + 8u * (3 * kStages + s); };
  const uint32_t bar1 = bar0 + 32u * kStages;
  // Scores written, and P of 64 keys written.  Where scores run ahead, steps j and
  // j + 1 may both be complete before the first of them is waited for: even and odd
  // steps have barriers of their own.
  auto sfull = [&](int t, int j) { return bar1 + 8u * (2 * t + (kAhead ? j & 1 : 0)); };
  auto pfull = [&](int t, int half, int j) { return bar1 + 8u * (2 * kTiles + 4 * t + 2 * half + (kAhead ? j & 1 : 0)); };
  auto turn = [&](int j) { return (uint32_t)(kAhead ? j >> 1 : j) & 1u; };  // their parity in step j
  auto ofull = [&](int t) { return bar1 + 8u * (6 * kTiles + t); };
  auto added = [&](int t) { return bar1 + 8u * (7 * kTiles + t); };  // kAhead: O += P(j) V is done
  // Else tile 0's first half of P(j) waits for V(j) and K(j + 1) as well: a wait less
  // for the product thread.  K may be there two steps ahead, so that odd steps
  // have a barrier of their own.
  const uint32_t pfirst_odd = bar1 + 8u * (8 * kTiles);
  auto pfirst = [&](int j) { return (j & 1) ? pfirst_odd : pfull(0, 0, 0); };
  const uint32_t qfull = pfirst_odd + 8u, k0full = qfull + 8u, drained = qfull + 16u;
  auto rfull = [&](int i) { return drained + 8u + 8u * i; };
  auto rempty = [&](int i) { return drained + 8u + 8u * (kRaw + i); };
  uint64_t* live_s = reinterpret_cast<uint64_t*>(smem + C::kOffLive);     // a byte per 16 keys: their page is there
  uint64_t* raw_live = reinterpret_cast<uint64_t*>(smem + C::kOffRawLive);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 8);
  __shared__ Request job_rq;  // the CTA's request, its index and the tile
  __shared__ int job_s[2], part_s[3];
  __shared__ long long scan_s[kThreads / 32];
  __shared__ uint2 order_s[kSorted];
  __shared__ int last_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  wait_for_preceding();
  // (The barriers and TMEM while the others' loads are on their way.)
  if (tid == 32 * (kMmaWarp + 2)) {
    for (int s = 0; s < kStages; ++s) {
      bar_init(kempty(s), 1);
      bar_init(vempty(s), 1);
      bar_init(kfull(s), kFeedWarps);
      bar_init(vfull(s), kFeedWarps);
    }
    for (int t = 0; t < kTiles; ++t) {
      for (int j = 0; j < (kAhead ? 2 : 1); ++j) {
        bar_init(sfull(t, j), 1);
        bar_init(pfull(t, 0, j), t == 0 && !kAhead ? 4 + kFeedWarps : 4);
        bar_init(pfull(t, 1, j), 4);
      }
      bar_init(ofull(t), 1);
      bar_init(added(t), 1);
    }
    bar_init(pfirst_odd, 4 + kFeedWarps);
    bar_init(qfull, kSoftWarps);
    bar_init(k0full, kFeedWarps);
    bar_init(drained, 1);
    for (int i = 0; i < kRaw; ++i) {
      bar_init(rfull(i), 1);
      bar_init(rempty(i), kFeedWarps);
    }
    *abort_flag = 0;
    job_s[0] = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s_u32(tmem_slot)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // --- which request and rows: the tiles of all requests in one line, heads next to
  // one another.  The requests with most keys a row first, so that the last CTAs are
  // short ones (four prompts, 21 heads, the longest of 3375 tokens first in the batch:
  // 91 us, and 102 in the batch's order, last to first); of a request the last tile
  // (under a causal mask the longest) first ----------------------------------------
  constexpr int kCtaRows = kRows * kTiles;
  auto tiles_of = [&](const Request& r) { return (int)(((int64_t)r.n_q * p.group + kCtaRows - 1) / kCtaRows); };
  const int2 share = share_of_requests(p, tid, kThreads);
  const int rb0 = share.x, rb1 = share.y;
  long long mine = 0;  // (q_starts that decrease can name more rows than there are)
  Request rq;
  for (int b = rb0; b < rb1; ++b) {
    rq = load_request(p, b);
    mine += tiles_of(rq);
  }
  // The first `whole` CTAs have a row tile of a KV head each, the others a piece
  // of one cut into `cut`.
  const int cut_id = (int)blockIdx.x - whole;
  const int piece = cut_id < 0 ? 0 : cut_id % cut;
  const int unit = cut_id < 0 ? (int)blockIdx.x : whole + cut_id / cut;
  if (tid == 0) {  // what the end needs of it, out of the registers until then
    part_s[0] = cut_id;
    part_s[1] = cut_id < 0 ? 1 : cut;
    part_s[2] = unit - whole;
  }
  const long long place = unit / p.kv_heads;
  long long first;  // the place of this thread's first tile in line
  if (p.batch <= kSorted) {
    uint32_t keys = 0;  // that a row tile sees, about
    if (tid < p.batch) {
      keys = (uint32_t)(p.window > 0 ? min((int64_t)rq.len, (int64_t)p.window + kCtaRows) : rq.len);
      order_s[tid] = make_uint2(keys, (uint32_t)mine);
    }
    __syncthreads();
    uint32_t ahead = 0;
    if (tid < p.batch)
      for (int i = 0; i < p.batch; ++i) {
        const uint2 o = order_s[i];
        if (o.x > keys || (o.x == keys && i > tid)) ahead += o.y;
      }
    first = ahead;
  } else {
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) scan_s[warp] = incl;
    __syncthreads();
    long long before = incl - mine, total = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += scan_s[i];
      total += scan_s[i];
    }
    first = total - before - mine;
  }
  if (place >= first && place < first + mine) {
    long long rest = first + mine - 1 - place;
    for (int b = rb0; b < rb1; ++b) {
      if (rb1 - rb0 > 1) rq = load_request(p, b);
      const int n = tiles_of(rq);
      if (rest < n) {
        job_s[0] = b;
        job_s[1] = (int)rest;
        job_rq = rq;
        break;
      }
      rest -= n;
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  Job job;
  job.b = job_s[0];
  if (job.b < 0) {  // there are fewer tiles than there could be
    if (warp == kMmaWarp)
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    return;
  }
  job.head = unit % p.kv_heads;
  job.rq = job_rq;
  job.row0 = job_s[1] * kCtaRows;
  job.n_rows = (int)min((int64_t)kCtaRows, (int64_t)job.rq.n_q * p.group - job.row0);
  {
    const int lo = seen_by(p, job.rq, (int)query_of_row(p, (uint32_t)job.row0)).x;
    const int hi = seen_by(p, job.rq, (int)query_of_row(p, (uint32_t)(job.row0 + job.n_rows - 1))).y;
    const int first = lo / kKeys, n = max(0, (hi + kKeys - 1) / kKeys - first);
    const int pieces = cut_id < 0 ? 1 : cut;
    const int from = (uint32_t)(n * piece) / (uint32_t)pieces, to = (uint32_t)(n * (piece + 1)) / (uint32_t)pieces;
    job.key0 = first + from;
    job.n_keys = to - from;
  }
  const int tiles = job.n_rows > kRows ? 2 : 1;

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ===================== softmax: one row a thread =====================
    const int t = warp >> 2, r = tid & (kRows - 1);
    const int row = t * kRows + r;
    const bool mine_row = row < job.n_rows;
    const uint32_t packed = (uint32_t)job.row0 + row, ti = query_of_row(p, packed);
    const int head = job.head * p.group + (int)(packed - ti * p.group);
    const int64_t tok = job.rq.row0 + (int64_t)ti;
    const int2 see = mine_row ? seen_by(p, job.rq, (int)ti) : make_int2(0, 0);
    // The warp's 32 rows into the swizzled Q tile as they are, kPer lanes a row, so
    // that the copies cover whole lines (a row a lane takes 32 lines a load: 4500
    // cycles a CTA, and as many to store); then, a row a lane, to FP16 scaled by a
    // power of two, in place.
    constexpr int kPer = D / 8, kPerLoad = 32 / kPer;  // lanes of a row, rows of a load
    const int64_t q_at = tok * p.ldq + (int64_t)head * D, o_at = tok * p.ldo + (int64_t)head * D;
    const int chunk = lane % kPer;
    auto q_place = [&](int qr, int c) {  // of 16-byte piece c of row qr
      return C::kOffQ + t * C::kOperand + (c >> 3) * C::kHalfBytes + qr * 128 + (((c & 7) ^ (qr & 7)) * 16);
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int src = i * kPerLoad + lane / kPer, qr = 32 * (warp & 3) + src;
      const int64_t at = __shfl_sync(0xFFFFFFFFu, q_at, src);
      const bool there = t * kRows + qr < job.n_rows;  // zeros else
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sbase + q_place(qr, chunk)),
                   "l"(p.q + (there ? at + 8 * chunk : 0)), "r"(there ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    float factor;
    {
      uint4 raw[kPer];
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        raw[i] = *reinterpret_cast<const uint4*>(smem + q_place(r, i));
        using nvfp4::max_abs_bf16x2;  // (a NaN is passed over: its own product is one)
        amax = max_abs_bf16x2(amax, max_abs_bf16x2(max_abs_bf16x2(raw[i].x, raw[i].y), max_abs_bf16x2(raw[i].z, raw[i].w)));
      }
      const int e = query_exponent(max(amax & 0x7FFFu, (amax >> 16) & 0x7FFFu));
      // A negative scale goes to the query, so that larger scores are larger sums.
      const float up = p.qk_scale < 0.0f ? -pow2(e) : pow2(e);
      factor = score_factor(p, e);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 x = __fmul2_rn(make_float2(bf16_lo(v[k]), bf16_hi(v[k])), make_float2(up, up));
          h[k] = pack_f16x2(x.x, x.y);
        }
        *reinterpret_cast<uint4*>(smem + q_place(r, i)) = make_uint4(h[0], h[1], h[2], h[3]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      warp_arrive(qfull, lane);
    }
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t to = tmem + lanes + C::kTmemO + t * D;
    int buf = t;  // of the scores
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    if (t < tiles) {
      // Key range that every row of this warp sees, for tiles that need no mask.
      int lo_max = mine_row ? see.x : 0, hi_min = mine_row ? see.y : 0x7FFFFFFF;
      lo_max = __reduce_max_sync(0xFFFFFFFFu, lo_max);
      hi_min = __reduce_min_sync(0xFFFFFFFFu, hi_min);
      float2 sum = make_float2(0.0f, 0.0f);
      for (int j = 0; j < job.n_keys; ++j) {
        const uint32_t ts = tmem + lanes + C::kTmemS + buf * kKeys;
        if constexpr (kAhead) buf = buf + tiles >= C::kBufs ? buf + tiles - C::kBufs : buf + tiles;
        if (!warp_wait(sfull(t, j), turn(j), abort_flag)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        // The row's 128 scores, all at once.
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_load_32(ts + 32 * c, v[c]);
        const uint64_t live = live_s[j % kLive];
        const int tok0 = (job.key0 + j) * kKeys;
        const bool edge = live != 0x0101010101010101ull || tok0 < lo_max || tok0 + kKeys > hi_min;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_wait_32(v[c]);
        if (edge) {  // scores of keys not seen become -inf
          const int c_lo = see.x - tok0, c_hi = see.y - tok0;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int lo = min(max(c_lo - 32 * c, 0), 32), hi = min(max(c_hi - 32 * c, 0), 32);
            uint32_t seen = (hi == 32 ? ~0u : (1u << hi) - 1u) & ~(lo == 32 ? ~0u : (1u << lo) - 1u);
            const uint32_t groups = (uint32_t)(live >> (16 * c));
            seen &= ((groups & 1u) ? 0xFFFFu : 0u) | ((groups & 0x100u) ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((seen >> i) & 1u)) v[c][i] = 0xFF800000u;
          }
        }
        float tops[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tops[c] = __uint_as_float(v[c][0]);
#pragma unroll
          for (int i = 1; i < 31; i += 2)
            tops[c] = fmaxf(fmaxf(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1])), tops[c]);
          tops[c] = fmaxf(__uint_as_float(v[c][31]), tops[c]);
        }
        float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        if (top != -INFINITY) top *= factor;
        if (__any_sync(0xFFFFFFFFu, top > m + kRaise)) {
          const float mn = fmaxf(m, top);
          const float keep = m == mn ? 1.0f : exp2_fast(m - mn);
          m = mn;
          sum.x *= keep;
          sum.y *= keep;
          if (j > 0) {
            if constexpr (kAhead) {
              // (The scores' commit covers O += P(j - 2) V, so this is the phase waited for.)
              if (!warp_wait(added(t), (j - 1) & 1, abort_flag)) {
                ok = false;
                break;
              }
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            }
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_load_16(to + 16 * c, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
              tmem_store_16(to + 16 * c, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.0f : kHead - m;
        // A step's weights are added up by themselves: many that are each below the last
        // place of the row's sum count by what they are together.
        float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t h[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[c][2 * i]), __uint_as_float(v[c][2 * i + 1])),
                                        make_float2(factor, factor), make_float2(off, off));
            const float2 w = make_float2(exp2_fast(x.x), exp2_fast(x.y));
            part = __fadd2_rn(part, w);
            h[i] = pack_f16x2(w.x, w.y);
          }
          tmem_store_16(ts + 16 * c, h);
          if (c & 1) {  // 64 keys' P: the product may start on them
            tmem_stored();
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            warp_arrive(!kAhead && t == 0 && c == 1 ? pfirst(j) : pfull(t, c >> 1, j), lane);
          }
        }
        sum = __fadd2_rn(sum, part);
      }
      l = sum.x + sum.y;
      // (Without keys no product has waited for the other warps' queries, over which the output is staged.)
      if (ok) ok = warp_wait(job.n_keys > 0 ? ofull(t) : qfull, 0, abort_flag);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      float weight[kMaxPieces];  // of the pieces' partial outputs
      const int part_id = part_s[0], pieces = part_s[1], cut_unit = part_s[2];  // (part_id: place of the partial result)
      if (pieces > 1) {  // (also when a wait has run out: all of these warps meet at the barriers)
        // Partial results, column by column: a warp's 32 rows lie together.
        float* part = p.part_o + (int64_t)part_id * (kCtaRows * D) + row;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          if (ok && job.n_keys > 0) {
            tmem_load_32(to + 32 * c, v);
            tmem_wait_32(v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) part[(32 * c + i) * kCtaRows] = __uint_as_float(v[i]);
        }
        p.part_ml[(int64_t)part_id * kCtaRows + row] = make_float2(m, l);
        __threadfence();
        asm volatile("bar.sync 1, %0;" ::"r"(kRows * tiles) : "memory");  // the softmax warps that have rows
        if (tid == 0) {
          last_s = atomicAdd(p.count + cut_unit, 1u) == (unsigned)(pieces - 1);
          if (last_s) p.count[cut_unit] = 0;  // as the next call needs it
        }
        asm volatile("bar.sync 1, %0;" ::"r"(kRows * tiles) : "memory");
        ok = ok && last_s != 0;  // the others are done
        if (ok) {
          __threadfence();
          const float2* ml = p.part_ml + (int64_t)cut_unit * pieces * kCtaRows + row;
          float ms[kMaxPieces], ls[kMaxPieces];
          m = -INFINITY;
#pragma unroll
          for (int i = 0; i < kMaxPieces; ++i) {
            const float2 x = i < pieces ? __ldcg(ml + i * kCtaRows) : make_float2(-INFINITY, 0.0f);
            ms[i] = x.x;
            ls[i] = x.y;
            m = fmaxf(m, x.x);
          }
          l = 0.0f;
#pragma unroll
          for (int i = 0; i < kMaxPieces; ++i) {
            weight[i] = ms[i] == m ? 1.0f : exp2_fast(ms[i] - m);
            l += weight[i] * ls[i];
          }
        }
      }
      if (ok) {
        const float inv = l > 0.0f ? p.v_scale / l : (l == 0.0f ? 0.0f : l);
        // Through shared memory (this warp's part of its Q tile, which the products
        // are done with), so that the stores cover whole lines.
        uint8_t* stage = smem + C::kOffQ + t * C::kOperand + (warp & 3) * (32 * D * 2);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          if (pieces > 1) {
            const float* part = p.part_o + (int64_t)cut_unit * pieces * (kCtaRows * D) + (32 * c) * kCtaRows + row;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0;
#pragma unroll 1
            for (int k = 0; k < pieces; ++k) {
              float w = weight[0];  // weight[k], without indexing registers
#pragma unroll
              for (int i = 1; i < kMaxPieces; ++i) w = k == i ? weight[i] : w;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                v[i] = __float_as_uint(
                    fmaf(w, __ldcg(part + (int64_t)k * (kCtaRows * D) + i * kCtaRows), __uint_as_float(v[i])));
            }
          } else if (job.n_keys > 0) {
            tmem_load_32(to + 32 * c, v);
            tmem_wait_32(v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_bf16x2(__uint_as_float(v[8 * i + 2 * k]) * inv * p.v_unit,
                                 __uint_as_float(v[8 * i + 2 * k + 1]) * inv * p.v_unit);
            *reinterpret_cast<uint4*>(stage + lane * (2 * D) + (((4 * c + i) ^ (lane & 7)) * 16)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int src = i * kPerLoad + lane / kPer;
          const int64_t at = __shfl_sync(0xFFFFFFFFu, o_at, src);
          const uint4 w = *reinterpret_cast<const uint4*>(stage + src * (2 * D) + ((chunk ^ (src & 7)) * 16));
          if (t * kRows + 32 * (warp & 3) + src < job.n_rows) *reinterpret_cast<uint4*>(p.out + at + 8 * chunk) = w;
        }
        if (mine_row && p.lse != nullptr)
          p.lse[tok * p.q_heads + head] = l == 0.0f ? -INFINITY : (m - kHead + log2f(l)) * 0.6931471805599453f;
      }
    }
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // ===================== feeding K and V =====================
    const int x = tid - 32 * kSoftWarps;
    constexpr int kCpr = D / 32;                 // 16-byte pieces (32 elements) of a row of codes
    constexpr int kPieces = kKeys * kCpr / 128;  // per thread and tile: 4 or 2
    const int part = x % kCpr;
    const int row_in = x / kCpr;                 // + piece * (128 / kCpr)
    // 32 elements to four 16-byte pieces of a swizzled row.
    auto put = [&](uint8_t* base, int row, const uint4& codes, uint32_t scales) {
      const uint32_t h = e4m3x2_to_f16x2(scales);
      const uint32_t s0 = __byte_perm(h, h, 0x1010), s1 = __byte_perm(h, h, 0x3232);
      // Lanes of the row's two halves take their pieces in different orders, so that no bank is asked twice.
      const bool turn = D == 128 && (part & 2);
      const uint32_t w[4] = {turn ? codes.z : codes.x, turn ? codes.w : codes.y, turn ? codes.x : codes.z,
                             turn ? codes.y : codes.w};
      const uint32_t sa = turn ? s1 : s0, sb = turn ? s0 : s1;
      uint8_t* dst = base + (D == 128 ? (part >> 1) * C::kHalfBytes : 0) + row * 128;
      const int c0 = (part & 1) * 4 + (turn ? 2 : 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t s = k < 2 ? sa : sb;
        *reinterpret_cast<uint4*>(dst + (((c0 ^ k) ^ (row & 7)) * 16)) =
            make_uint4(hmul2(e2m1x2_to_f16x2<0>(w[k]), s), hmul2(e2m1x2_to_f16x2<1>(w[k]), s),
                       hmul2(e2m1x2_to_f16x2<2>(w[k]), s), hmul2(e2m1x2_to_f16x2<3>(w[k]), s));
      }
    };
    bool ok = true;
    for (int n = 0; n < 2 * job.n_keys && ok; ++n) {  // K and V of a tile in turns
      const int j = n >> 1, s = j % kStages, slot = n % kRaw;
      const bool is_v = n & 1;
      ok = warp_wait(rfull(slot), (n / kRaw) & 1, abort_flag);
      if (!ok) break;
      const uint8_t* raw = smem + C::kOffRaw + slot * C::kRawBytes;
      const uint64_t live = raw_live[slot];
      uint4 codes[kPieces];
      uint32_t scales[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int row = row_in + i * (128 / kCpr);
        codes[i] = *reinterpret_cast<const uint4*>(raw + row * (D / 2) + 16 * part);
        scales[i] = *reinterpret_cast<const uint16_t*>(raw + C::kRawCodes + row * (D / 16) + 2 * part);
        // Rows of no token and of tokens that no query sees get scales of 0, so that nothing of a page's rest,
        // nor of a page that is no longer the request's, gets into a sum.
        const int tk = (job.key0 + j) * kKeys + row;
        if (!((live >> (8 * (row >> 4))) & 1u) || tk < job.rq.lo || tk >= job.rq.hi) scales[i] = 0;
      }
      warp_arrive(rempty(slot), lane);
      ok = warp_wait(is_v ? vempty(s) : kempty(s), ((j / kStages) & 1) ^ 1u, abort_flag);
      if (!ok) break;
      uint8_t* dst = smem + (is_v ? C::kOffV : C::kOffK) + s * C::kOperand;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) put(dst, row_in + i * (128 / kCpr), codes[i], scales[i]);
      if (!is_v && x == 0) live_s[j % kLive] = live;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      if constexpr (kAhead)
        warp_arrive(is_v ? vfull(s) : kfull(s), lane);
      else if (!is_v)
        warp_arrive(j == 0 ? k0full : pfirst(j - 1), lane);  // V(j - 1) is there, too
      else if (j + 1 == job.n_keys)
        warp_arrive(pfirst(j), lane);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kMmaWarp) {
    // ===================== the products =====================
    auto scores = [&](int t, int buf, int s) {  // S_t = Q_t K^T
      const uint64_t a = sw128_desc(sbase + C::kOffQ + t * C::kOperand, 16);
      const uint64_t b = sw128_desc(sbase + C::kOffK + s * C::kOperand, 16);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t step = (k >> 2) * C::kHalfBytes + (k & 3) * 32;
        mma_ss(tmem + C::kTmemS + buf * kKeys, desc_add(a, step), desc_add(b, step), idesc(kKeys, false), k > 0);
      }
    };
    auto output = [&](int t, int buf, int s, int half, bool accumulate) {  // O_t += P_t V over 64 keys
      const uint64_t b = sw128_desc(sbase + C::kOffV + s * C::kOperand, C::kHalfBytes);
#pragma unroll
      for (int k = 4 * half; k < 4 * half + 4; ++k)
        mma_ts(tmem + C::kTmemO + t * D, tmem + C::kTmemS + buf * kKeys + 8 * k, desc_add(b, k * 2048),
               idesc(D, true), accumulate || k > 0);
    };
    if (elect()) {  // one thread waits and issues: no votes between a wait and its product
      if constexpr (kAhead) {
        // In the order (tile 0, tile 1) of step 0, of step 1, ...; scores are tiles + 1
        // places ahead of outputs, in the columns that the last output has read P from.
        const int n_all = job.n_keys * tiles;
        int s_n = 0, s_j = 0, s_t = 0, s_buf = 0;
        auto next_scores = [&]() {
          if (s_t == 0) {
            if (!bar_wait(kfull(s_j % kStages), (s_j / kStages) & 1, abort_flag)) return false;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          }
          scores(s_t, s_buf, s_j % kStages);
          commit(sfull(s_t, s_j));
          if (s_t == tiles - 1) commit(kempty(s_j % kStages));
          s_buf = s_buf + 1 == C::kBufs ? 0 : s_buf + 1;
          if (++s_t == tiles) s_t = 0, ++s_j;
          ++s_n;
          return true;
        };
        bool ok = n_all > 0 && bar_wait(qfull, 0, abort_flag);
        while (ok && s_n < min(tiles + 1, n_all)) ok = next_scores();
        int buf = 0;
        for (int j = 0; j < job.n_keys && ok; ++j) {
          if (p.stall && blockIdx.x == 0 && j == 2) break;  // test hook: the others run into their bounded waits
          const int s = j % kStages;
          for (int t = 0; t < tiles && ok; ++t) {
            ok = bar_wait(pfull(t, 0, j), turn(j), abort_flag) &&
                 (t > 0 || bar_wait(vfull(s), (j / kStages) & 1, abort_flag));
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            output(t, buf, s, 0, j > 0);
            ok = bar_wait(pfull(t, 1, j), turn(j), abort_flag);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            output(t, buf, s, 1, true);
            commit(added(t));
            if (j + 1 == job.n_keys) commit(ofull(t));
            if (t == tiles - 1) commit(vempty(s));
            buf = buf + 1 == C::kBufs ? 0 : buf + 1;
            if (s_n < n_all) ok = next_scores();
          }
        }
      } else {
        bool ok = job.n_keys > 0 && bar_wait(qfull, 0, abort_flag) && bar_wait(k0full, 0, abort_flag);
        if (ok) {
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          for (int t = 0; t < tiles; ++t) {
            scores(t, t, 0);
            commit(sfull(t, 0));
          }
          commit(kempty(0));
        }
        for (int j = 0; j < job.n_keys && ok; ++j) {
          if (p.stall && blockIdx.x == 0 && j == 2) break;  // test hook: the others run into their bounded waits
          const int s = j % kStages, sn = (j + 1) % kStages;
          const bool more = j + 1 < job.n_keys;
          for (int t = 0; t < tiles && ok; ++t) {
            ok = t == 0 ? bar_wait(pfirst(j), (j >> 1) & 1, abort_flag) : bar_wait(pfull(t, 0, j), j & 1, abort_flag);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            output(t, t, s, 0, j > 0);
            ok = bar_wait(pfull(t, 1, j), j & 1, abort_flag);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            output(t, t, s, 1, true);
            if (!more) commit(ofull(t));
            if (more) {
              scores(t, t, sn);
              commit(sfull(t, j + 1));
            }
            if (t == tiles - 1) {
              commit(vempty(s));
              if (more) commit(kempty(sn));
            }
          }
        }
      }
      commit(drained);
    }
    __syncwarp();
    bar_drain(drained, 0);
    } else if (warp == kCopyWarp) {
      // ===================== bringing codes and scales =====================
      // Lanes 0..7: codes of a tile's (up to eight) pieces of a page each, lanes
      // 8..15: their scales.  Sizes are multiples of 16 tokens, so of 16 bytes.
      const int shift = min(p.page_shift, 7), piece = lane & 7;  // 2^shift tokens a piece
      const bool is_scale = lane & 8;
      const uint32_t per_token = is_scale ? D / 16 : D / 2;
      const bool mine_piece = lane < 16 && piece < (kKeys >> shift);
      const int32_t* row = p.table + (int64_t)job.b * p.max_pages;
      auto look_up = [&](int j) {  // the entry of the piece's page, -1 where there is nothing to read
        const int tk = (job.key0 + j) * kKeys + (piece << shift);
        return mine_piece && j < job.n_keys && tk < job.rq.hi ? row[tk >> p.page_shift] : -1;
      };
      int entry = look_up(0);
      int issued = 0;
      for (int j = 0; j < job.n_keys; ++j) {
        const int page = entry < p.num_pages ? entry : -1;
        entry = look_up(j + 1);  // (not looked at before the next step)
        const int tk = (job.key0 + j) * kKeys + (piece << shift);
        const int tokens = page >= 0 ? min(1 << shift, (job.rq.hi - tk + 15) & ~15) : 0;
        const int64_t at = page >= 0 ? (((int64_t)page * p.kv_heads + job.head) << p.page_shift) + (tk & ((1 << p.page_shift) - 1)) : 0;
        const uint32_t bytes = tokens * per_token;
        const uint32_t total = __reduce_add_sync(0xFFFFFFFFu, bytes);
        // Group g of 16 tokens lies in piece g >> (shift - 4).
        const int g_tokens = __shfl_sync(0xFFFFFFFFu, tokens, piece >> (shift - 4));
        const bool g_live = g_tokens > 16 * (piece & ((1 << (shift - 4)) - 1));
        bool ok = true;
        for (int v = 0; v < 2 && ok; ++v) {
          const int n = 2 * j + v, slot = n % kRaw;
          ok = warp_wait(rempty(slot), ((n / kRaw) & 1) ^ 1u, abort_flag);
          if (!ok) break;
          if (lane < 8) reinterpret_cast<uint8_t*>(raw_live + slot)[lane] = g_live ? 1 : 0;
          __syncwarp();
          if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(rfull(slot)), "r"(total) : "memory");
          __syncwarp();
          if (bytes != 0) {
            const uint8_t* src = (is_scale ? (v ? p.v_scales : p.k_scales) : (v ? p.v_codes : p.k_codes)) + at * per_token;
            const uint32_t dst = sbase + C::kOffRaw + slot * C::kRawBytes + (is_scale ? C::kRawCodes : 0) +
                                 (uint32_t)(piece << shift) * per_token;
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                "l"(src), "r"(bytes), "r"(rfull(slot))
                : "memory");
          }
          ++issued;
        }
        if (!ok) break;
      }
      // Copies in flight end before the CTA does.
      for (int n = max(0, issued - kRaw); n < issued; ++n) bar_drain(rfull(n % kRaw), (n / kRaw) & 1);
    }
  }

  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == kMmaWarp) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

template <int D>
cudaError_t launch_prefill(const AttnParams& p, int64_t whole, int64_t rest, int cut, cudaStream_t s) {
  using C = Cfg<D>;
  static DeviceTable configured;
  int dev = 0;
  cudaGetDevice(&dev);
  const int cfg = per_device(configured, dev, [](int) {
    const cudaError_t e =
        cudaFuncSetAttribute(kv_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    return e == cudaSuccess ? 1 : -(int)e;
  });
  if (cfg <= 0) return (cudaError_t)(-cfg);
  return launch_overlapping(kv_prefill_kernel<D>, dim3((unsigned)(whole + rest * cut)), dim3(kThreads), C::kSmem, s, p,
                            (int)whole, cut);
}

// As many row tiles (of all KV heads) as there can be: a request's last one may be short.
int64_t most_units(const KvAttnShape& shape) {
  constexpr int64_t kCtaRows = kRows * kTiles;
  const int64_t rows = shape.total_q * (shape.q_heads / shape.kv_heads), most = rows < shape.batch ? rows : shape.batch;
  return (rows + (kCtaRows - 1) * most) / kCtaRows * shape.kv_heads;
}

// How a call's row tiles go to CTAs: `whole` of them as they are, the `rest`
// that would be an unfilled wave cut into `cut` pieces each.
struct Plan {
  int64_t whole, rest;
  int cut;
  double cost;  // in key tiles, one after another
};

// As many pieces as shorten the call, a CTA taking about as long as three key
// tiles to start and finish, and the join of pieces as long as two.
Plan plan_for(int64_t units, int64_t max_kv, int sms) {
  const double keys = (double)((max_kv + kKeys - 1) / kKeys);
  Plan plan;
  plan.whole = units / sms * sms;
  plan.rest = units - plan.whole;
  plan.cut = 1;
  double best = plan.rest > 0 ? keys + 3 : 0.0;
  for (int n = 2; n <= kMaxPieces && plan.rest * n <= kMaxPieceCtas; ++n) {
    const double c = (double)((plan.rest * n + sms - 1) / sms) * (ceil(keys / n) + 3) + 2;
    if (c < best) {
      best = c;
      plan.cut = n;
    }
  }
  if (plan.cut == 1) {
    plan.whole += plan.rest;
    plan.rest = 0;
  }
  plan.cost = (double)(units / sms) * (keys + 3) + best;
  return plan;
}

}  // namespace

size_t kv_attn_tiles_workspace(const KvAttnShape& s) {
  // (No less for more units, of which fewer may be cut: a workspace serves smaller calls too.)
  const int64_t units = most_units(s), ctas = units * kMaxPieces < kMaxPieceCtas ? units * kMaxPieces : kMaxPieceCtas;
  return kCounters * sizeof(unsigned) + (size_t)ctas * (kRows * kTiles) * (size_t)(s.head_dim + 2) * sizeof(float);
}

double kv_attn_tiles_cost(const KvAttnShape& s, int64_t max_kv) {
  // 1.8 us a key tile, whatever d and the rows of the last tile; tiles of many requests end at different times.
  return 7.0 + 1.8 * (s.batch >= 8 ? 0.85 : 1.0) * plan_for(most_units(s), max_kv, sm_count()).cost;
}

cudaError_t launch_kv_attn_tiles(const AttnParams& params, const KvAttnShape& shape, int64_t max_kv, void* workspace,
                                 cudaStream_t s) {
  AttnParams p = params;
  const Plan plan = plan_for(most_units(shape), max_kv, sm_count());
  p.count = static_cast<unsigned*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.count + kCounters);
  p.part_o = reinterpret_cast<float*>(p.part_ml + plan.rest * plan.cut * (kRows * kTiles));
  return shape.head_dim == 128 ? launch_prefill<128>(p, plan.whole, plan.rest, plan.cut, s)
                               : launch_prefill<64>(p, plan.whole, plan.rest, plan.cut, s);
}

cudaError_t read_and_clear_kv_error(unsigned int* bits) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv_error, sizeof v);
  if (e != cudaSuccess) return e;
  if (v != 0) e = cudaMemcpyToSymbol(g_kv_error, &zero, sizeof zero);  // (clearing takes as long as reading)
  *bits = v;
  return e;
}

}  // namespace fh
