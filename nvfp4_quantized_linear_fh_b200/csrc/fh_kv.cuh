// fh_kv.cuh -- what the kernels of the paged NVFP4 key/value cache share: the
// cache's geometry on the device and the conversions of its codes and scales.
//
// A cache holds one attention layer's keys and values in pages of page_size
// tokens.  Keys and values each have codes [num_pages, kv_heads, page_size,
// d / 2] (E2M1, element 2j of a head in the low nibble of byte j) and scales
// [num_pages, kv_heads, page_size, d / 16] (E4M3), with x ~ code * scale * s_g.
// A token's slot is page * page_size + its place in the page.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fh {
namespace kv {

// Nothing that the stream's preceding kernels write may be read, and nothing that
// they read be written, before this; the next kernel's CTAs may come up from here on.
// Every thread of a kernel comes here first, so a kernel that has ended says that
// all before it have, too.
__device__ __forceinline__ void wait_for_preceding() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Two nibbles (the low one first) of byte `i` of w as FP16 values: E2M1 is a
// subset of FP16, so the conversion is exact.
template <int kByte>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
  static_assert(kByte >= 0 && kByte < 4, "byte of a word");
  uint32_t r;
  if constexpr (kByte == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (kByte == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (kByte == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Two E4M3 bytes (the low one first) as FP16 values (exact: FP16 holds every E4M3 value).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t w) {
  __half2 h;
  *reinterpret_cast<uint32_t*>(&h) = w;
  return __half22float2(h);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// log2 of the power of two that brings a query row whose largest BF16 magnitude
// (bits) is `amax` to [2^13, 2^14): scaled so, the row goes to FP16 without a
// rounding that matters (elements 2^-27 of the largest and more stay exact, the
// others are off by at most half an FP16 subnormal's step, 2^-25, which is 2^-38
// of the largest), and its products with keys of up to
// 2688 stay far inside FP32.  0 for a zero or non-finite row.
__device__ __forceinline__ int query_exponent(uint32_t amax) {
  const int e = (int)(amax >> 7);
  if (amax == 0 || e == 255) return 0;
  return min(140 - e, 126);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // -126 <= e <= 127

}  // namespace kv
}  // namespace fh
