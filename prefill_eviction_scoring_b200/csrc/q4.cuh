// The 4-bit paged cache's format (include/waits.h, waits_q4_cache) on the
// device: where a slot's bytes are, e2m1 conversions, the scale of a group.
#pragma once

#include <cuda_fp16.h>

#include "waits_internal.cuh"

namespace waits {

// One page (block_size tokens of one KV head): K codes, K scales, V codes, V
// scales.
template <int D>
struct Q4Page {
  static constexpr int kCode = D / 2;     // bytes of codes per token
  static constexpr int kScale = D / 16;   // bytes of scales per token (bf16 per 32)
  static constexpr int kToken = 2 * (kCode + kScale);
  __host__ __device__ static size_t bytes(int log_bs) { return (size_t)kToken << log_bs; }
  // K's (which = 0) or V's codes of token `off` in the page; its scales
  __device__ static int code(int which, int log_bs, int off) {
    return which * ((kToken / 2) << log_bs) + off * kCode;
  }
  __device__ static int scale(int which, int log_bs, int off) {
    return which * ((kToken / 2) << log_bs) + (kCode << log_bs) + off * kScale;
  }
};

__device__ inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ inline uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The four bytes of w, two e2m1 codes each -> four half pairs (exact).
__device__ inline void e2m1_to_half(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

__device__ inline float2 half2_to_float2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace waits
