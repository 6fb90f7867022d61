// mx_b128.cuh -- arithmetic of E4M3 blocks of 128 under one fp32 scale, shared by the kernels that
// write such operands:
//   a = max(abs-max, 2^-100);  r = 448 / a;  scale = a / 448;  code_i = E4M3(x_i * r),
// every step one fp32 operation rounded to nearest even, the code saturating at 448 and keeping the
// sign of zero. A block holding a NaN or an infinity gets scale NaN and codes 0x7F.
#pragma once

#include "mx_device.cuh"
#include "mx_expert.h"

namespace mxq {

struct Factors {
  float r, scale;
};

__device__ __forceinline__ Factors block_factors_b128(uint32_t amax_bits) {
  Factors f;
  const float a = fmaxf(__uint_as_float(amax_bits), kB128AmaxFloor);
  f.r = __fdiv_rn(448.0f, a);
  f.scale = __fdiv_rn(a, 448.0f);
  if (amax_bits >= 0x7F800000u) f.r = f.scale = __uint_as_float(0x7FC00000u);
  return f;
}

// Sign-free bf16x2 abs-max accumulation; the two halves are joined by amax_bits. NaN propagates:
// the patterns are compared as integers, and those of NaN lie above that of infinity.
__device__ __forceinline__ uint32_t amax2(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t amax_join(uint32_t m) {  // -> fp32 bits
  return max(m & 0xFFFFu, m >> 16) << 16;
}

// four values (bf16x2 words w0, w1: lower index in the low half) times r -> four code bytes
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float r) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(d)
      : "f"(__fmul_rn(bf16_lo(w0), r)), "f"(__fmul_rn(bf16_hi(w0), r)),
        "f"(__fmul_rn(bf16_lo(w1), r)), "f"(__fmul_rn(bf16_hi(w1), r)));
  return d;
}

// two values (separate fp32) -> two code bytes
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(d) : "f"(lo), "f"(hi));
  return d;
}

// Codes are written once and not read again here: evict-first.
__device__ __forceinline__ void store16B(void* p, const uint32_t* r) {
  asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

}  // namespace mxq
