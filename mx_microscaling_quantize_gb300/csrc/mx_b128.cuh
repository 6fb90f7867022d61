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

// four fp32 values (lower index first) -> four code bytes
__device__ __forceinline__ uint32_t codes4(float w, float x, float y, float z) {
  uint32_t d;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(d)
      : "f"(w), "f"(x), "f"(y), "f"(z));
  return d;
}

// four code bytes -> two pairs of their exact values
__device__ __forceinline__ void values4(uint32_t w, uint64_t& a, uint64_t& b) {
  asm("{\n\t.reg .b16 lo, hi, p, q;\n\t.reg .b32 h;\n\t.reg .f32 x, y;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 h, lo;\n\tmov.b32 {p, q}, h;\n\t"
      "cvt.f32.f16 x, p;\n\tcvt.f32.f16 y, q;\n\tmov.b64 %0, {x, y};\n\t"
      "cvt.rn.f16x2.e4m3x2 h, hi;\n\tmov.b32 {p, q}, h;\n\t"
      "cvt.f32.f16 x, p;\n\tcvt.f32.f16 y, q;\n\tmov.b64 %1, {x, y};\n\t}"
      : "=l"(a), "=l"(b)
      : "r"(w));
}

// Two fp32 values in a register pair, and packed arithmetic on them: half the instructions.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ uint64_t pair(float v) { return pair(v, v); }
__device__ __forceinline__ uint64_t bf16_pair(uint32_t w) { return pair(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ float lo_of(uint64_t p) {
  float lo;
  asm("mov.b64 {%0, _}, %1;" : "=f"(lo) : "l"(p));
  return lo;
}
__device__ __forceinline__ float hi_of(uint64_t p) {
  float hi;
  asm("mov.b64 {_, %0}, %1;" : "=f"(hi) : "l"(p));
  return hi;
}
__device__ __forceinline__ uint32_t codes4(uint64_t a, uint64_t b) {
  return codes4(lo_of(a), hi_of(a), lo_of(b), hi_of(b));
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint32_t bf16_word(uint64_t p) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo_of(p)), "f"(hi_of(p)));
  return r;
}

// abs-max of the 2 N values of N pairs, as sign-free fp32 bits; NaN propagates.
template <int N>
__device__ __forceinline__ uint32_t absmax_pairs(const uint64_t* v) {
  float m = absmax3(lo_of(v[0]), hi_of(v[0]), hi_of(v[0]));
#pragma unroll
  for (int i = 1; i < N; ++i) m = absmax3(m, lo_of(v[i]), hi_of(v[i]));
  return __float_as_uint(m) & 0x7FFFFFFFu;
}

// Maxima of N values of each lane over 2^STEPS lanes (those that differ in STEPS bits, the lowest of them bit
// LOW), N of them, found by halves: the first steps exchange half of the values that are left and keep the other
// half, so log2 N of them give each lane one value, index (its highest log2 N bits of STEPS). take gives a lane any
// of the N from the lane that has it.
template <int N, int STEPS, int LOW = 0>
struct RunMax {
  static constexpr int kHalvings = N == 8 ? 3 : N == 4 ? 2 : N == 2 ? 1 : 0;
  static_assert(N == 1 || N == 2 || N == 4 || N == 8, "values of a lane");
  static_assert(kHalvings <= STEPS, "more values than lanes");

  int lane;
  __device__ __forceinline__ int index() const { return (lane >> LOW & ((1 << STEPS) - 1)) >> (STEPS - kHalvings); }
  // whether this lane is the first that has its value
  __device__ __forceinline__ bool first() const { return (lane >> LOW & ((1 << (STEPS - kHalvings)) - 1)) == 0; }
  __device__ __forceinline__ uint32_t reduce(uint32_t (&m)[N]) const {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int d = 1 << (LOW + STEPS - 1 - s), left = N >> (s + 1);
      if (s < kHalvings) {
        const bool high = lane & d;
#pragma unroll
        for (int j = 0; j < left; ++j) {
          const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, high ? m[j] : m[j + left], d);
          m[j] = max(high ? m[j + left] : m[j], got);
        }
      } else {
        m[0] = max(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], d));
      }
    }
    return m[0];
  }
  __device__ __forceinline__ float take(float v, int j) const {
    const int others = lane & ~(((1 << STEPS) - 1) << LOW);
    return __shfl_sync(0xFFFFFFFFu, v, others | j << (LOW + STEPS - kHalvings));
  }
};

// N runs of 8 consecutive values per lane (in pairs) whose blocks 16 lanes hold: their codes, put(n, lo, hi)
// with 8 bytes of run n, and their scales, scale(n, s) from one lane of the 16. Each lane works out the
// factors of one of the runs' blocks: a block's two quotients take as many instructions as the codes of ten
// values.
template <int N, typename Put, typename Scale>
__device__ __forceinline__ void run_codes(const uint64_t (&v)[N][4], int lane, Put&& put, Scale&& scale) {
  const RunMax<N, 4> max_of{lane};
  uint32_t m[N];
#pragma unroll
  for (int n = 0; n < N; ++n) m[n] = absmax_pairs<4>(v[n]);
  const Factors f = block_factors_b128(max_of.reduce(m));
  if (max_of.first()) scale(max_of.index(), f.scale);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint64_t r = pair(max_of.take(f.r, n));
    put(n, codes4(mul_pair(v[n][0], r), mul_pair(v[n][1], r)),
        codes4(mul_pair(v[n][2], r), mul_pair(v[n][3], r)));
  }
}

// Codes are written once and not read again here: evict-first.
__device__ __forceinline__ void store8B(void* p, uint32_t lo, uint32_t hi) {
  asm volatile("st.global.cs.v2.b32 [%0], {%1, %2};" ::"l"(p), "r"(lo), "r"(hi) : "memory");
}

// two values (separate fp32) -> two code bytes
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(d) : "f"(lo), "f"(hi));
  return d;
}

__device__ __forceinline__ void store16B(void* p, const uint32_t* r) {
  asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

}  // namespace mxq
