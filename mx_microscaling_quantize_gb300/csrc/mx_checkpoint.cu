// mx_checkpoint.cu -- what a backward pass makes of an activation checkpoint (E4M3 codes with a scale per
// 1 x 128 block, as the quantisation of rows writes them): its values, and the transposed operand with a
// scale per 128 x 1 block that the weights' gradient contracts over (b128_recols_kernel).
#include "mx_b128.cuh"
#include "mx_device.cuh"
#include "mx_launch.h"
#include "mx_train.h"

namespace mxq {

namespace {

// A lane's 16 codes of a row times their block's scale: 17 bytes read, 32 or 64 written. Bound by memory:
// 8192 x 8192 into bf16 31.5 us (30.4 at the rate of a plain copy), into fp32 49.5.
template <bool F32>
__global__ void __launch_bounds__(256) b128_dequant_kernel(DequantB128Args a, int64_t chunks, int64_t items) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (it >= items) return;
  const int64_t r = it / chunks, col = it % chunks * 16;
  const int64_t src = a.index ? load_s32(a.index + r) : r;
  float v[16];
  if (src >= 0 && src < a.M) {
    uint32_t w[4];
    load16B(a.codes + src * a.K + col, w);
    const float s = load_f32(a.scales + col / kB128 * a.M + src);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      e4m3x2_to_f32(w[j] & 0xFFFFu, v[4 * j], v[4 * j + 1]);
      e4m3x2_to_f32(w[j] >> 16, v[4 * j + 2], v[4 * j + 3]);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __fmul_rn(v[j], s);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = 0.0f;
  }
  uint32_t o[8];
  if constexpr (F32) {
    float* to = static_cast<float*>(a.y) + r * a.K + col;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(v[8 * h + j]);
      store32B(to + 8 * h, o);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(o[j]) : "f"(v[2 * j]), "f"(v[2 * j + 1]));
    }
    store32B(static_cast<uint16_t*>(a.y) + r * a.K + col, o);
  }
}

}  // namespace

cudaError_t launch_b128_dequant(const DequantB128Args& a, cudaStream_t stream) {
  const int64_t chunks = a.K / 16, items = a.R * chunks;
  const dim3 grid((unsigned)((items + 255) / 256)), block(256);
  return a.f32 ? launch_pdl(&b128_dequant_kernel<true>, grid, block, 0, stream, a, chunks, items)
               : launch_pdl(&b128_dequant_kernel<false>, grid, block, 0, stream, a, chunks, items);
}

}  // namespace mxq
