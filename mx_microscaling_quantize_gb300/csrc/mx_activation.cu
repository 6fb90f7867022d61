// mx_activation.cu -- the (gated) activation whose output is an operand in 8 bits, and its gradient from
// the activation's input or from an 8-bit checkpoint of it.
//
//   u = [gate | up] (gated) or gate:  h = f(gate) up  or  f(gate);
//   d gate = dh up f'(gate), d up = dh f(gate)  or  d gate = dh f'(gate).
//   f: silu g s(g), s the logistic function, f' = s + g s (1 - s); gelu g Phi(g), f' = Phi + g phi;
//   its tanh form g s(2 z), z = sqrt(2 / pi) (g + 0.044715 g^3) (0.5 (1 + tanh z) is s(2 z)).
// All in fp32, rounded once: to codes under the scale of the block of 128 that they form, or to bf16.
//
// Bound by memory: u is read once, h and (asked for) its checkpoint are written by the same pass. A warp
// takes RW rows of 512 columns, a lane 16 of each, as in the quantisation of rows; eight lanes hold a
// block.
#include "mx_b128.cuh"
#include "mx_device.cuh"
#include "mx_launch.h"
#include "mx_train.h"
#include "mxq.h"

namespace mxq {

namespace {

constexpr int kActThreads = 256;
constexpr int kActCols = 512;  // columns of a warp's tile

__device__ __forceinline__ float rcp(float v) { return __fdividef(1.0f, v); }

// s(g) and 1 - s(g). exp(-g) beyond fp32 leaves 0 and 1 (kept from infinity times zero).
__device__ __forceinline__ void logistic(float g, float& s, float& one_minus) {
  const float e = __expf(-g);
  s = rcp(1.0f + e);
  one_minus = s * fminf(e, 3.402823466e38f);
}

template <int KIND>
__device__ __forceinline__ float act(float g) {
  if (KIND == MX_ACT_SILU) return g * rcp(1.0f + __expf(-g));
  if (KIND == MX_ACT_GELU) return g * 0.5f * erfcf(g * -0.70710678118654752f);
  const float z2 = 1.5957691216057308f * fmaf(0.044715f * g * g, g, g);
  return g * rcp(1.0f + __expf(-z2));
}

// f(g) and f'(g)
template <int KIND>
__device__ __forceinline__ void act_grad(float g, float& h, float& d) {
  if (KIND == MX_ACT_GELU) {
    const float p = 0.5f * erfcf(g * -0.70710678118654752f);
    h = g * p;
    d = fmaf(g * 0.39894228040143268f, __expf(-0.5f * g * g), p);
    return;
  }
  float s, q;
  if (KIND == MX_ACT_SILU) {
    logistic(g, s, q);
    h = g * s;
    d = fmaf(h, q, s);
  } else {
    const float g2 = 0.044715f * g * g;
    logistic(1.5957691216057308f * fmaf(g2, g, g), s, q);
    h = g * s;
    d = fmaf(h * q, 1.5957691216057308f * fmaf(3.0f, g2, 1.0f), s);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ void unpack(const uint32_t (&w)[8], float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

// Factors of the block that this lane's 16 values and those of its seven neighbours form.
__device__ __forceinline__ Factors block_of(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
  return block_factors_b128(m);
}

__device__ __forceinline__ void store_codes(const float (&v)[16], float r, uint8_t* to) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = codes2(__fmul_rn(v[4 * j], r), __fmul_rn(v[4 * j + 1], r)) |
           codes2(__fmul_rn(v[4 * j + 2], r), __fmul_rn(v[4 * j + 3], r)) << 16;
  }
  store16B(to, w);
}

// 16 codes times their scale, in fp32.
__device__ __forceinline__ void decode(const uint32_t* w, float s, float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    e4m3x2_to_f32(w[j] & 0xFFFFu, v[4 * j], v[4 * j + 1]);
    e4m3x2_to_f32(w[j] >> 16, v[4 * j + 2], v[4 * j + 3]);
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __fmul_rn(v[j], s);
}

template <int KIND, bool GATED, int RW>
__global__ void __launch_bounds__(kActThreads) activation_kernel(ActArgs a, int64_t col_tiles,
                                                                 int64_t tiles) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, sub = lane & 7, blk = lane >> 3;
  const int64_t tile = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (tile >= tiles) return;
  const int64_t r0 = tile / col_tiles * RW;
  const int64_t col = tile % col_tiles * kActCols + lane * 16, U = GATED ? 2 * a.H : a.H;
  const int64_t kb = col / kB128, up_blocks = a.H / kB128;
  const uint16_t* u = static_cast<const uint16_t*>(a.u);
  uint32_t g[RW][8], p[GATED ? RW : 1][8];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    if (r0 + i < a.R && col < a.H) {
      load32B(u + (r0 + i) * U + col, g[i]);
      if constexpr (GATED) load32B(u + (r0 + i) * U + a.H + col, p[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = 0u;
      if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[i][j] = 0u;
      }
    }
  }
  float mine = 0.0f, mine_g = 0.0f, mine_p = 0.0f;  // lane sub keeps the scales of row sub
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const bool there = r0 + i < a.R && col < a.H;
    float v[16], h[16];
    unpack(g[i], v);
    const int64_t at = (r0 + i) * U + col;
    if (a.u_codes) {
      const Factors f = block_of(absmax_f32x16(v));
      if (sub == i) mine_g = f.scale;
      if (there) store_codes(v, f.r, a.u_codes + at);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) h[j] = act<KIND>(v[j]);
    if constexpr (GATED) {
      unpack(p[i], v);
      if (a.u_codes) {
        const Factors f = block_of(absmax_f32x16(v));
        if (sub == i) mine_p = f.scale;
        if (there) store_codes(v, f.r, a.u_codes + at + a.H);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) h[j] *= v[j];
    }
    const Factors f = block_of(absmax_f32x16(h));
    if (sub == i) mine = f.scale;
    if (there) store_codes(h, f.r, a.codes + (r0 + i) * a.H + col);
  }
  if (sub < RW && r0 + sub < a.R && col - sub * 16 < a.H) {
    a.scales[kb * a.R + r0 + sub] = mine;
    if (a.u_codes) {
      a.u_scales_out[kb * a.R + r0 + sub] = mine_g;
      if constexpr (GATED) a.u_scales_out[(up_blocks + kb) * a.R + r0 + sub] = mine_p;
    }
  }
}

template <int KIND, bool GATED, bool CODES, int RW>
__global__ void __launch_bounds__(kActThreads) activation_backward_kernel(ActArgs a, int64_t col_tiles,
                                                                          int64_t tiles) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int64_t tile = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (tile >= tiles) return;
  const int64_t r0 = tile / col_tiles * RW;
  const int64_t col = tile % col_tiles * kActCols + lane * 16, U = GATED ? 2 * a.H : a.H;
  const int64_t kb = col / kB128, up_blocks = a.H / kB128;
  constexpr int kWords = CODES ? 4 : 8;
  uint32_t dh[RW][8], g[RW][kWords], p[GATED ? RW : 1][kWords];
  float gs[RW], ps[RW];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    gs[i] = ps[i] = 0.0f;
    if (r0 + i < a.R && col < a.H) {
      const int64_t at = (r0 + i) * U + col;
      if constexpr (CODES) {
        const uint8_t* u = static_cast<const uint8_t*>(a.u);
        load16B(u + at, g[i]);
        gs[i] = load_f32(a.u_scales + kb * a.R + r0 + i);
        if constexpr (GATED) {
          load16B(u + at + a.H, p[i]);
          ps[i] = load_f32(a.u_scales + (up_blocks + kb) * a.R + r0 + i);
        }
      } else {
        const uint16_t* u = static_cast<const uint16_t*>(a.u);
        load32B(u + at, g[i]);
        if constexpr (GATED) load32B(u + at + a.H, p[i]);
      }
      load32B(static_cast<const uint16_t*>(a.dh) + (r0 + i) * a.H + col, dh[i]);
    } else {
#pragma unroll
      for (int j = 0; j < kWords; ++j) g[i][j] = 0u;
      if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) p[i][j] = 0u;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) dh[i][j] = 0u;
    }
  }
  float mine_g = 0.0f, mine_p = 0.0f;
  auto put = [&](const float (&v)[16], int64_t at, bool there, float& mine, bool keep) {
    if (a.du && there) {
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
      store32B(static_cast<uint16_t*>(a.du) + at, o);
    }
    if (a.codes) {
      const Factors f = block_of(absmax_f32x16(v));
      if (keep) mine = f.scale;
      if (there) store_codes(v, f.r, a.codes + at);
    }
  };
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const bool there = r0 + i < a.R && col < a.H;
    const int64_t at = (r0 + i) * U + col;
    float v[16], d[16], e[16];
    if constexpr (CODES) {
      decode(g[i], gs[i], v);
    } else {
      unpack(g[i], v);
    }
    unpack(dh[i], e);
    if constexpr (GATED) {
      float up[16];
      if constexpr (CODES) {
        decode(p[i], ps[i], up);
      } else {
        unpack(p[i], up);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float h, der;
        act_grad<KIND>(v[j], h, der);
        d[j] = e[j] * up[j] * der;
        e[j] *= h;
      }
      put(e, at + a.H, there, mine_p, sub == i);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float h, der;
        act_grad<KIND>(v[j], h, der);
        d[j] = e[j] * der;
      }
    }
    put(d, at, there, mine_g, sub == i);
  }
  if (a.codes && sub < RW && r0 + sub < a.R && col - sub * 16 < a.H) {
    a.scales[kb * a.R + r0 + sub] = mine_g;
    if constexpr (GATED) a.scales[(up_blocks + kb) * a.R + r0 + sub] = mine_p;
  }
}

template <typename F>
cudaError_t by_kind(int kind, F&& f) {
  if (kind == MX_ACT_SILU) return f(std::integral_constant<int, MX_ACT_SILU>());
  if (kind == MX_ACT_GELU) return f(std::integral_constant<int, MX_ACT_GELU>());
  return f(std::integral_constant<int, MX_ACT_GELU_TANH>());
}

template <int RW, typename K>
cudaError_t run(K kernel, const ActArgs& a, int threads, cudaStream_t stream) {
  const int64_t col_tiles = (a.H + kActCols - 1) / kActCols, warps = threads / 32;
  const int64_t tiles = (a.R + RW - 1) / RW * col_tiles;
  return launch_pdl(kernel, dim3((unsigned)((tiles + warps - 1) / warps)), dim3(threads), 0, stream, a,
                    col_tiles, tiles);
}

}  // namespace

cudaError_t launch_activation(const ActArgs& a, cudaStream_t stream) {
  return by_kind(a.kind, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    return a.gated ? run<1>(&activation_kernel<KIND, true, 1>, a, kActThreads, stream)
                   : run<1>(&activation_kernel<KIND, false, 1>, a, kActThreads, stream);
  });
}

cudaError_t launch_activation_backward(const ActArgs& a, cudaStream_t stream) {
  return by_kind(a.kind, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    if (a.u_scales) {
      return a.gated ? run<1>(&activation_backward_kernel<KIND, true, true, 1>, a, kActThreads, stream)
                     : run<1>(&activation_backward_kernel<KIND, false, true, 1>, a, kActThreads, stream);
    }
    return a.gated ? run<1>(&activation_backward_kernel<KIND, true, false, 1>, a, kActThreads, stream)
                   : run<1>(&activation_backward_kernel<KIND, false, false, 1>, a, kActThreads, stream);
  });
}

}  // namespace mxq
