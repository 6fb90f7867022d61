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
// takes 512 columns of a row (1024 forward without a gate), a lane a run of 8 of each 256 in packed pairs; 16 lanes
// hold a block. CTAs of four warps, whose places on an SM are taken again as soon as these four are done, as many
// of them as their values' registers allow. 4096 x 28672 gated against its bytes at the rate of a plain copy: silu
// 89 us (88), with a checkpoint 127 (122), backward from it into bf16 and an operand 179 (178); with eight warps a
// CTA 96, 139 and 178, with two 115 (the rate at which CTAs start), 129 and 179. gelu 108, 142 and 190, bound by its
// instructions, 25 for a value and 40 backward; ungated gelu 80 (53).
#include "mx_b128.cuh"
#include "mx_device.cuh"
#include "mx_launch.h"
#include "mx_train.h"
#include "mxq.h"

namespace mxq {

namespace {

constexpr int kActThreads = 128;
// Runs of 8 columns per lane; a warp's tile has 256 times as many columns. Without a gate the forward pass has
// registers for twice as many (4096 x 28672 gelu 91 -> 80 us), the backward pass has not (bf16 102 -> 111).
template <bool GATED>
constexpr int kForwardRuns = GATED ? 2 : 4;
constexpr int kBackwardRuns = 2;

// The hardware's approximate exponential of two and reciprocal (relative 2^-22 and 2^-23; results below
// 2^-126 are 0).
__device__ __forceinline__ float exp2_fast(float v) {
  float d;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float d;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(d) : "f"(v));
  return d;
}
__device__ __forceinline__ uint64_t exp2_pair(uint64_t v) { return pair(exp2_fast(lo_of(v)), exp2_fast(hi_of(v))); }
__device__ __forceinline__ uint64_t rcp_pair(uint64_t v) { return pair(rcp_fast(lo_of(v)), rcp_fast(hi_of(v))); }
__device__ __forceinline__ uint64_t scaled(uint64_t v, float s) { return mul_pair(v, pair(s)); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhGain = 1.5957691216057308f;  // 2 sqrt(2 / pi)

// Phi(g), and e = exp(-g^2 / 2). The tail Phi(-|g|) is e t Q(t), t = 1 / (1 + 0.38 |g| / sqrt 2): Mills'
// ratio, smooth in t, by a polynomial fitted (least squares at Chebyshev nodes, reweighted towards the
// smallest largest error), relative 4.5e-8 at worst with these coefficients. In fp32 Phi(-|g|) is off by 4e-7 up to
// |g| = 1, and, for the roundings of the exponential's argument, g^2 / 2 log2 e, by 1e-6 at 4, 2e-6 at 6, 5e-6 at 10
// and 8e-6 at 12.9; Phi(|g|) by 4e-7. Beside the exponential and the reciprocal it takes 9 FMAs, and the exponential
// is the gradient's too.
__device__ __forceinline__ uint64_t normal_cdf(uint64_t g, uint64_t& e) {
  e = exp2_pair(mul_pair(scaled(g, -0.5f * kLog2e), g));
  const uint64_t t = rcp_pair(fma_pair(pair(0.26870056986808777f), pair(fabsf(lo_of(g)), fabsf(hi_of(g))), pair(1.0f)));
  uint64_t p = pair(0.029425911605358124f);
  p = fma_pair(p, t, pair(-0.13084791600704193f));
  p = fma_pair(p, t, pair(0.18129514157772064f));
  p = fma_pair(p, t, pair(-0.07996146380901337f));
  p = fma_pair(p, t, pair(0.1144489124417305f));
  p = fma_pair(p, t, pair(0.06958147138357162f));
  p = fma_pair(p, t, pair(0.10188283026218414f));
  p = fma_pair(p, t, pair(0.10697033256292343f));
  p = fma_pair(p, t, pair(0.10720480233430862f));
  const uint64_t tail = mul_pair(mul_pair(p, t), e);
  const uint64_t rest = fma_pair(tail, pair(-1.0f), pair(1.0f));
  return pair(lo_of(g) < 0.0f ? lo_of(tail) : lo_of(rest), hi_of(g) < 0.0f ? hi_of(tail) : hi_of(rest));
}

// The logistic function of z, from -z log2 e: 0 below exp(-88), where its value is under 2^-126.
__device__ __forceinline__ uint64_t logistic(uint64_t z) {
  return rcp_pair(add_pair(exp2_pair(z), pair(1.0f)));
}

// f(g) of a pair, and with GRAD its derivative d.
template <int KIND, bool GRAD>
__device__ __forceinline__ uint64_t act(uint64_t g, uint64_t& d) {
  uint64_t s, h;
  if constexpr (KIND == MX_ACT_GELU) {
    uint64_t e;
    s = normal_cdf(g, e);
    h = mul_pair(g, s);
    if constexpr (GRAD) d = fma_pair(scaled(g, 0.39894228040143268f), e, s);
    return h;
  }
  if constexpr (KIND == MX_ACT_SILU) {
    s = logistic(scaled(g, -kLog2e));
    h = mul_pair(g, s);
    if constexpr (GRAD) d = fma_pair(h, fma_pair(s, pair(-1.0f), pair(1.0f)), s);
    return h;
  }
  const uint64_t g2 = mul_pair(scaled(g, 0.044715f), g);
  s = logistic(mul_pair(scaled(g, -kLog2e * kTanhGain), add_pair(g2, pair(1.0f))));
  h = mul_pair(g, s);
  if constexpr (GRAD) {
    const uint64_t q = mul_pair(h, fma_pair(s, pair(-1.0f), pair(1.0f)));  // h (1 - s)
    // (bounded: where g^2 overflows q is 0)
    const uint64_t some = pair(fminf(lo_of(g2), 1e30f), fminf(hi_of(g2), 1e30f));
    d = fma_pair(q, scaled(fma_pair(some, pair(3.0f), pair(1.0f)), kTanhGain), s);
  }
  return h;
}

// What a warp's tile is of: a row, and a lane's runs of 8 columns of it. A CTA has 2^across warps side by side
// on a row and the others on rows below (no quotient of indexes: a 64-bit one takes a fifth of the instructions
// of a tile).
struct ActTile {
  int64_t row, R;
  int H, U, col0, lane;  // columns of h and of u, first column of the lane's runs
  __device__ __forceinline__ int column(int p) const { return col0 + p * 256; }
  __device__ __forceinline__ bool has(int p) const { return column(p) < H; }
};
template <int RUNS, bool GATED>
__device__ __forceinline__ bool act_tile(const ActArgs& a, int across, ActTile& t) {
  constexpr int kWarps = kActThreads / 32;
  const int warp = threadIdx.x >> 5;
  t.lane = threadIdx.x & 31;
  t.row = (int64_t)blockIdx.x * (kWarps >> across) + (warp >> across);
  const int tile = ((int)(blockIdx.y + gridDim.y * blockIdx.z) << across) + (warp & ((1 << across) - 1));
  t.col0 = tile * (RUNS * 256) + t.lane * 8;
  t.H = (int)a.H;
  t.U = GATED ? 2 * t.H : t.H;
  t.R = a.R;
  return t.row < t.R && t.col0 - t.lane * 8 < t.H;
}

// N runs (RUNS of each of N / RUNS parts of rows of `width` columns, a part H columns) as codes and scales.
template <int RUNS, int N>
__device__ __forceinline__ void store_runs(const uint64_t (&v)[N][4], const ActTile& t, int width,
                                           uint8_t* codes, float* scales) {
  uint8_t* to = codes + t.row * width;
  run_codes<N>(
      v, t.lane,
      [&](int n, uint32_t lo, uint32_t hi) {
        const int p = n % RUNS;
        if (t.has(p)) store8B(to + (n / RUNS) * t.H + t.column(p), lo, hi);
      },
      [&](int n, float s) {
        const int p = n % RUNS;
        const int kb = ((n / RUNS) * t.H + t.column(p)) / kB128;
        if ((t.column(p) & ~(kB128 - 1)) < t.H) scales[kb * t.R + t.row] = s;
      });
}

// A lane's runs of `part` (0: gate, 1: up) of its row of u, bf16 or codes, or of dh.
template <bool CODES, int RUNS>
struct ActRuns {
  uint32_t raw[RUNS][CODES ? 2 : 4];
  float scale[RUNS];

  __device__ __forceinline__ void load(const void* u, const float* scales, const ActTile& t, int width,
                                       int part) {
#pragma unroll
    for (int p = 0; p < RUNS; ++p) {
      scale[p] = 0.0f;
#pragma unroll
      for (int j = 0; j < (CODES ? 2 : 4); ++j) raw[p][j] = 0u;
      if (!t.has(p)) continue;
      const int col = part * t.H + t.column(p);
      if constexpr (CODES) {
        asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];"
                     : "=r"(raw[p][0]), "=r"(raw[p][1])
                     : "l"(static_cast<const uint8_t*>(u) + t.row * width + col));
        scale[p] = load_f32(scales + col / kB128 * t.R + t.row);
      } else {
        load16B(static_cast<const uint16_t*>(u) + t.row * width + col, raw[p]);
      }
    }
  }
  __device__ __forceinline__ void values(int p, uint64_t (&v)[4]) const {
    if constexpr (CODES) {
      values4(raw[p][0], v[0], v[1]);
      values4(raw[p][1], v[2], v[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = mul_pair(v[j], pair(scale[p]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = bf16_pair(raw[p][j]);
    }
  }
};

template <int KIND, bool GATED>
__global__ void __launch_bounds__(kActThreads, GATED ? 9 : 8) activation_kernel(ActArgs a, int across) {
  constexpr int kParts = GATED ? 2 : 1, kRuns = kForwardRuns<GATED>;
  pdl_launch_dependents();
  pdl_wait();
  ActTile t;
  if (!act_tile<kRuns, GATED>(a, across, t)) return;
  ActRuns<false, kRuns> in[kParts];
#pragma unroll
  for (int k = 0; k < kParts; ++k) in[k].load(a.u, nullptr, t, t.U, k);
  uint64_t u[kParts * kRuns][4], h[kRuns][4];
#pragma unroll
  for (int n = 0; n < kParts * kRuns; ++n) in[n / kRuns].values(n % kRuns, u[n]);
  if (a.u_codes) store_runs<kRuns, kParts * kRuns>(u, t, t.U, a.u_codes, a.u_scales_out);
#pragma unroll
  for (int p = 0; p < kRuns; ++p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint64_t none;
      h[p][j] = act<KIND, false>(u[p][j], none);
      if constexpr (GATED) h[p][j] = mul_pair(h[p][j], u[kRuns + p][j]);
    }
  }
  store_runs<kRuns, kRuns>(h, t, a.H, a.codes, a.scales);
}

template <int KIND, bool GATED, bool CODES>
__global__ void __launch_bounds__(kActThreads, GATED ? 8 : 9) activation_backward_kernel(ActArgs a, int across) {
  constexpr int kParts = GATED ? 2 : 1, kRuns = kBackwardRuns;
  pdl_launch_dependents();
  pdl_wait();
  ActTile t;
  if (!act_tile<kRuns, GATED>(a, across, t)) return;
  ActRuns<CODES, kRuns> in[kParts];
  ActRuns<false, kRuns> dh;
#pragma unroll
  for (int k = 0; k < kParts; ++k) in[k].load(a.u, a.u_scales, t, t.U, k);
  dh.load(a.dh, nullptr, t, a.H, 0);
  uint64_t du[kParts * kRuns][4];
#pragma unroll
  for (int p = 0; p < kRuns; ++p) {
    uint64_t g[4], up[4], e[4];
    in[0].values(p, g);
    if constexpr (GATED) in[kParts - 1].values(p, up);
    dh.values(p, e);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint64_t d;
      const uint64_t h = act<KIND, true>(g[j], d);
      if constexpr (GATED) {
        du[kRuns + p][j] = mul_pair(e[j], h);
        du[p][j] = mul_pair(mul_pair(e[j], up[j]), d);
      } else {
        du[p][j] = mul_pair(e[j], d);
      }
    }
  }
  if (a.du) {
#pragma unroll
    for (int n = 0; n < kParts * kRuns; ++n) {
      if (!t.has(n % kRuns)) continue;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = bf16_word(du[n][j]);
      store16B(static_cast<uint16_t*>(a.du) + t.row * t.U + (n / kRuns) * a.H + t.column(n % kRuns), o);
    }
  }
  if (a.codes) store_runs<kRuns, kParts * kRuns>(du, t, t.U, a.codes, a.scales);
}

template <typename F>
cudaError_t by_kind(int kind, F&& f) {
  if (kind == MX_ACT_SILU) return f(std::integral_constant<int, MX_ACT_SILU>());
  if (kind == MX_ACT_GELU) return f(std::integral_constant<int, MX_ACT_GELU>());
  return f(std::integral_constant<int, MX_ACT_GELU_TANH>());
}

cudaError_t run(void (*kernel)(ActArgs, int), int runs, const ActArgs& a, cudaStream_t stream) {
  const int cols = runs * 256;
  const int64_t col_tiles = (a.H + cols - 1) / cols;
  constexpr int kWarps = kActThreads / 32;
  int across = 0;
  while ((1 << across) < kWarps && (1 << across) < col_tiles) ++across;
  const int rows = kWarps >> across;
  // columns over y and, where those are too many, z
  const int64_t n = (col_tiles + (1 << across) - 1) >> across, z = (n + 65534) / 65535;
  const dim3 grid((unsigned)((a.R + rows - 1) / rows), (unsigned)((n + z - 1) / z), (unsigned)z);
  return launch_pdl(kernel, grid, dim3(kActThreads), 0, stream, a, across);
}

}  // namespace

cudaError_t launch_activation(const ActArgs& a, cudaStream_t stream) {
  return by_kind(a.kind, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    return a.gated ? run(&activation_kernel<KIND, true>, kForwardRuns<true>, a, stream)
                   : run(&activation_kernel<KIND, false>, kForwardRuns<false>, a, stream);
  });
}

cudaError_t launch_activation_backward(const ActArgs& a, cudaStream_t stream) {
  return by_kind(a.kind, [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    if (a.u_scales) {
      return run(a.gated ? &activation_backward_kernel<KIND, true, true>
                         : &activation_backward_kernel<KIND, false, true>, kBackwardRuns, a, stream);
    }
    return run(a.gated ? &activation_backward_kernel<KIND, true, false>
                       : &activation_backward_kernel<KIND, false, false>, kBackwardRuns, a, stream);
  });
}

}  // namespace mxq
