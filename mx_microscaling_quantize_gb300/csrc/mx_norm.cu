// mx_norm.cu -- layer norm, its gradients, and its output as an operand in 8 bits.
//
//   mean = sum x / K (0 where not centred), rstd = 1 / sqrt(sum (x - mean)^2 / K + eps),
//   y = (x - mean) rstd w + b;
//   backward, with xhat = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum g / K - xhat sum(g xhat) / K)   (without the second term where not centred),
//   dw = sum over rows of dy xhat, db = sum over rows of dy.
//
// A row lives in the registers of a group of warps and is read once. Its variance is that of the
// differences from the mean (each warp's own mean and squares, joined by the counts), so a large mean
// costs no digits. All sums are in fp32 in a fixed order.
#include "mx_b128.cuh"
#include "mx_device.cuh"
#include "mx_launch.h"
#include "mx_train.h"

namespace mxq {

namespace {

constexpr int kForwardWarps = 8;  // of a CTA, and of a group that holds one row
constexpr int kMaxWarps = 16;     // the same of the backward pass
constexpr int kRingBytes = 200 * 1024;
constexpr int kMaxParts = 304;  // of the weight's gradient: rows are split over at most so many CTAs

// Barrier of one group of warps (ids 1 ..; a group of one warp needs none beyond its own order).
__device__ __forceinline__ void group_sync(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
  return v;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ float load_as_f32(const void* p, bool f32, int64_t i) {
  return f32 ? load_f32(static_cast<const float*>(p) + i)
             : __uint_as_float(load_u16(static_cast<const uint16_t*>(p) + i) << 16);
}

__device__ __forceinline__ void store_from_f32(void* p, bool f32, int64_t i, float v) {
  if (f32) {
    static_cast<float*>(p)[i] = v;
  } else {
    static_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16(v, 0.0f);
  }
}

// N consecutive values of a weight or a bias (aligned to 16 bytes), kept in L1 for the next rows.
template <int N>
__device__ __forceinline__ void load_param(const void* p, bool f32, int64_t i, float* v) {
  if (f32) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const uint4 q = load_v4(static_cast<const float*>(p) + i + j);
      v[j] = __uint_as_float(q.x);
      v[j + 1] = __uint_as_float(q.y);
      v[j + 2] = __uint_as_float(q.z);
      v[j + 3] = __uint_as_float(q.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; j += 8) {
      const uint4 q = load_v4(static_cast<const uint16_t*>(p) + i + j);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[j + 2 * k] = bf16_lo(w[k]);
        v[j + 2 * k + 1] = bf16_hi(w[k]);
      }
    }
  }
}

// ------------------------------------------------------------------------------------------
// forward
// ------------------------------------------------------------------------------------------
// C chunks of 16 values per lane: with VEC a lane's chunk is 16 consecutive columns (32-byte loads),
// else its columns are the group's width apart, for rows of any length and alignment.
template <bool XF32, int C, bool VEC, bool QUANT>
struct NormRow {
  static constexpr int kWords = C * (XF32 || !VEC ? 16 : 8);
  uint32_t raw[kWords];

  __device__ __forceinline__ void load(const NormArgs& a, int64_t row, int t, int T) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (VEC) {
        const int64_t col = (int64_t)(c * T + t) * 16;
        if (col < a.K) {
          const char* p = static_cast<const char*>(a.x) + (row * a.K + col) * (XF32 ? 4 : 2);
          load32B(p, raw + c * (XF32 ? 16 : 8));
          if constexpr (XF32) load32B(p + 32, raw + c * 16 + 8);
        } else {
#pragma unroll
          for (int j = 0; j < (XF32 ? 16 : 8); ++j) raw[c * (XF32 ? 16 : 8) + j] = 0u;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int64_t col = (int64_t)(c * 16 + j) * T + t;
          raw[c * 16 + j] = col < a.K ? __float_as_uint(load_as_f32(a.x, XF32, row * a.K + col)) : 0u;
        }
      }
    }
  }
  __device__ __forceinline__ void values(float (&v)[16 * C]) const {
    if constexpr (XF32 || !VEC) {
#pragma unroll
      for (int i = 0; i < 16 * C; ++i) v[i] = __uint_as_float(raw[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8 * C; ++i) {
        v[2 * i] = bf16_lo(raw[i]);
        v[2 * i + 1] = bf16_hi(raw[i]);
      }
    }
  }
};

// 16 values of one row's block (eight lanes hold a block) as codes and a scale.
__device__ __forceinline__ void store_block_codes(const float* v, uint8_t* codes, float* scales, int64_t M,
                                                  int64_t K, int64_t row, int64_t col) {
  uint32_t m = absmax_f32x16(v);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
  if (col >= K) return;
  const Factors f = block_factors_b128(m);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = codes2(__fmul_rn(v[4 * j], f.r), __fmul_rn(v[4 * j + 1], f.r)) |
           codes2(__fmul_rn(v[4 * j + 2], f.r), __fmul_rn(v[4 * j + 3], f.r)) << 16;
  }
  store16B(codes + row * K + col, w);
  if ((col & (kB128 - 1)) == 0) scales[col / kB128 * M + row] = f.scale;
}

template <bool XF32, int C, bool VEC, bool QUANT>
__global__ void __launch_bounds__(32 * kForwardWarps) norm_kernel(NormArgs a, int W) {
  __shared__ float2 part[2][kForwardWarps];  // a warp's mean and sum of squared differences from it
  __shared__ float count[kForwardWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int T = 32 * W, group = threadIdx.x / T, t = threadIdx.x - group * T;
  const int lane = threadIdx.x & 31, w0 = group * W, wi = t >> 5;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / T);
  int64_t row = (int64_t)blockIdx.x * (blockDim.x / T) + group;
  int mine = 0;  // columns of this lane
#pragma unroll
  for (int i = 0; i < 16 * C; ++i) {
    mine += (VEC ? (int64_t)((i / 16) * T + t) * 16 + i % 16 : (int64_t)i * T + t) < a.K;
  }
  const float n = (float)__reduce_add_sync(0xFFFFFFFFu, (unsigned)mine);
  if (lane == 0) count[w0 + wi] = n;
  if (W > 1) group_sync(group, T);
  const float per_n = n > 0.0f ? __fdiv_rn(1.0f, n) : 0.0f, per_k = __fdiv_rn(1.0f, (float)a.K);
  NormRow<XF32, C, VEC, QUANT> next;
  if (row < a.M) next.load(a, row, t, T);
  for (int slot = 0; row < a.M; row += step, slot ^= 1) {
    float v[16 * C];
    next.values(v);
    if (row + step < a.M) next.load(a, row + step, t, T);
    float mean = 0.0f;
    if (a.center) {
      float s[4] = {};
#pragma unroll
      for (int i = 0; i < 16 * C; ++i) s[i & 3] += v[i];
      mean = warp_sum((s[0] + s[1]) + (s[2] + s[3])) * per_n;
    }
    float s[4] = {};
#pragma unroll
    for (int i = 0; i < 16 * C; ++i) {
      const bool there = (VEC ? (int64_t)((i / 16) * T + t) * 16 : (int64_t)i * T + t) < a.K;
      const float d = there ? v[i] - mean : 0.0f;
      s[i & 3] = fmaf(d, d, s[i & 3]);
    }
    float sq = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (W > 1) {
      if (lane == 0) part[slot][w0 + wi] = make_float2(mean, sq);
      group_sync(group, T);
      float total = 0.0f, m = 0.0f;
      if (a.center) {
        for (int i = 0; i < W; ++i) m = fmaf(part[slot][w0 + i].x, count[w0 + i], m);
        m *= per_k;
      }
      for (int i = 0; i < W; ++i) {
        const float2 p = part[slot][w0 + i];
        total += fmaf((p.x - m) * count[w0 + i], p.x - m, p.y);
      }
      mean = m;
      sq = total;
    }
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(sq, per_k, a.eps)));
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (VEC) {
        const int64_t col = (int64_t)(c * T + t) * 16;
        if constexpr (QUANT) {
          if (a.x_codes) store_block_codes(v + 16 * c, a.x_codes, a.x_scales_out, a.M, a.K, row, col);
        }
        float y[16];
        if (col < a.K) {
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = (v[16 * c + j] - mean) * rstd;
          float p[16];
          if (a.weight) {
            load_param<16>(a.weight, a.w_type == kTypeFp32, col, p);
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] *= p[j];
          }
          if (a.bias) {
            load_param<16>(a.bias, a.w_type == kTypeFp32, col, p);
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] += p[j];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = 0.0f;
        }
        if constexpr (QUANT) {
          store_block_codes(y, a.codes, a.scales, a.M, a.K, row, col);
        } else if (col < a.K) {
          uint32_t o[8];
          if (a.y_type == kTypeFp32) {
            float* to = static_cast<float*>(a.y) + row * a.K + col;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(y[8 * h + j]);
              store32B(to + 8 * h, o);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = pack_bf16(y[2 * j], y[2 * j + 1]);
            store32B(static_cast<uint16_t*>(a.y) + row * a.K + col, o);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int64_t col = (int64_t)(c * 16 + j) * T + t;
          if (col >= a.K) continue;
          float y = (v[16 * c + j] - mean) * rstd;
          if (a.weight) y *= load_as_f32(a.weight, a.w_type == kTypeFp32, col);
          if (a.bias) y += load_as_f32(a.bias, a.w_type == kTypeFp32, col);
          store_from_f32(a.y, a.y_type == kTypeFp32, row * a.K + col, y);
        }
      }
    }
  }
}

// ------------------------------------------------------------------------------------------
// backward
// ------------------------------------------------------------------------------------------
// Gradient of the input, and each CTA's share of the parameters' gradients, which norm_reduce_kernel
// adds up. C chunks of 8 values per lane. With VEC a thread's pieces of the next rows are on their way
// into places of its own in shared memory (cp.async: no barrier); without, values are loaded one by one.
struct NormRing {
  int stages, bytes;             // of shared memory
  int x_piece, x_pieces;         // bytes of a copy of x and copies per chunk
  int dy_at, dy_pieces, scale_at;  // within a stage
};

__device__ __forceinline__ void copy_async(uint32_t to, const void* from, int bytes) {
  if (bytes == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  } else if (bytes == 8) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
  }
}

template <int C, bool VEC, int XT>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) norm_backward_kernel(NormArgs a, int W, NormRing r) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 part[2][kMaxWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int threads = blockDim.x, T = 32 * W, group = threadIdx.x / T, t = threadIdx.x - group * T;
  const int lane = threadIdx.x & 31, w0 = group * W, wi = t >> 5, tid = threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * (threads / T);
  int64_t row = (int64_t)blockIdx.x * (threads / T) + group;
  const bool dy_f32 = a.y_type == kTypeFp32, dx_f32 = a.dx_type == kTypeFp32;
  const float per_k = __fdiv_rn(1.0f, (float)a.K);
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring);

  auto column = [&](int c, int j) -> int64_t {
    return VEC ? (int64_t)(c * T + t) * 8 + j : (int64_t)(c * 8 + j) * T + t;
  };
  auto request = [&](int64_t at, int stage) {  // VEC: this thread's pieces of a row
    if (at < a.M) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t col = column(c, 0);
        if (col >= a.K) break;
        const uint32_t to = base + stage * r.bytes;
        const char* x = static_cast<const char*>(a.x) + (at * a.K + col) * (r.x_piece * r.x_pieces / 8);
        for (int p = 0; p < r.x_pieces; ++p) {
          copy_async(to + ((c * r.x_pieces + p) * threads + tid) * r.x_piece, x + p * r.x_piece, r.x_piece);
        }
        const char* dy = static_cast<const char*>(a.y) + (at * a.K + col) * (2 * r.dy_pieces);
        for (int p = 0; p < r.dy_pieces; ++p) {
          copy_async(to + r.dy_at + ((c * r.dy_pieces + p) * threads + tid) * 16, dy + p * 16, 16);
        }
        if (XT == kTypeB128) {
          copy_async(to + r.scale_at + (c * threads + tid) * 4, a.x_scales + col / kB128 * a.M + at, 4);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  float w[8 * C], dw[8 * C], db[8 * C];
#pragma unroll
  for (int i = 0; i < 8 * C; ++i) {
    const int64_t col = column(i / 8, i % 8);
    w[i] = a.weight && col < a.K ? load_as_f32(a.weight, a.w_type == kTypeFp32, col) : 1.0f;
    dw[i] = db[i] = 0.0f;
  }
  if constexpr (VEC) {
    for (int s = 0; s < r.stages; ++s) request(row + s * step, s);
  }
  float mean_next = 0.0f, rstd_next = 0.0f;
  if (row < a.M) {
    rstd_next = load_f32(a.rstd + row);
    if (a.mean) mean_next = load_f32(a.mean + row);
  }
  int stage = 0;
  for (int slot = 0; row < a.M; row += step, slot ^= 1) {
    const float mean = mean_next, rstd = rstd_next;
    if (row + step < a.M) {
      rstd_next = load_f32(a.rstd + row + step);
      if (a.mean) mean_next = load_f32(a.mean + row + step);
    }
    float xh[8 * C], g[8 * C];
    if constexpr (VEC) {
      if (r.stages == 4) {
        asm volatile("cp.async.wait_group 3;" ::: "memory");
      } else if (r.stages == 2) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (VEC) {
        if (column(c, 0) < a.K) {
          const uint8_t* at = ring + stage * r.bytes;
          if (XT == kTypeBf16) {
            const uint4 q = reinterpret_cast<const uint4*>(at)[c * threads + tid];
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              xh[8 * c + 2 * j] = bf16_lo(u[j]);
              xh[8 * c + 2 * j + 1] = bf16_hi(u[j]);
            }
          } else if (XT == kTypeFp32) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const float4 q = reinterpret_cast<const float4*>(at)[(2 * c + p) * threads + tid];
              xh[8 * c + 4 * p] = q.x;
              xh[8 * c + 4 * p + 1] = q.y;
              xh[8 * c + 4 * p + 2] = q.z;
              xh[8 * c + 4 * p + 3] = q.w;
            }
          } else {
            const uint2 q = reinterpret_cast<const uint2*>(at)[c * threads + tid];
            const float s = reinterpret_cast<const float*>(at + r.scale_at)[c * threads + tid];
            const uint32_t u[2] = {q.x, q.y};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              e4m3x2_to_f32(u[j] & 0xFFFFu, xh[8 * c + 4 * j], xh[8 * c + 4 * j + 1]);
              e4m3x2_to_f32(u[j] >> 16, xh[8 * c + 4 * j + 2], xh[8 * c + 4 * j + 3]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) xh[8 * c + j] = __fmul_rn(xh[8 * c + j], s);
          }
          if (dy_f32) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const float4 q = reinterpret_cast<const float4*>(at + r.dy_at)[(2 * c + p) * threads + tid];
              g[8 * c + 4 * p] = q.x;
              g[8 * c + 4 * p + 1] = q.y;
              g[8 * c + 4 * p + 2] = q.z;
              g[8 * c + 4 * p + 3] = q.w;
            }
          } else {
            const uint4 q = reinterpret_cast<const uint4*>(at + r.dy_at)[c * threads + tid];
            const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              g[8 * c + 2 * j] = bf16_lo(u[j]);
              g[8 * c + 2 * j + 1] = bf16_hi(u[j]);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            xh[8 * c + j] = mean;  // xhat 0
            g[8 * c + j] = 0.0f;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t col = column(c, j), i = row * a.K + col;
          xh[8 * c + j] = mean;
          g[8 * c + j] = 0.0f;
          if (col >= a.K) continue;
          if (XT == kTypeB128) {
            float lo, hi;
            e4m3x2_to_f32(load_u8(static_cast<const uint8_t*>(a.x) + i), lo, hi);
            xh[8 * c + j] = __fmul_rn(lo, load_f32(a.x_scales + col / kB128 * a.M + row));
          } else {
            xh[8 * c + j] = load_as_f32(a.x, XT == kTypeFp32, i);
          }
          g[8 * c + j] = load_as_f32(a.y, dy_f32, i);
        }
      }
    }
    if constexpr (VEC) {  // into the places just read, by this thread alone
      request(row + r.stages * step, stage);
      stage = stage + 1 == r.stages ? 0 : stage + 1;
    }
    float c1[2] = {}, c2[2] = {};
#pragma unroll
    for (int i = 0; i < 8 * C; ++i) {
      xh[i] = (xh[i] - mean) * rstd;
      dw[i] = fmaf(g[i], xh[i], dw[i]);
      db[i] += g[i];
      g[i] *= w[i];
      c1[i & 1] += g[i];
      c2[i & 1] = fmaf(g[i], xh[i], c2[i & 1]);
    }
    float s1 = warp_sum(c1[0] + c1[1]), s2 = warp_sum(c2[0] + c2[1]);
    if (W > 1) {
      if (lane == 0) part[slot][w0 + wi] = make_float2(s1, s2);
      group_sync(group, T);
      s1 = s2 = 0.0f;
      for (int i = 0; i < W; ++i) {
        const float2 p = part[slot][w0 + i];
        s1 += p.x;
        s2 += p.y;
      }
    }
    s1 = a.mean ? s1 * per_k : 0.0f;
    s2 *= per_k;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (VEC) {
        const int64_t col = column(c, 0);
        if (col >= a.K) continue;
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = (g[8 * c + j] - s1 - xh[8 * c + j] * s2) * rstd;
        if (dx_f32) {
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(d[j]);
          float* to = static_cast<float*>(a.dx) + row * a.K + col;
          store16B(to, o);
          store16B(to + 4, o + 4);
        } else {
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = pack_bf16(d[2 * j], d[2 * j + 1]);
          store16B(static_cast<uint16_t*>(a.dx) + row * a.K + col, o);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t col = column(c, j);
          if (col >= a.K) continue;
          store_from_f32(a.dx, dx_f32, row * a.K + col,
                         (g[8 * c + j] - s1 - xh[8 * c + j] * s2) * rstd);
        }
      }
    }
  }
  if (!a.dweight && !a.dbias) return;
  // The groups' shares, joined in their order through shared memory, the first gradient after the other.
  const int groups = threads / T;
  float* out = a.workspace + (int64_t)blockIdx.x * a.K;
  const int64_t whole = (int64_t)gridDim.x * a.K;
  if constexpr (VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");
  float* sm = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!(k ? a.dbias : a.dweight)) continue;
    if (groups > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8 * C; ++i) {
        const int64_t col = column(i / 8, i % 8);
        if (col < a.K) sm[group * a.K + col] = k ? db[i] : dw[i];
      }
      __syncthreads();
      for (int64_t col = tid; col < a.K; col += threads) {
        float s = 0.0f;
        for (int i = 0; i < groups; ++i) s += sm[i * a.K + col];
        out[k * whole + col] = s;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8 * C; ++i) {
        const int64_t col = column(i / 8, i % 8);
        if (col < a.K) out[k * whole + col] = k ? db[i] : dw[i];
      }
    }
  }
}

// Adds up the CTAs' shares of a parameter's gradient (blockIdx.y: which): 32 columns a CTA, the shares
// over 16 warps.
__global__ void __launch_bounds__(512) norm_reduce_kernel(NormArgs a, int parts) {
  __shared__ float sum[16][33];
  pdl_launch_dependents();
  pdl_wait();
  float* to = blockIdx.y ? a.dbias : a.dweight;
  if (!to) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  const float* from = a.workspace + (int64_t)blockIdx.y * parts * a.K;
  float s = 0.0f;
  if (col < a.K) {
#pragma unroll 4
    for (int p = warp; p < parts; p += 16) s += load_f32(from + p * a.K + col);
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < a.K) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sum[i][lane];
    to[col] = s;
  }
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <bool XF32, int C, bool VEC, bool QUANT>
cudaError_t run_norm(const NormArgs& a, int W, int G, cudaStream_t stream) {
  const auto kernel = &norm_kernel<XF32, C, VEC, QUANT>;
  const int threads = 32 * W * G;
  const int64_t slots = resident_ctas(reinterpret_cast<const void*>(kernel), threads, 0, 0);
  if (slots <= 0) return cudaErrorInvalidConfiguration;
  const int64_t ctas = (a.M + G - 1) / G;
  return launch_pdl(kernel, dim3((unsigned)(ctas < slots ? ctas : slots)), dim3(threads), 0, stream, a, W);
}

template <bool XF32, int C>
cudaError_t pick_norm(const NormArgs& a, int W, int G, bool vec, cudaStream_t stream) {
  if (a.codes) return run_norm<XF32, C, true, true>(a, W, G, stream);
  if (vec) return run_norm<XF32, C, true, false>(a, W, G, stream);
  return run_norm<XF32, C, false, false>(a, W, G, stream);
}

template <int C, bool VEC, int XT>
cudaError_t run_backward(const NormArgs& a, int W, int G, cudaStream_t stream) {
  const auto kernel = &norm_backward_kernel<C, VEC, XT>;
  const int threads = 32 * W * G;
  NormRing r{};
  if (VEC) {
    r.x_piece = XT == kTypeB128 ? 8 : 16;
    r.x_pieces = XT == kTypeFp32 ? 2 : 1;
    r.dy_pieces = a.y_type == kTypeFp32 ? 2 : 1;
    r.dy_at = C * threads * r.x_piece * r.x_pieces;
    r.scale_at = r.dy_at + C * threads * 16 * r.dy_pieces;
    r.bytes = r.scale_at + (XT == kTypeB128 ? C * threads * 4 : 0);
    r.stages = r.bytes * 4 <= kRingBytes ? 4 : r.bytes * 2 <= kRingBytes ? 2 : 1;
  }
  const bool params = a.dweight || a.dbias;
  size_t smem = (size_t)r.stages * r.bytes;
  if (params && G > 1 && smem < (size_t)G * a.K * 4) smem = (size_t)G * a.K * 4;
  const int64_t slots = resident_ctas(reinterpret_cast<const void*>(kernel), threads, smem, 0);
  if (slots <= 0) return cudaErrorInvalidConfiguration;
  int64_t ctas = (a.M + G - 1) / G;
  if (ctas > slots) ctas = slots;
  if (params && ctas > kMaxParts) ctas = kMaxParts;
  const cudaError_t err =
      launch_pdl(kernel, dim3((unsigned)ctas), dim3(threads), smem, stream, a, W, r);
  if (err != cudaSuccess || !params) return err;
  return launch_pdl(&norm_reduce_kernel, dim3((unsigned)((a.K + 31) / 32), 2), dim3(512), 0, stream, a,
                    (int)ctas);
}

template <int C, bool VEC>
cudaError_t pick_backward(const NormArgs& a, int W, int G, cudaStream_t stream) {
  if (a.x_type == kTypeBf16) return run_backward<C, VEC, kTypeBf16>(a, W, G, stream);
  if (a.x_type == kTypeFp32) return run_backward<C, VEC, kTypeFp32>(a, W, G, stream);
  return run_backward<C, VEC, kTypeB128>(a, W, G, stream);
}

}  // namespace

int64_t norm_workspace_floats(int64_t M, int64_t K) { return 2 * (M < kMaxParts ? M : kMaxParts) * K; }

cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
  const bool vec = a.codes || (a.K % 16 == 0 && aligned_to(a.x, 32) && aligned_to(a.y, 32) &&
                               aligned_to(a.weight, 16) && aligned_to(a.bias, 16));
  const int C = a.K <= kForwardWarps * 1024 ? 2 : 4;
  const int W = (int)((a.K + 512 * C - 1) / (512 * C));
  const int G = kForwardWarps / W;
  if (a.x_type == kTypeFp32) {
    return C == 2 ? pick_norm<true, 2>(a, W, G, vec, stream) : pick_norm<true, 4>(a, W, G, vec, stream);
  }
  return C == 2 ? pick_norm<false, 2>(a, W, G, vec, stream) : pick_norm<false, 4>(a, W, G, vec, stream);
}

cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t stream) {
  const bool vec = a.K % 8 == 0 && aligned_to(a.x, a.x_type == kTypeB128 ? 8 : 16) &&
                   aligned_to(a.y, 16) && aligned_to(a.dx, 16);
  const int C = a.K <= kMaxWarps * 512 ? 2 : 4;
  const int W = (int)((a.K + 256 * C - 1) / (256 * C));
  const int G = kMaxWarps / W;
  if (C == 2) return vec ? pick_backward<2, true>(a, W, G, stream) : pick_backward<2, false>(a, W, G, stream);
  return vec ? pick_backward<4, true>(a, W, G, stream) : pick_backward<4, false>(a, W, G, stream);
}

}  // namespace mxq
