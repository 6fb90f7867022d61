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

constexpr int kMaxParts = 304;  // of the weight's gradient: rows are split over at most so many CTAs
constexpr int kBackwardThreads = 512;

// Barrier of one group of warps (ids 1 ..; a group of one warp needs none beyond its own order).
__device__ __forceinline__ void group_sync(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}

// Sum over the lanes that differ in the bits below N; over the warp.
template <int N = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int s = N / 2; s; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
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

// 8 consecutive values of a weight or a bias (aligned to 32 bytes), kept in L1 for the next rows.
__device__ __forceinline__ void load_param(const void* p, bool f32, int i, uint64_t (&v)[4]) {
  if (f32) {
    asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];"
                 : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3])
                 : "l"(static_cast<const float*>(p) + i));
  } else {
    const uint4 q = load_v4(static_cast<const uint16_t*>(p) + i);
    v[0] = bf16_pair(q.x);
    v[1] = bf16_pair(q.y);
    v[2] = bf16_pair(q.z);
    v[3] = bf16_pair(q.w);
  }
}

// N values of a weight or a bias (fallback where there is none), a group's width apart.
template <int N, typename F>
__device__ __forceinline__ void load_params(const void* p, bool f32, int K, F&& column, float fallback,
                                            float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = fallback;
  if (!p) return;
  if (f32) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (column(i) < K) v[i] = load_f32(static_cast<const float*>(p) + column(i));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (column(i) < K) v[i] = load_as_f32(p, false, column(i));
    }
  }
}

// N values of a row (0 where there is none) and their way back.
template <int N, typename F>
__device__ __forceinline__ void load_values(const char* row, bool f32, int K, F&& column, float (&v)[N]) {
  load_params(row, f32, K, column, 0.0f, v);
}
template <int N, typename F>
__device__ __forceinline__ void store_values(char* row, bool f32, int K, F&& column, const float (&v)[N]) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (column(i) < K) reinterpret_cast<float*>(row)[column(i)] = v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (column(i) < K) reinterpret_cast<uint16_t*>(row)[column(i)] = (uint16_t)pack_bf16(v[i], 0.0f);
    }
  }
}

// ------------------------------------------------------------------------------------------
// forward
// ------------------------------------------------------------------------------------------
// Mean and 1 / deviation of a row from each warp's mean and sum of squared differences from it (part: of the
// CTA's warps), count(w) values in warp w of the group: the warps' sums about their own means are joined with
// their means' distance from the row's.
template <int WARPS, typename F>
__device__ __forceinline__ void join_stats(const NormArgs& a, float2* part, int group, int W, F&& count,
                                           float& mean, float& sq) {
  const int lane = threadIdx.x & 31, i = lane & (WARPS - 1), w0 = group * W;
  if (lane == 0) part[threadIdx.x >> 5] = make_float2(mean, sq);
  group_sync(group, 32 * W);
  const float2 p = i < W ? part[w0 + i] : make_float2(0.0f, 0.0f);
  const float n = i < W ? (float)count(i) : 0.0f;
  mean = a.center ? __fdividef(warp_sum<WARPS>(p.x * n), (float)a.K) : 0.0f;
  sq = warp_sum<WARPS>(fmaf((p.x - mean) * n, p.x - mean, p.y));
}

// 1 / sqrt(sq / K + eps), within 2^-22 (an approximate root; 1 / K and the quotient round too).
__device__ __forceinline__ float deviation(const NormArgs& a, float sq) {
  return rsqrtf(fmaf(sq, __fdividef(1.0f, (float)a.K), a.eps));
}

__device__ __forceinline__ void store_stats(const NormArgs& a, int64_t row, float mean, float rstd) {
  if (a.mean) a.mean[row] = mean;
  if (a.rstd) a.rstd[row] = rstd;
}

// P runs of 8 columns per lane (run p: columns 8 (p T + t) ..) as codes, with their blocks' scales.
template <int P>
__device__ __forceinline__ void store_codes(const uint64_t (&v)[P][4], uint8_t* codes, float* scales,
                                            int64_t M, int K, int64_t row, int t, int T) {
  run_codes<P>(
      v,
      [&](int p, uint32_t lo, uint32_t hi) {
        const int col = (p * T + t) * 8;
        if (col < K) store8B(codes + row * K + col, lo, hi);
      },
      [&](int p, float scale) {
        const int kb = (p * T + t) >> 4;
        if (kb * kB128 < K) scales[kb * M + row] = scale;
      });
}

// A group of W warps per row, P runs of 8 columns per lane in fp32 pairs: the loads of a row are in flight
// together, and what hides its chain (load, two sums over the group, weights, stores) is the other rows of
// the SM. THREADS: of a CTA, at most.
template <bool XF32, int P, bool QUANT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) norm_kernel(NormArgs a, int W) {
  constexpr int kWarps = THREADS / 32;
  __shared__ float2 part[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int T = 32 * W, group = threadIdx.x / T, t = threadIdx.x - group * T, K = (int)a.K;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / T) + group;
  if (row >= a.M) return;
  auto column = [&](int p) { return (p * T + t) * 8; };
  auto count = [&](int w) {  // columns of the group's warp w
    int n = 0;
#pragma unroll
    for (int p = 0; p < P; ++p) n += min(max(K - (p * T + 32 * w) * 8, 0), 256);
    return n;
  };
  uint64_t x[P][4];
  const char* from = static_cast<const char*>(a.x) + row * K * (XF32 ? 4 : 2);
  uint32_t raw[P][XF32 ? 8 : 4];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (column(p) < K) {
      if constexpr (XF32) {
        load32B(from + column(p) * 4, raw[p]);
      } else {
        load16B(from + column(p) * 2, raw[p]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < (XF32 ? 8 : 4); ++j) raw[p][j] = 0u;
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (XF32) {
        x[p][j] = pair(__uint_as_float(raw[p][2 * j]), __uint_as_float(raw[p][2 * j + 1]));
      } else {
        x[p][j] = bf16_pair(raw[p][j]);
      }
    }
  }
  if constexpr (QUANT) {
    if (a.x_codes) store_codes<P>(x, a.x_codes, a.x_scales_out, a.M, K, row, t, T);
  }
  float mean = 0.0f;
  if (a.center) {
    uint64_t s[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4 * P; ++i) s[i & 1] = add_pair(s[i & 1], x[i / 4][i % 4]);
    s[0] = add_pair(s[0], s[1]);
    const int n = count(t >> 5);
    mean = n > 0 ? __fdividef(warp_sum(lo_of(s[0]) + hi_of(s[0])), (float)n) : 0.0f;
  }
  uint64_t s[2] = {0u, 0u};
  const uint64_t less = pair(-mean);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (column(p) >= K) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t d = add_pair(x[p][j], less);
      s[j & 1] = fma_pair(d, d, s[j & 1]);
    }
  }
  s[0] = add_pair(s[0], s[1]);
  float sq = warp_sum(lo_of(s[0]) + hi_of(s[0]));
  if (W > 1) join_stats<kWarps>(a, part, group, W, count, mean, sq);
  const float rstd = deviation(a, sq);
  if (t == 0) store_stats(a, row, mean, rstd);
  const uint64_t minus = pair(-mean), r2 = pair(rstd);
  const bool w_f32 = a.w_type == kTypeFp32;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (column(p) >= K) continue;  // zeros
    uint64_t w[4], b[4];
    if (a.weight) load_param(a.weight, w_f32, column(p), w);
    if (a.bias) load_param(a.bias, w_f32, column(p), b);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[p][j] = mul_pair(add_pair(x[p][j], minus), r2);
    if (a.weight) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[p][j] = mul_pair(x[p][j], w[j]);
    }
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[p][j] = add_pair(x[p][j], b[j]);
    }
    if constexpr (!QUANT) {
      uint32_t o[8];
      if (a.y_type == kTypeFp32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[2 * j] = __float_as_uint(lo_of(x[p][j]));
          o[2 * j + 1] = __float_as_uint(hi_of(x[p][j]));
        }
        store32B(static_cast<float*>(a.y) + row * K + column(p), o);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = bf16_word(x[p][j]);
        store16B(static_cast<uint16_t*>(a.y) + row * K + column(p), o);
      }
    }
  }
  if constexpr (QUANT) store_codes<P>(x, a.codes, a.scales, a.M, K, row, t, T);
}

// The same for rows of any length and alignment: 16 columns per lane, a group's width apart, loaded and
// stored one by one.
template <bool XF32, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) norm_any_kernel(NormArgs a, int W) {
  constexpr int kWarps = THREADS / 32;
  __shared__ float2 part[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int T = 32 * W, group = threadIdx.x / T, t = threadIdx.x - group * T, K = (int)a.K;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / T) + group;
  if (row >= a.M) return;
  auto column = [&](int i) { return i * T + t; };
  auto count = [&](int w) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) n += min(max(K - i * T - 32 * w, 0), 32);
    return n;
  };
  float x[16], p[16];
  load_values(static_cast<const char*>(a.x) + row * K * (XF32 ? 4 : 2), XF32, K, column, x);
  float mean = 0.0f;
  if (a.center) {
    float s[2] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i & 1] += x[i];
    const int n = count(t >> 5);
    mean = n > 0 ? __fdividef(warp_sum(s[0] + s[1]), (float)n) : 0.0f;
  }
  float s[2] = {};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float d = column(i) < K ? x[i] - mean : 0.0f;
    s[i & 1] = fmaf(d, d, s[i & 1]);
  }
  float sq = warp_sum(s[0] + s[1]);
  if (W > 1) join_stats<kWarps>(a, part, group, W, count, mean, sq);
  const float rstd = deviation(a, sq);
  if (t == 0) store_stats(a, row, mean, rstd);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = (x[i] - mean) * rstd;
  const bool w_f32 = a.w_type == kTypeFp32;
  load_params(a.weight, w_f32, K, column, 1.0f, p);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] *= p[i];
  load_params(a.bias, w_f32, K, column, 0.0f, p);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] += p[i];
  const bool y_f32 = a.y_type == kTypeFp32;
  store_values(static_cast<char*>(a.y) + row * K * (y_f32 ? 4 : 2), y_f32, K, column, x);
}

// ------------------------------------------------------------------------------------------
// backward
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

__device__ __forceinline__ void unpack8(uint4 q, uint64_t* v) {
  v[0] = bf16_pair(q.x);
  v[1] = bf16_pair(q.y);
  v[2] = bf16_pair(q.z);
  v[3] = bf16_pair(q.w);
}

// Chunks of 8 values per lane: the pieces of a row that a thread copies into places of its own in shared
// memory (so no barrier is needed), `stages` rows ahead.
template <int C, int XT, bool DYF32>
struct NormRing {
  static constexpr int kX = XT == kTypeB128 ? 8 : XT == kTypeFp32 ? 32 : 16, kDy = DYF32 ? 32 : 16;
  static constexpr int kScale = XT == kTypeB128 ? 4 : 0;
  static constexpr int kChunk = kX + kDy + kScale;  // bytes of shared memory per thread, chunk and stage
  static constexpr int kFit = 200 * 1024 / (kBackwardThreads * C * kChunk);
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static_assert(kStages >= 1, "a row fits shared memory");

  uint8_t* sm;
  int threads, tid;

  __device__ __forceinline__ uint8_t* place(int stage, int c) const {
    return sm + (stage * C + c) * kChunk * threads;
  }
  __device__ __forceinline__ void request(const NormArgs& a, int64_t row, int col, int stage, int c) const {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(place(stage, c));
    const char* x = static_cast<const char*>(a.x) + (row * a.K + col) * (kX / 8);
    const char* dy = static_cast<const char*>(a.y) + (row * a.K + col) * (kDy / 8);
    if constexpr (XT == kTypeB128) {
      copy8(at + tid * 8, x);
    } else {
#pragma unroll
      for (int p = 0; p < kX / 16; ++p) copy16(at + (p * threads + tid) * 16, x + p * 16);
    }
#pragma unroll
    for (int p = 0; p < kDy / 16; ++p) copy16(at + kX * threads + (p * threads + tid) * 16, dy + p * 16);
    if constexpr (XT == kTypeB128) {
      copy4(at + (kX + kDy) * threads + tid * 4, a.x_scales + col / kB128 * a.M + row);
    }
  }
  __device__ __forceinline__ void read(int stage, int c, uint64_t* x, uint64_t* dy) const {
    const uint8_t* at = place(stage, c);
    if constexpr (XT == kTypeBf16) {
      unpack8(reinterpret_cast<const uint4*>(at)[tid], x);
    } else if constexpr (XT == kTypeFp32) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        *reinterpret_cast<ulonglong2*>(x + 2 * p) = reinterpret_cast<const ulonglong2*>(at)[p * threads + tid];
      }
    } else {
      const uint2 q = reinterpret_cast<const uint2*>(at)[tid];
      const float s = reinterpret_cast<const float*>(at + (kX + kDy) * threads)[tid];
      values4(q.x, x[0], x[1]);
      values4(q.y, x[2], x[3]);
      // (not packed: ptxas joins a packed product and the sum after it, and with it two roundings)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = pair(__fmul_rn(lo_of(x[j]), s), __fmul_rn(hi_of(x[j]), s));
    }
    const uint8_t* dys = at + kX * threads;
    if constexpr (DYF32) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        *reinterpret_cast<ulonglong2*>(dy + 2 * p) = reinterpret_cast<const ulonglong2*>(dys)[p * threads + tid];
      }
    } else {
      unpack8(reinterpret_cast<const uint4*>(dys)[tid], dy);
    }
  }
};

// Two sums over the row of a group of W warps (slot: of two, taken in turn): the two halves of a warp take one
// each, so that five exchanges do for both.
__device__ __forceinline__ void row_sums(float (&part)[2][2][kBackwardThreads / 32], int slot, int group, int W,
                                         float& s1, float& s2) {
  constexpr int kWarps = kBackwardThreads / 32;
  const int lane = threadIdx.x & 31, half = lane >> 4;
  float mine = half ? s2 : s1;
  mine += __shfl_xor_sync(0xFFFFFFFFu, half ? s1 : s2, 16);
  mine = warp_sum<16>(mine);
  if (W > 1) {
    const int i = lane & (kWarps - 1);
    if (i == 0) part[slot][half][threadIdx.x >> 5] = mine;
    group_sync(group, 32 * W);
    mine = warp_sum<kWarps>(i < W ? part[slot][half][group * W + i] : 0.0f);
  }
  const float other = __shfl_xor_sync(0xFFFFFFFFu, mine, 16);
  s1 = half ? other : mine;
  s2 = half ? mine : other;
}

// The groups' shares of dw and db (N columns of a thread), joined in their order through shared memory, to
// this CTA's row of the workspace; of a single CTA to where they belong.
template <int N, typename F, typename W1, typename W2>
__device__ __forceinline__ void store_shares(const NormArgs& a, float* sm, int W, F&& column, W1&& dw,
                                             W2&& db) {
  const int T = 32 * W, groups = blockDim.x / T, group = threadIdx.x / T, K = (int)a.K;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* whole = k ? a.dbias : a.dweight;
    if (!whole) continue;
    float* out = gridDim.x == 1 ? whole : a.workspace + (k * (int64_t)gridDim.x + blockIdx.x) * K;
    float* to = groups > 1 ? sm + group * K : out;
    if (groups > 1) __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (column(i) < K) to[column(i)] = k ? db(i) : dw(i);
    }
    if (groups == 1) continue;
    __syncthreads();
    for (int col = threadIdx.x; col < K; col += blockDim.x) {
      float s = 0.0f;
      for (int i = 0; i < groups; ++i) s += sm[i * K + col];
      out[col] = s;
    }
  }
}

// Gradient of the input, and each CTA's share of the parameters' gradients, which norm_reduce_kernel
// adds up. A CTA walks rows gridDim.x groups apart, its sums of dw and db in registers. With two chunks a
// lane keeps xhat and g over the sums of the row, with four it reads the row from its places again.
template <int C, int XT, bool DYF32>
__global__ void __launch_bounds__(kBackwardThreads, 1) norm_backward_kernel(NormArgs a, int W) {
  extern __shared__ __align__(16) uint8_t ring_shared[];
  __shared__ float part[2][2][kBackwardThreads / 32];
  using Ring = NormRing<C, XT, DYF32>;
  constexpr bool kKeep = C <= 2;
  pdl_launch_dependents();
  pdl_wait();
  const int T = 32 * W, group = threadIdx.x / T, t = threadIdx.x - group * T, K = (int)a.K;
  const Ring ring{ring_shared, (int)blockDim.x, (int)threadIdx.x};
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / T);
  int64_t row = (int64_t)blockIdx.x * (blockDim.x / T) + group;
  const bool dx_f32 = a.dx_type == kTypeFp32, w_f32 = a.w_type == kTypeFp32;
  const float per_k = __fdiv_rn(1.0f, (float)K);

  auto column = [&](int i) { return ((i / 8) * T + t) * 8 + i % 8; };
  auto request = [&](int64_t at, int stage) {
    if (at < a.M) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (column(8 * c) < K) ring.request(a, at, column(8 * c), stage, c);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto load_weight = [&](int c, uint64_t (&w)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pair(1.0f);
    if (a.weight && column(8 * c) < K) load_param(a.weight, w_f32, column(8 * c), w);
  };
  auto store = [&](int c, const uint64_t* g, const uint64_t* xh, float s1, float s2, float rstd) {
    uint64_t d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[j] = mul_pair(fma_pair(xh[j], pair(-s2), add_pair(g[j], pair(-s1))), pair(rstd));
    }
    uint32_t o[8];
    if (dx_f32) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[2 * j] = __float_as_uint(lo_of(d[j]));
        o[2 * j + 1] = __float_as_uint(hi_of(d[j]));
      }
      store16B(static_cast<float*>(a.dx) + row * K + column(8 * c), o);
      store16B(static_cast<float*>(a.dx) + row * K + column(8 * c) + 4, o + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = bf16_word(d[j]);
      store16B(static_cast<uint16_t*>(a.dx) + row * K + column(8 * c), o);
    }
  };

  uint64_t w[kKeep ? C : 1][4], dw[4 * C], db[4 * C];
#pragma unroll
  for (int i = 0; i < 4 * C; ++i) dw[i] = db[i] = 0u;
  if constexpr (kKeep) {
#pragma unroll
    for (int c = 0; c < C; ++c) load_weight(c, w[c]);
  }
#pragma unroll
  for (int s = 0; s < Ring::kStages; ++s) request(row + s * step, s);
  float mean_next = 0.0f, rstd_next = 0.0f;
  if (row < a.M) {
    rstd_next = load_f32(a.rstd + row);
    if (a.mean) mean_next = load_f32(a.mean + row);
  }
  int stage = 0;
  for (int slot = 0; row < a.M; row += step, slot ^= 1) {
    const float mean = mean_next, rstd = rstd_next;
    const uint64_t minus = pair(-mean), r2 = pair(rstd);
    if (row + step < a.M) {
      rstd_next = load_f32(a.rstd + row + step);
      if (a.mean) mean_next = load_f32(a.mean + row + step);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(Ring::kStages - 1) : "memory");
    uint64_t xh[kKeep ? C : 1][4], g[kKeep ? C : 1][4];
    uint64_t c1 = 0u, c2 = 0u;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      constexpr int kOne = 0;
      uint64_t(&x)[4] = xh[kKeep ? c : kOne];
      uint64_t(&y)[4] = g[kKeep ? c : kOne];
      uint64_t(&u)[4] = w[kKeep ? c : kOne];
      if (column(8 * c) < K) {
        ring.read(stage, c, x, y);
        if constexpr (!kKeep) load_weight(c, u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = mul_pair(add_pair(x[j], minus), r2);
          dw[4 * c + j] = fma_pair(y[j], x[j], dw[4 * c + j]);
          db[4 * c + j] = add_pair(db[4 * c + j], y[j]);
          y[j] = mul_pair(y[j], u[j]);
          c1 = add_pair(c1, y[j]);
          c2 = fma_pair(y[j], x[j], c2);
        }
      }
    }
    if constexpr (kKeep) {  // into the places just read, by this thread alone
      request(row + Ring::kStages * step, stage);
    }
    float s1 = lo_of(c1) + hi_of(c1), s2 = lo_of(c2) + hi_of(c2);
    row_sums(part, slot, group, W, s1, s2);
    s1 = a.mean ? s1 * per_k : 0.0f;
    s2 *= per_k;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (column(8 * c) >= K) continue;
      if constexpr (kKeep) {
        store(c, g[c], xh[c], s1, s2, rstd);
      } else {
        ring.read(stage, c, xh[0], g[0]);
        load_weight(c, w[0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xh[0][j] = mul_pair(add_pair(xh[0][j], minus), r2);
          g[0][j] = mul_pair(g[0][j], w[0][j]);
        }
        store(c, g[0], xh[0], s1, s2, rstd);
      }
    }
    if constexpr (!kKeep) request(row + Ring::kStages * step, stage);
    stage = stage + 1 == Ring::kStages ? 0 : stage + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (a.dweight || a.dbias) {
    store_shares<8 * C>(
        a, reinterpret_cast<float*>(ring_shared), W, column,
        [&](int i) { return i & 1 ? hi_of(dw[i / 2]) : lo_of(dw[i / 2]); },
        [&](int i) { return i & 1 ? hi_of(db[i / 2]) : lo_of(db[i / 2]); });
  }
}

// The same for rows of any length and alignment: N values of a lane, a group's width apart, loaded one by
// one.
template <int N>
__global__ void __launch_bounds__(kBackwardThreads, 1) norm_backward_any_kernel(NormArgs a, int W) {
  extern __shared__ __align__(16) uint8_t ring_shared[];
  __shared__ float part[2][2][kBackwardThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int T = 32 * W, group = threadIdx.x / T, t = threadIdx.x - group * T, K = (int)a.K;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / T);
  int64_t row = (int64_t)blockIdx.x * (blockDim.x / T) + group;
  const bool x_f32 = a.x_type == kTypeFp32, dy_f32 = a.y_type == kTypeFp32, dx_f32 = a.dx_type == kTypeFp32;
  const bool codes = a.x_type == kTypeB128, w_f32 = a.w_type == kTypeFp32;
  const float per_k = __fdiv_rn(1.0f, (float)K);
  auto column = [&](int i) { return i * T + t; };
  float dw[N], db[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = db[i] = 0.0f;
  for (int slot = 0; row < a.M; row += step, slot ^= 1) {
    const float rstd = load_f32(a.rstd + row), mean = a.mean ? load_f32(a.mean + row) : 0.0f;
    const char* x = static_cast<const char*>(a.x) + row * K * (codes ? 1 : x_f32 ? 4 : 2);
    const char* dy = static_cast<const char*>(a.y) + row * K * (dy_f32 ? 4 : 2);
    float xh[N], g[N], w[N];
    if (codes) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        xh[i] = 0.0f;
        if (column(i) >= K) continue;
        float lo, hi;
        e4m3x2_to_f32(load_u8(x + column(i)), lo, hi);
        xh[i] = __fmul_rn(lo, load_f32(a.x_scales + column(i) / kB128 * a.M + row));
      }
    } else {
      load_values(x, x_f32, K, column, xh);
    }
    load_values(dy, dy_f32, K, column, g);
    load_params(a.weight, w_f32, K, column, 1.0f, w);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {  // (g is 0 where there is no column)
      xh[i] = (xh[i] - mean) * rstd;
      dw[i] = fmaf(g[i], xh[i], dw[i]);
      db[i] += g[i];
      g[i] *= w[i];
      s1 += g[i];
      s2 = fmaf(g[i], xh[i], s2);
    }
    row_sums(part, slot, group, W, s1, s2);
    s1 = a.mean ? s1 * per_k : 0.0f;
    s2 *= per_k;
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = fmaf(-xh[i], s2, g[i] - s1) * rstd;
    store_values(static_cast<char*>(a.dx) + row * K * (dx_f32 ? 4 : 2), dx_f32, K, column, g);
  }
  if (a.dweight || a.dbias) {
    store_shares<N>(
        a, reinterpret_cast<float*>(ring_shared), W, column, [&](int i) { return dw[i]; },
        [&](int i) { return db[i]; });
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

cudaError_t run_norm(void (*kernel)(NormArgs, int), const NormArgs& a, int W, cudaStream_t stream) {
  const int G = W >= 8 ? 1 : 8 / W;  // rows of a CTA
  return launch_pdl(kernel, dim3((unsigned)((a.M + G - 1) / G)), dim3(32 * W * G), 0, stream, a, W);
}

// Rows of up to 512 columns are one warp's with one or two runs per lane; longer ones a group's with four.
template <bool XF32, bool QUANT>
cudaError_t pick_norm(const NormArgs& a, cudaStream_t stream) {
  if (a.K <= 256) return run_norm(&norm_kernel<XF32, 1, QUANT, 256>, a, 1, stream);
  if (a.K <= 512) return run_norm(&norm_kernel<XF32, 2, QUANT, 256>, a, 1, stream);
  const int W = (int)((a.K + 1023) / 1024);
  return run_norm(W <= 8 ? &norm_kernel<XF32, 4, QUANT, 256> : &norm_kernel<XF32, 4, QUANT, 512>, a, W, stream);
}

template <bool XF32>
cudaError_t pick_norm(const NormArgs& a, bool vec, cudaStream_t stream) {
  if (a.codes) return pick_norm<XF32, true>(a, stream);
  if (vec) return pick_norm<XF32, false>(a, stream);
  const int W = (int)((a.K + 511) / 512);
  return run_norm(W <= 8 ? &norm_any_kernel<XF32, 256> : &norm_any_kernel<XF32, 1024>, a, W, stream);
}

cudaError_t run_backward(void (*kernel)(NormArgs, int), int ring_bytes, const NormArgs& a, int W,
                         cudaStream_t stream) {
  const int G = kBackwardThreads / 32 / W, threads = 32 * W * G;  // G rows of a CTA at once
  const bool params = a.dweight || a.dbias;
  size_t smem = (size_t)ring_bytes * threads;
  if (params && G > 1 && smem < (size_t)G * a.K * 4) smem = (size_t)G * a.K * 4;
  const int64_t slots = resident_ctas(reinterpret_cast<const void*>(kernel), threads, smem, 0);
  if (slots <= 0) return cudaErrorInvalidConfiguration;
  int64_t ctas = (a.M + G - 1) / G;
  if (ctas > slots) ctas = slots;
  if (params && ctas > kMaxParts) ctas = kMaxParts;
  const cudaError_t err = launch_pdl(kernel, dim3((unsigned)ctas), dim3(threads), smem, stream, a, W);
  if (err != cudaSuccess || !params || ctas == 1) return err;
  return launch_pdl(&norm_reduce_kernel, dim3((unsigned)((a.K + 31) / 32), 2), dim3(512), 0, stream, a,
                    (int)ctas);
}

template <int C, int XT, bool DYF32>
cudaError_t run_ring(const NormArgs& a, int W, cudaStream_t stream) {
  using Ring = NormRing<C, XT, DYF32>;
  return run_backward(&norm_backward_kernel<C, XT, DYF32>, Ring::kStages * C * Ring::kChunk, a, W, stream);
}

template <int C>
cudaError_t pick_ring(const NormArgs& a, cudaStream_t stream) {
  const int W = (int)((a.K + 256 * C - 1) / (256 * C));
  const bool dy_f32 = a.y_type == kTypeFp32;
  if (a.x_type == kTypeBf16) {
    return dy_f32 ? run_ring<C, kTypeBf16, true>(a, W, stream) : run_ring<C, kTypeBf16, false>(a, W, stream);
  }
  if (a.x_type == kTypeFp32) {
    return dy_f32 ? run_ring<C, kTypeFp32, true>(a, W, stream) : run_ring<C, kTypeFp32, false>(a, W, stream);
  }
  return dy_f32 ? run_ring<C, kTypeB128, true>(a, W, stream) : run_ring<C, kTypeB128, false>(a, W, stream);
}

}  // namespace

int64_t norm_workspace_floats(int64_t M, int64_t K) { return 2 * (M < kMaxParts ? M : kMaxParts) * K; }

cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
  const bool vec = a.codes || (a.K % 8 == 0 && aligned_to(a.x, 32) && aligned_to(a.y, 32) &&
                               aligned_to(a.weight, 32) && aligned_to(a.bias, 32));
  return a.x_type == kTypeFp32 ? pick_norm<true>(a, vec, stream) : pick_norm<false>(a, vec, stream);
}

cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t stream) {
  const bool vec = a.K % 8 == 0 && aligned_to(a.x, a.x_type == kTypeB128 ? 8 : 16) &&
                   aligned_to(a.y, 16) && aligned_to(a.dx, 16) && aligned_to(a.weight, 32);
  if (vec) return a.K <= 8192 ? pick_ring<2>(a, stream) : pick_ring<4>(a, stream);
  const int W = (int)((a.K + (a.K <= 8192 ? 511 : 1023)) / (a.K <= 8192 ? 512 : 1024));
  return a.K <= 8192 ? run_backward(&norm_backward_any_kernel<16>, 0, a, W, stream)
                     : run_backward(&norm_backward_any_kernel<32>, 0, a, W, stream);
}

}  // namespace mxq
