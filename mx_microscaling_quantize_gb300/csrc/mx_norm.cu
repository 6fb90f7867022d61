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
// costs what its own sum in fp32 is off by, not the digits of its square. All sums are in fp32 in a fixed order.
//
// x[8192, 8192] against its bytes at the rate of a plain copy (6.7 TB/s): bf16 into bf16 47 us (40), fp32 into
// bf16 64 (60), bf16 into codes 42 (30), with a checkpoint 52 (41), fp32 into codes 58 (50); gradients bf16 68 (60;
// 61 without those of the parameters), fp32 x 109 (100), from a checkpoint 70 (50); of fp32 dy into bf16 101 (80),
// 136 (100) and 93 (71), with 32 to 48 bytes of registers spilled. Rows of 2048, 4001 of them: into codes 9.5 us, gradients 18. One
// row of 8192: 2.7 and 4.3.
#include "mx_b128.cuh"
#include "mx_device.cuh"
#include "mx_launch.h"
#include "mx_tcgen05.cuh"
#include "mx_train.h"

namespace mxq {

namespace {

constexpr int kMaxParts = 304;  // of the weight's gradient: rows are split over at most so many CTAs
constexpr int kNormThreads = 512, kMaxStages = 4;  // of a CTA
constexpr int kNormSmem = 224 * 1024;  // of a CTA, dynamic
constexpr unsigned long long kNormDrainNs = 2000000000ull;  // 2 s, whatever the limit of other waits

// Barrier of one group of warps: of several warps barrier group + 1 (there are 16, the CTA's among them), of one
// warp the warp's.
static_assert(kNormThreads / 64 <= 15, "groups of several warps have a barrier each");
__device__ __forceinline__ void group_sync(int group, int threads) {
  if (threads == 32) {
    __syncwarp();
  } else {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
  }
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

// 8 consecutive values (aligned to their size)
__device__ __forceinline__ void load_run(const char* p, bool f32, uint64_t (&v)[4]) {
  if (f32) {
    asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];"
                 : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3])
                 : "l"(p));
  } else {
    const uint4 q = load_v4(p);
    v[0] = bf16_pair(q.x);
    v[1] = bf16_pair(q.y);
    v[2] = bf16_pair(q.z);
    v[3] = bf16_pair(q.w);
  }
}
__device__ __forceinline__ void store_run(void* p, bool f32, int64_t at, const uint64_t (&y)[4]) {
  uint32_t o[8];
  if (f32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[2 * j] = __float_as_uint(lo_of(y[j]));
      o[2 * j + 1] = __float_as_uint(hi_of(y[j]));
    }
    store32B(static_cast<float*>(p) + at, o);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = bf16_word(y[j]);
    store16B(static_cast<uint16_t*>(p) + at, o);
  }
}

// N values of a lane, 32 apart from its first on, of which `left` places from there on are in the row: all of most
// warps, which then ask nothing value by value and address them all from one register. Of a weight or a bias
// (fallback where there is none):
template <int N, typename F>
__device__ __forceinline__ void for_values(int left, F&& f) {
  if (left > (N - 1) * 32) {
#pragma unroll
    for (int i = 0; i < N; ++i) f(i);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i * 32 < left) f(i);
    }
  }
}
template <int N>
__device__ __forceinline__ void load_params(const void* p, bool f32, int col, int left, float fallback, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = fallback;
  if (!p) return;
  if (f32) {
    const float* at = static_cast<const float*>(p) + col;
    for_values<N>(left, [&](int i) { v[i] = load_f32(at + i * 32); });
  } else {
    const uint16_t* at = static_cast<const uint16_t*>(p) + col;
    for_values<N>(left, [&](int i) { v[i] = __uint_as_float(load_u16(at + i * 32) << 16); });
  }
}
// Of a row from `at` on (0 where there is none), as they lie in memory, so that nothing waits for them before they
// are used (value_of), and their way back.
template <int N>
__device__ __forceinline__ void load_values(const char* at, bool f32, int left, uint32_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0u;
  if (f32) {
    for_values<N>(left, [&](int i) { v[i] = __float_as_uint(load_f32(reinterpret_cast<const float*>(at) + i * 32)); });
  } else {
    for_values<N>(left, [&](int i) { v[i] = load_u16(reinterpret_cast<const uint16_t*>(at) + i * 32); });
  }
}
__device__ __forceinline__ float value_of(uint32_t raw, bool f32) { return __uint_as_float(raw << (f32 ? 0 : 16)); }
template <int N>
__device__ __forceinline__ void store_values(char* at, bool f32, int left, const float (&v)[N]) {
  if (f32) {
    for_values<N>(left, [&](int i) { reinterpret_cast<float*>(at)[i * 32] = v[i]; });
  } else {
    for_values<N>(left, [&](int i) { reinterpret_cast<uint16_t*>(at)[i * 32] = (uint16_t)pack_bf16(v[i], 0.0f); });
  }
}

// ------------------------------------------------------------------------------------------
// rows through shared memory
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ void unpack8(uint4 q, uint64_t* v) {
  v[0] = bf16_pair(q.x);
  v[1] = bf16_pair(q.y);
  v[2] = bf16_pair(q.z);
  v[3] = bf16_pair(q.w);
}
// 8 values of a row at a shared address
template <bool F32>
__device__ __forceinline__ void read8(uint32_t at, uint64_t* v) {
  if constexpr (F32) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[2 * p]), "=l"(v[2 * p + 1]) : "r"(at + 16 * p));
    }
  } else {
    uint4 q;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at));
    unpack8(q, v);
  }
}
__device__ __forceinline__ void bulk_copy(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
      "l"(from), "r"(bytes), "r"(bar)
      : "memory");
}

// The rows that a group asks for: S stages, each with a barrier, taken in turn. A thread whose wait runs out waits once
// more, with one limit, for all that it has asked for, so that no copy outlives the CTA; after that it asks for nothing
// and waits for nothing, but goes on arriving, so that the barriers go on for the threads that wait.
struct RowStages {
  uint32_t bars;
  int S, ahead, stage = 0, parity = 0;  // ahead: rows asked for when one is waited for
  bool failed = false;

  __device__ __forceinline__ RowStages(uint64_t* full, int S_, int ahead_)
      : bars((uint32_t)__cvta_generic_to_shared(full)), S(S_), ahead(ahead_) {}
  __device__ __forceinline__ void init(uint32_t arrivals) const {
    for (int s = 0; s < S; ++s) tc::mbar_init(bars + s * 8, arrivals);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tc::fence_proxy_async_smem();
  }
  __device__ __forceinline__ uint32_t bar(int s) const { return bars + s * 8; }
  // One attempt. The hardware's own wait takes any time up to kAttemptNs and more (a limit given to it does not end it
  // sooner), so shorter limits look without waiting.
  static constexpr uint32_t kAttemptNs = 1000000;
  static __device__ __forceinline__ bool landed(uint32_t bar, uint32_t parity, bool look) {
    uint32_t ok;
    if (look) {
      asm volatile(
          "{\n\t.reg .pred P;\n\tmbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, P;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity)
          : "memory");
    } else {
      asm volatile(
          "{\n\t.reg .pred P;\n\tmbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, P;\n\t}"
          : "=r"(ok)
          : "r"(bar), "r"(parity), "r"(kAttemptNs)
          : "memory");
    }
    return ok != 0;
  }
  __device__ __forceinline__ void wait(const NormArgs& a, int64_t row, int64_t step) {
    if (failed) return;
    const bool look = a.wait_limit_ns <= 100ull * kAttemptNs;
    if (landed(bar(stage), parity, look)) return;
    const unsigned long long t0 = tc::global_ns();
    while (!landed(bar(stage), parity, look)) {
      if (tc::global_ns() - t0 > a.wait_limit_ns) {
        failed = true;
        atomicOr(a.err, 1u);
        break;
      }
    }
    if (!failed) return;
    const unsigned long long t1 = tc::global_ns();
#pragma unroll 1
    for (int k = 0; k < ahead && row + k * step < a.M; ++k) {
      const int s = stage + k < S ? stage + k : stage + k - S;
      while (!landed(bar(s), s == stage + k ? parity : parity ^ 1, false)) {
        if (tc::global_ns() - t1 > kNormDrainNs) {
          atomicOr(a.err, 1u);
          break;
        }
      }
    }
  }
  __device__ __forceinline__ void next() {
    if (++stage == S) {
      stage = 0;
      parity ^= 1;
    }
  }
};

// A parameter of the columns of a group, in fp32: run c of lane l of warp w as two pieces of 16 bytes 512 apart,
// so that a warp's reads meet no bank twice. store: each lane of a group its own runs; at: of (w, l), run 0.
template <int P>
struct ParamRuns {
  static constexpr int kBytes = P * 32;  // per thread
  static __device__ __forceinline__ uint32_t at(uint32_t base, int w, int lane) {
    return base + w * P * 1024 + lane * 16;
  }
  static __device__ __forceinline__ void store(uint32_t at, const void* p, bool f32, int col, int K, float none) {
    uint64_t v[P][4];
#pragma unroll
    for (int c = 0; c < P; ++c) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[c][j] = pair(none);
      if (p && col + c * 256 < K) load_run(static_cast<const char*>(p) + (col + c * 256) * (f32 ? 4 : 2), f32, v[c]);
    }
#pragma unroll
    for (int c = 0; c < P; ++c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(at + c * 1024 + h * 512), "l"(v[c][2 * h]),
                     "l"(v[c][2 * h + 1])
                     : "memory");
      }
    }
  }
  static __device__ __forceinline__ void read(uint32_t at, int c, uint64_t* v) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                   : "=l"(v[2 * h]), "=l"(v[2 * h + 1])
                   : "r"(at + c * 1024 + h * 512));
    }
  }
};

// ------------------------------------------------------------------------------------------
// forward
// ------------------------------------------------------------------------------------------
// sum / n from per_n = 1 / n, with what the rounding of per_n leaves put right: n times the first quotient is taken
// from the sum in one operation. A sum that is n times a value gives the value, so a row of equal values of which the
// sums are exact (all of bf16) has the differences 0. Beside the product with per_n alone: one row of 8192 2.46 ->
// 2.50 us, 8192 x 8192 of them into codes 42.6 -> 42.3. Correcting the mean by the sum of the differences to it would
// give that for sums that are not exact too, for 42.6 -> 47.4.
__device__ __forceinline__ float quotient(float sum, float n, float per_n) {
  const float q = __fmul_rn(sum, per_n), r = fmaf(fmaf(-n, q, sum), per_n, q);
  return r == r ? r : q;  // (an infinity stays one)
}

__device__ __forceinline__ float deviation(const NormArgs& a, float sq) {
  return __frsqrt_rn(fmaf(sq, __fdiv_rn(1.0f, (float)a.K), a.eps));
}

__device__ __forceinline__ void store_stats(const NormArgs& a, int64_t row, float mean, float rstd) {
  if (a.mean) a.mean[row] = mean;
  if (a.rstd) a.rstd[row] = rstd;
}

// R rows from `row` on, P runs of 8 columns per lane and row, 256 apart from col on, as codes with their
// blocks' scales.
template <int R, int P, bool FULL>
__device__ __forceinline__ void store_codes(const uint64_t (&v)[R * P][4], int lane, uint8_t* codes, float* scales,
                                            int64_t M, int K, int64_t row, int col) {
  const bool second = row + 1 < M;
  uint8_t* to = codes + row * K + col;
  run_codes<R * P>(
      v, lane,
      [&](int n, uint32_t lo, uint32_t hi) {
        const int p = n % P, r = n / P;
        if ((FULL || col + p * 256 < K) && (r == 0 || second)) store8B(to + r * K + p * 256, lo, hi);
      },
      [&](int n, float scale) {
        const int p = n % P, r = n / P, kb = (col + p * 256) / kB128;
        if ((FULL || kb * kB128 < K) && (r == 0 || second)) scales[kb * M + row + r] = scale;
      });
}

// Sums over a warp of a value of each of R rows: of two rows, the halves of the warp take one each.
template <int R>
__device__ __forceinline__ void warp_sums(float (&v)[R], bool high) {
  static_assert(R == 1 || R == 2, "rows of a group");
  if constexpr (R == 1) {
    v[0] = warp_sum(v[0]);
  } else {
    float mine = high ? v[1] : v[0];
    mine = warp_sum<16>(mine + __shfl_xor_sync(0xFFFFFFFFu, high ? v[0] : v[1], 16));
    const float other = __shfl_xor_sync(0xFFFFFFFFu, mine, 16);
    v[0] = high ? other : mine;
    v[1] = high ? mine : other;
  }
}

// A group of W warps for R adjacent rows, a warp's lanes P runs of 8 columns of each, 256 apart, in fp32 pairs.
// One CTA an SM: its groups walk rows, each with S times R rows on their way into its own shared memory (bulk
// copies; their place is free once the group has them in registers and met for the sums), beside one copy of
// the parameters for all. Two rows share what is done once: the reads of the parameters (which with the
// rows' own are as much of the shared memory's time as a row's bytes are of the memory's), the steps of the
// sums and a block's quotients (8192 x 8192 into codes: one row 54 us, two 42). FULL: K is a multiple of a
// warp's columns.
// Codes take 12 instructions for a value and 16 with a checkpoint, issued in 54 % of the cycles by 16 warps (an
// SM's registers hold no more), which wait for shared memory, for results and for the arithmetic pipes in like
// parts: dropping one in fifteen of them, or half of the exchanges over the warps, changed nothing for bf16. 32
// warps of half as many values each share the steps of a row among fewer values: 42 -> 53 us.
template <bool XF32, int P, int R, bool QUANT, bool FULL>
__global__ void __launch_bounds__(kNormThreads, 1) norm_kernel(NormArgs a, int W, int S) {
  extern __shared__ __align__(16) uint8_t norm_shared[];
  using Param = ParamRuns<P>;
  constexpr int kSize = XF32 ? 4 : 2, kStage = R * P * 8 * kSize;  // bytes of R rows per thread
  __shared__ float2 part[2][R][kNormThreads / 32];
  __shared__ __align__(8) uint64_t full[kNormThreads / 32][kMaxStages];
  const int T = 32 * W, group = threadIdx.x / T, t = threadIdx.x - group * T, K = (int)a.K;
  const int lane = threadIdx.x & 31, wi = t >> 5, col = wi * (P * 256) + lane * 8;
  const bool high = lane & 16;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(norm_shared);
  const uint32_t w_at = Param::at(base, wi, lane), b_at = Param::at(base + T * Param::kBytes, wi, lane);
  const uint32_t rows_at = base + 2 * T * Param::kBytes + group * S * T * kStage;
  RowStages rows(full[group], S, S);
  if (t == 0) rows.init(1);
  pdl_launch_dependents();
  __syncthreads();
  pdl_wait();
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / T) * R;
  int64_t row = ((int64_t)blockIdx.x * (blockDim.x / T) + group) * R;
  const uint32_t row_bytes = K * kSize;
  auto request = [&](int64_t at, int stage) {
    if (t != 0 || at >= a.M) return;
    if (rows.failed) {
      tc::mbar_arrive(rows.bar(stage));
      return;
    }
    const uint32_t bytes = (uint32_t)(a.M - at < R ? a.M - at : R) * row_bytes;
    tc::mbar_arrive_expect_tx(rows.bar(stage), bytes);
    bulk_copy(rows_at + stage * T * kStage, static_cast<const char*>(a.x) + at * row_bytes, bytes,
              rows.bar(stage));
  };
  for (int s = 0; s < S; ++s) request(row + s * step, s);
  const bool w_f32 = a.w_type == kTypeFp32, y_f32 = a.y_type == kTypeFp32;
  if (group == 0) {
    Param::store(w_at, a.weight, w_f32, col, K, 1.0f);
    Param::store(b_at, a.bias, w_f32, col, K, 0.0f);
  }
  __syncthreads();
  auto there = [&](int p) { return FULL || col + p * 256 < K; };
  auto count = [&](int w) { return (float)min(max(K - w * (P * 256), 0), P * 256); };  // columns of warp w
  const float mine = count(wi), per_mine = __fdiv_rn(1.0f, mine), per_k = __fdiv_rn(1.0f, (float)K);
  // lanes of the sums over warps: of all 32 for one row, of a half for each of two
  const int w_of = R == 1 ? lane : lane & 15;
  const float theirs = w_of < W ? count(w_of) : 0.0f;
  for (int slot = 0; row < a.M; row += step, slot ^= 1) {
    rows.wait(a, row, step);
    uint64_t x[R * P][4];
    const uint32_t from = rows_at + rows.stage * T * kStage + col * kSize;
#pragma unroll
    for (int n = 0; n < R * P; ++n) {
      if (there(n % P) && (n < P || row + 1 < a.M)) {
        read8<XF32>(from + (n / P) * row_bytes + (n % P) * 256 * kSize, x[n]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[n][j] = 0u;
      }
    }
    float mean[R], sq[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      uint64_t s[2] = {x[r * P][0], x[r * P][1]};
#pragma unroll
      for (int i = 2; i < 4 * P; ++i) s[i & 1] = add_pair(s[i & 1], x[r * P + i / 4][i % 4]);
      s[0] = add_pair(s[0], s[1]);
      mean[r] = lo_of(s[0]) + hi_of(s[0]);
    }
    warp_sums<R>(mean, high);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = a.center ? quotient(mean[r], mine, per_mine) : 0.0f;
      const uint64_t minus = pair(-mean[r]);
      uint64_t s[2] = {0u, 0u};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        if (!there(p)) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t d = add_pair(x[r * P + p][j], minus);
          s[j & 1] = fma_pair(d, d, s[j & 1]);
        }
      }
      s[0] = add_pair(s[0], s[1]);
      sq[r] = lo_of(s[0]) + hi_of(s[0]);
    }
    warp_sums<R>(sq, high);
    if (W > 1) {  // the warps' sums about their own means, joined with the means' distances from the row's
      if (lane == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) part[slot][r][threadIdx.x >> 5] = make_float2(mean[r], sq[r]);
      }
      group_sync(group, T);
      constexpr int kLanes = R == 1 ? 32 : 16;
      const float2 q = w_of < W ? part[slot][R == 1 ? 0 : high][group * W + w_of] : make_float2(0.0f, 0.0f);
      const float m = quotient(warp_sum<kLanes>(q.x * theirs), (float)K, per_k);
      const float v = warp_sum<kLanes>(fmaf((q.x - m) * theirs, q.x - m, q.y));
      mean[0] = m;
      sq[0] = v;
      if constexpr (R == 2) {
        const float m2 = __shfl_xor_sync(0xFFFFFFFFu, m, 16), v2 = __shfl_xor_sync(0xFFFFFFFFu, v, 16);
        mean[0] = high ? m2 : m;
        mean[R - 1] = high ? m : m2;
        sq[0] = high ? v2 : v;
        sq[R - 1] = high ? v : v2;
      }
    } else {
      __syncwarp();
    }
    request(row + S * step, rows.stage);
    rows.next();
    if constexpr (QUANT) {
      if (a.x_codes) store_codes<R, P, FULL>(x, lane, a.x_codes, a.x_scales_out, a.M, K, row, col);
    }
    uint64_t minus[R], r2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float rstd = __frsqrt_rn(fmaf(sq[r], per_k, a.eps));
      if (t == 0 && row + r < a.M) store_stats(a, row + r, mean[r], rstd);
      minus[r] = pair(-mean[r]);
      r2[r] = pair(rstd);
    }
    const int64_t at = row * K + col;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (!there(p)) continue;  // zeros
      uint64_t w[4], b[4];
      Param::read(w_at, p, w);
      Param::read(b_at, p, b);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint64_t(&y)[4] = x[r * P + p];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = fma_pair(mul_pair(add_pair(y[j], minus[r]), r2[r]), w[j], b[j]);
        if constexpr (!QUANT) {
          if (row + r >= a.M) continue;
          store_run(a.y, y_f32, at + (int64_t)r * K + p * 256, y);
        }
      }
    }
    if constexpr (QUANT) store_codes<R, P, FULL>(x, lane, a.codes, a.scales, a.M, K, row, col);
  }
}

// The same, to the bit, for few rows: a CTA's one row and its parameters come straight to registers, all of them at
// once. One row of 8192 into codes 2.7 us, 64 rows 3.1, most of it the wait for memory and two sums.
template <bool XF32, int P, bool QUANT>
__global__ void __launch_bounds__(kNormThreads) norm_row_kernel(NormArgs a) {
  __shared__ float2 part[kNormThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int W = blockDim.x / 32, K = (int)a.K, lane = threadIdx.x & 31, wi = threadIdx.x >> 5;
  const int col = wi * (P * 256) + lane * 8;
  const int64_t row = blockIdx.x, at = row * K + col;
  auto there = [&](int p) { return col + p * 256 < K; };
  uint64_t x[P][4], w[P][4], b[P][4];
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[p][j] = b[p][j] = 0u;
      w[p][j] = pair(1.0f);
    }
    if (there(p)) load_run(static_cast<const char*>(a.x) + (at + p * 256) * (XF32 ? 4 : 2), XF32, x[p]);
  }
  const int w_size = a.w_type == kTypeFp32 ? 4 : 2;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (!there(p)) continue;
    const int64_t from = (int64_t)(col + p * 256) * w_size;
    if (a.weight) load_run(static_cast<const char*>(a.weight) + from, w_size == 4, w[p]);
    if (a.bias) load_run(static_cast<const char*>(a.bias) + from, w_size == 4, b[p]);
  }
  auto count = [&](int k) { return (float)min(max(K - k * (P * 256), 0), P * 256); };  // columns of warp k
  const float per_k = __fdiv_rn(1.0f, (float)K);
  uint64_t s[2] = {x[0][0], x[0][1]};
#pragma unroll
  for (int i = 2; i < 4 * P; ++i) s[i & 1] = add_pair(s[i & 1], x[i / 4][i % 4]);
  s[0] = add_pair(s[0], s[1]);
  float mean = warp_sum(lo_of(s[0]) + hi_of(s[0]));
  mean = a.center ? quotient(mean, count(wi), __fdiv_rn(1.0f, count(wi))) : 0.0f;
  uint64_t minus = pair(-mean);
  s[0] = s[1] = 0u;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (!there(p)) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t d = add_pair(x[p][j], minus);
      s[j & 1] = fma_pair(d, d, s[j & 1]);
    }
  }
  s[0] = add_pair(s[0], s[1]);
  float sq = warp_sum(lo_of(s[0]) + hi_of(s[0]));
  if (W > 1) {
    if (lane == 0) part[wi] = make_float2(mean, sq);
    __syncthreads();
    const float theirs = lane < W ? count(lane) : 0.0f;
    const float2 q = lane < W ? part[lane] : make_float2(0.0f, 0.0f);
    mean = quotient(warp_sum(q.x * theirs), (float)K, per_k);
    sq = warp_sum(fmaf((q.x - mean) * theirs, q.x - mean, q.y));
  }
  const float rstd = __frsqrt_rn(fmaf(sq, per_k, a.eps));
  if (threadIdx.x == 0) store_stats(a, row, mean, rstd);
  if constexpr (QUANT) {
    if (a.x_codes) store_codes<1, P, false>(x, lane, a.x_codes, a.x_scales_out, a.M, K, row, col);
  }
  minus = pair(-mean);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (!there(p)) continue;  // zeros
#pragma unroll
    for (int j = 0; j < 4; ++j) x[p][j] = fma_pair(mul_pair(add_pair(x[p][j], minus), pair(rstd)), w[p][j], b[p][j]);
    if constexpr (!QUANT) store_run(a.y, a.y_type == kTypeFp32, at + p * 256, x[p]);
  }
  if constexpr (QUANT) store_codes<1, P, false>(x, lane, a.codes, a.scales, a.M, K, row, col);
}

// The same for rows of any length and alignment: 512 columns a warp, 16 a lane, loaded and
// stored one by one; up to 8192 columns the parameters stay in registers (they would be half of the loads) and the
// next row is on its way. 3000 x 7777 bf16 31.5 us (14 of bytes), 56 without both; with the parameters in shared
// memory and 32 warps 32.5. 23 instructions for a value (11 in packed pairs and wide loads), issued in 45 % of the
// cycles by 16 warps. Longer rows, 32 warps of 64 registers that spill 8 bytes and load the parameters with every row:
// 2000 x 9999 40 us (12 of bytes).
template <bool XF32, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_any_kernel(NormArgs a, int W) {
  constexpr int kWarps = THREADS / 32;
  constexpr bool kKeep = THREADS <= 512;
  __shared__ float2 part[2][kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int T = 32 * W, group = threadIdx.x / T, t = threadIdx.x - group * T, K = (int)a.K;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / T);
  int64_t row = (int64_t)blockIdx.x * (blockDim.x / T) + group;
  auto count = [&](int w) { return (float)min(max(K - w * 512, 0), 512); };  // columns of the group's warp w
  const int lane = threadIdx.x & 31, col = (t >> 5) * 512 + lane, left = K - col;
  const float mine = count(t >> 5), theirs = lane < W ? count(lane) : 0.0f;
  const bool w_f32 = a.w_type == kTypeFp32, y_f32 = a.y_type == kTypeFp32;
  float x[16], w[16], b[16];
  uint32_t raw[16];
  auto load = [&](int64_t at) {
    load_values(static_cast<const char*>(a.x) + (at * K + col) * (XF32 ? 4 : 2), XF32, left, raw);
  };
  auto params = [&] {
    load_params(a.weight, w_f32, col, left, 1.0f, w);
    load_params(a.bias, w_f32, col, left, 0.0f, b);
  };
  if constexpr (kKeep) {
    if (row < a.M) load(row);
    params();
  }
  for (int slot = 0; row < a.M; row += step, slot ^= 1) {
    if constexpr (!kKeep) load(row);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = value_of(raw[i], XF32);
    if (kKeep && row + step < a.M) load(row + step);
    float mean = 0.0f;
    if (a.center) {
      float s[2] = {};
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i & 1] += x[i];
      mean = mine > 0.0f ? __fdiv_rn(warp_sum(s[0] + s[1]), mine) : 0.0f;
    }
    float s[2] = {};
    for_values<16>(left, [&](int i) { s[i & 1] = fmaf(x[i] - mean, x[i] - mean, s[i & 1]); });
    float sq = warp_sum(s[0] + s[1]);
    if (W > 1) {  // the warps' sums about their own means, joined with the means' distances from the row's
      if (lane == 0) part[slot][threadIdx.x >> 5] = make_float2(mean, sq);
      group_sync(group, T);
      const float2 q = lane < W ? part[slot][group * W + lane] : make_float2(0.0f, 0.0f);
      mean = __fdiv_rn(warp_sum(q.x * theirs), (float)K);
      sq = warp_sum(fmaf((q.x - mean) * theirs, q.x - mean, q.y));
    }
    const float rstd = deviation(a, sq);
    if (t == 0) store_stats(a, row, mean, rstd);
    if constexpr (!kKeep) params();
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fmaf((x[i] - mean) * rstd, w[i], b[i]);
    store_values(static_cast<char*>(a.y) + (row * K + col) * (y_f32 ? 4 : 2), y_f32, left, x);
  }
}

// ------------------------------------------------------------------------------------------
// backward
// ------------------------------------------------------------------------------------------
// Rows of x and dy on their way into a group's shared memory, one bulk copy each; a lane reads four runs of 8
// columns, 256 apart from `col` on.
template <int XT, bool DYF32>
struct NormRing {
  static constexpr int kRuns = 4, kX = XT == kTypeB128 ? 8 : XT == kTypeFp32 ? 32 : 16, kDy = DYF32 ? 32 : 16;
  // bytes of shared memory per thread: the weights (of a group) in fp32, and for each stage its columns of
  // both with a scale per block of 128
  static constexpr int kWeights = ParamRuns<kRuns>::kBytes, kStage = kRuns * (kX + kDy) + (XT == kTypeB128 ? 1 : 0);

  uint32_t sm;  // this group's stages
  int t, T, K, col;

  __device__ __forceinline__ uint32_t x_at(int stage) const { return sm + stage * kStage * T; }
  __device__ __forceinline__ uint32_t dy_at(int stage) const { return x_at(stage) + kRuns * T * kX; }
  __device__ __forceinline__ uint32_t scale_at(int stage) const { return dy_at(stage) + kRuns * T * kDy; }

  // Asks for a row: called by all of the group, once the stage has been read by all of them.
  __device__ __forceinline__ void request(const NormArgs& a, const RowStages& rows, int64_t row, int stage) const {
    if (row >= a.M) return;
    const uint32_t bar = rows.bar(stage);
    if (rows.failed) {
      if (XT == kTypeB128) tc::mbar_arrive(bar);
      if (t == 0) tc::mbar_arrive(bar);
      return;
    }
    if constexpr (XT == kTypeB128) {
      if (t < (K + kB128 - 1) / kB128) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(scale_at(stage) + t * 4),
                     "l"(a.x_scales + t * a.M + row)
                     : "memory");
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
    }
    if (t == 0) {
      const uint32_t xb = K / 8 * kX, dyb = K / 8 * kDy;
      tc::mbar_arrive_expect_tx(bar, xb + dyb);
      bulk_copy(x_at(stage), static_cast<const char*>(a.x) + row * xb, xb, bar);
      bulk_copy(dy_at(stage), static_cast<const char*>(a.y) + row * dyb, dyb, bar);
    }
  }
  // A run of x and its dy. Of a checkpoint not its values but (code scale rstd) f + less in one operation, with f
  // and less of the row: a value is rounded with what is done to it, not on its own.
  __device__ __forceinline__ void read(int stage, int c, float rstd, float f, uint64_t less, uint64_t* x,
                                       uint64_t* dy) const {
    if constexpr (XT == kTypeB128) {
      uint32_t lo, hi;
      float s;
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(lo), "=r"(hi) : "r"(x_at(stage) + col + c * 256));
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(s) : "r"(scale_at(stage) + col / kB128 * 4 + c * 8));
      values4(lo, x[0], x[1]);
      values4(hi, x[2], x[3]);
      const uint64_t by = pair(s * rstd * f);  // (rstd f, or rstd^2, may be beyond fp32 where this is not)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = fma_pair(x[j], by, less);
    } else {
      read8<XT == kTypeFp32>(x_at(stage) + (col + c * 256) * (kX / 8), x);
    }
    read8<DYF32>(dy_at(stage) + (col + c * 256) * (kDy / 8), dy);
  }
};

// Two sums over the row of a group of W warps (slot: of two, taken in turn): the two halves of a warp take one
// each, so that five exchanges do for both.
__device__ __forceinline__ void row_sums(float (&part)[2][2][kNormThreads / 32], int slot, int group, int W,
                                         float& s1, float& s2) {
  const int lane = threadIdx.x & 31, half = lane >> 4;
  float mine = half ? s2 : s1;
  mine += __shfl_xor_sync(0xFFFFFFFFu, half ? s1 : s2, 16);
  mine = warp_sum<16>(mine);
  if (W == 1) {
    __syncwarp();
  } else {
    const int i = lane & 15;
    if (i == 0) part[slot][half][threadIdx.x >> 5] = mine;
    group_sync(group, 32 * W);
    mine = warp_sum<16>(i < W ? part[slot][half][group * W + i] : 0.0f);
  }
  const float other = __shfl_xor_sync(0xFFFFFFFFu, mine, 16);
  s1 = half ? other : mine;
  s2 = half ? mine : other;
}

// Where this CTA's share of a gradient (k: 0 dw, 1 db) goes: its row of the workspace, or of a single CTA the
// gradient itself.
__device__ __forceinline__ float* share(const NormArgs& a, int k) {
  float* whole = k ? a.dbias : a.dweight;
  return !whole || gridDim.x == 1 ? whole : a.workspace + (k * (int64_t)gridDim.x + blockIdx.x) * a.K;
}
// Adds up the groups' rows [2][groups][K] in shared memory (first dw's, then db's), in their order.
__device__ __forceinline__ void join_shares(const NormArgs& a, const float* sm, int groups) {
  const int K = (int)a.K;
  __syncthreads();
  constexpr int kAhead = 4;  // columns of a thread whose reads are on their way together
  const int threads = blockDim.x;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(sm);
  for (int k = 0; k < 2; ++k) {
    float* out = share(a, k);
    if (!out) continue;
    for (int col0 = threadIdx.x; col0 < K; col0 += kAhead * threads) {
      float s[kAhead] = {};
#pragma unroll 2
      for (int i = 0; i < groups; ++i) {
        const uint32_t at = base + ((k * groups + i) * K + col0) * 4;
        float v[kAhead] = {};
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (col0 + j * threads >= K) continue;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[j]) : "r"(at + j * threads * 4));
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) s[j] += v[j];
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (col0 + j * threads < K) out[col0 + j * threads] = s[j];
      }
    }
  }
}

// Gradient of the input, and each CTA's share of the parameters' gradients, which norm_reduce_kernel adds up.
// Groups of W warps walk rows, their sums of dw and db in registers, the next rows on their way into the group's
// stages, the weights in shared memory. A row is read from its stage twice, for the sums over it and for dx: dw
// and db leave no registers to keep it in (8192 x 8192 from a checkpoint with xhat kept in shared memory in
// between: 77 -> 87 us). Two groups and more work beside each other up to 8192 columns, one while the other waits
// for its sums; one alone has 4096 x 16384 in 100 us for 60 of bytes. From a checkpoint bound by its instructions,
// 22 for a value, issued in 58 % of the cycles; the parameters' gradients cost 6 us, for the groups' join, the
// shares and the launch that adds them up.
// MODE: K is a multiple of a warp's 1024 columns or not; or, of any such K, no more rows than CTAs: one group a
// CTA, whose sums leave its registers as its share (one row of 8192 6.0 -> 4.3 us; as a branch of the others it
// cost them registers, 8192 x 8192 bf16 68.6 -> 72.5).
constexpr int kAnyCols = 0, kFullCols = 1, kSingleRows = 2;
template <int XT, bool DYF32, int MODE>
__global__ void __launch_bounds__(kNormThreads, 1) norm_backward_kernel(NormArgs a, int W, int S) {
  extern __shared__ __align__(16) uint8_t ring_shared[];
  using Ring = NormRing<XT, DYF32>;
  constexpr int C = Ring::kRuns;
  __shared__ float part[2][2][kNormThreads / 32];
  __shared__ __align__(8) uint64_t full[kNormThreads / 32][kMaxStages];
  const int T = 32 * W, group = threadIdx.x / T, t = threadIdx.x - group * T, K = (int)a.K;
  const int col = (t >> 5) * 1024 + (threadIdx.x & 31) * 8;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(ring_shared);
  const Ring ring{base + T * Ring::kWeights + group * T * S * Ring::kStage, t, T, K, col};
  RowStages rows(full[group], S, S > 1 ? S - 1 : 1);
  if (t == 0) rows.init(XT == kTypeB128 ? T + 1 : 1);
  pdl_launch_dependents();
  __syncthreads();
  pdl_wait();
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / T);
  int64_t row = (int64_t)blockIdx.x * (blockDim.x / T) + group;
  for (int s = 0; s < rows.ahead; ++s) ring.request(a, rows, row + s * step, s);
  using Param = ParamRuns<C>;
  const uint32_t w_at = Param::at(base, t >> 5, threadIdx.x & 31);
  if (group == 0) Param::store(w_at, a.weight, a.w_type == kTypeFp32, col, K, 1.0f);
  __syncthreads();
  const bool dx_f32 = a.dx_type == kTypeFp32;
  const float per_k = __fdiv_rn(1.0f, (float)K);
  auto there = [&](int c) { return MODE == kFullCols || col + c * 256 < K; };

  uint64_t dw[C][4], db[C][4];
#pragma unroll
  for (int i = 0; i < 4 * C; ++i) dw[i / 4][i % 4] = db[i / 4][i % 4] = 0u;
  float mean_next = 0.0f, rstd_next = 0.0f;
  if (row < a.M) {
    rstd_next = load_f32(a.rstd + row);
    if (a.mean) mean_next = load_f32(a.mean + row);
  }
  for (int slot = 0; row < a.M; row += step, slot ^= 1) {
    const int stage = rows.stage;
    constexpr bool kFold = XT == kTypeB128;
    const float rstd = rstd_next, mean = mean_next;
    const uint64_t minus = pair(-mean), r2 = pair(rstd), less = pair(-mean * rstd);
    if (row + step < a.M) {
      rstd_next = load_f32(a.rstd + row + step);
      if (a.mean) mean_next = load_f32(a.mean + row + step);
    }
    rows.wait(a, row, step);
    uint64_t c1 = 0u, c2 = 0u;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!there(c)) continue;
      uint64_t x[4], y[4], w[4];
      ring.read(stage, c, rstd, 1.0f, less, x, y);
      Param::read(w_at, c, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (!kFold) x[j] = mul_pair(add_pair(x[j], minus), r2);
        dw[c][j] = fma_pair(y[j], x[j], dw[c][j]);
        db[c][j] = add_pair(db[c][j], y[j]);
        y[j] = mul_pair(y[j], w[j]);
        c1 = add_pair(c1, y[j]);
        c2 = fma_pair(y[j], x[j], c2);
      }
    }
    float s1 = lo_of(c1) + hi_of(c1), s2 = lo_of(c2) + hi_of(c2);
    row_sums(part, slot, group, W, s1, s2);
    // all of the group have read the row before this one for the last time
    if (S > 1) ring.request(a, rows, row + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);
    // dx = rstd g - rstd s1 - xhat rstd s2
    const float c0 = a.mean ? -s1 * per_k * rstd : 0.0f, cx = -s2 * per_k * rstd;
    const uint64_t m1 = pair(c0), m2 = pair(cx), rest = pair(fmaf(lo_of(less), cx, c0));
    const int64_t at = row * K + col;
    // (fp32 rows one run at a time: with the runs beside each other registers spill, 8192 x 8192 109 -> 112 us; bf16
    // rows and checkpoints lose without, 4096 x 16384 97 -> 99 and 76 -> 83)
    constexpr int kBeside = XT == kTypeFp32 ? 1 : C;
#pragma unroll kBeside
    for (int c = 0; c < C; ++c) {
      if (!there(c)) continue;
      uint64_t x[4], y[4], w[4];
      ring.read(stage, c, rstd, cx, rest, x, y);
      Param::read(w_at, c, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (!kFold) x[j] = fma_pair(mul_pair(add_pair(x[j], minus), r2), m2, m1);
        y[j] = fma_pair(mul_pair(y[j], w[j]), r2, x[j]);
      }
      uint32_t o[8];
      if (dx_f32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[2 * j] = __float_as_uint(lo_of(y[j]));
          o[2 * j + 1] = __float_as_uint(hi_of(y[j]));
        }
        store16B(static_cast<float*>(a.dx) + at + c * 256, o);
        store16B(static_cast<float*>(a.dx) + at + c * 256 + 4, o + 4);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = bf16_word(y[j]);
        store16B(static_cast<uint16_t*>(a.dx) + at + c * 256, o);
      }
    }
    if (S == 1) {
      group_sync(group, T);
      ring.request(a, rows, row + step, 0);
    }
    rows.next();
  }
  if (!a.dweight && !a.dbias) return;
  if constexpr (MODE == kSingleRows) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float* to = share(a, k);
      if (!to) continue;
      const bool wide = (reinterpret_cast<uintptr_t>(to) & 31) == 0;
      to += col;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (!there(c)) continue;
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          o[2 * j] = __float_as_uint(lo_of(k ? db[c][j] : dw[c][j]));
          o[2 * j + 1] = __float_as_uint(hi_of(k ? db[c][j] : dw[c][j]));
        }
        if (wide) {
          store32B(to + c * 256, o);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) to[c * 256 + j] = __uint_as_float(o[j]);
        }
      }
    }
    return;
  }
  // through shared memory, one group too
  const int groups = blockDim.x / T;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* to = reinterpret_cast<float*>(ring_shared) + (k * groups + group) * K + col;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (!there(c)) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint64_t p = k ? db[c][2 * j] : dw[c][2 * j], q = k ? db[c][2 * j + 1] : dw[c][2 * j + 1];
        *reinterpret_cast<float4*>(to + c * 256 + 4 * j) = make_float4(lo_of(p), hi_of(p), lo_of(q), hi_of(q));
      }
    }
  }
  join_shares(a, reinterpret_cast<const float*>(ring_shared), groups);
}

// The same for rows of any length and alignment: 32 N columns a warp, N a lane, loaded one by one; up to 8192
// columns (16 values) with the weights in registers and the next row on its way: 3000 x 7777 bf16 55 us (21 of
// bytes), 130 without both. A lane's columns a group's width apart, asked for one by one, took 73 us. 32 instructions
// for a value, issued in 38 % of the cycles; 164 bytes of registers are spilled. With 32 values (over 8192 columns, 708
// bytes spilled) 2000 x 9999 take 90 us (18 of bytes).
template <int N>
__global__ void __launch_bounds__(kNormThreads, 1) norm_backward_any_kernel(NormArgs a, int W, int) {
  extern __shared__ __align__(16) uint8_t ring_shared[];
  __shared__ float part[2][2][kNormThreads / 32];
  constexpr bool kKeep = N <= 16;
  pdl_launch_dependents();
  pdl_wait();
  const int T = 32 * W, group = threadIdx.x / T, t = threadIdx.x - group * T, K = (int)a.K;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x / T);
  int64_t row = (int64_t)blockIdx.x * (blockDim.x / T) + group;
  const bool x_f32 = a.x_type == kTypeFp32, dy_f32 = a.y_type == kTypeFp32, dx_f32 = a.dx_type == kTypeFp32;
  const bool codes = a.x_type == kTypeB128, w_f32 = a.w_type == kTypeFp32;
  const float per_k = __fdiv_rn(1.0f, (float)K);
  const int col = (t >> 5) * (32 * N) + (threadIdx.x & 31), left = K - col;
  float dw[N], db[N], w[N];
  uint32_t x[N], dy[N];
  auto load = [&](int64_t at) {
    const char* from = static_cast<const char*>(a.x) + (at * K + col) * (codes ? 1 : x_f32 ? 4 : 2);
    if (codes) {
      const float* scales = a.x_scales + (int64_t)(t >> 5) * (32 * N / kB128) * a.M + at;
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = 0u;
      for_values<N>(left, [&](int i) {
        float lo, hi;
        e4m3x2_to_f32(load_u8(from + i * 32), lo, hi);
        x[i] = __float_as_uint(__fmul_rn(lo, load_f32(scales + i / 4 * a.M)));
      });
    } else {
      load_values(from, x_f32, left, x);
    }
    load_values(static_cast<const char*>(a.y) + (at * K + col) * (dy_f32 ? 4 : 2), dy_f32, left, dy);
  };
#pragma unroll
  for (int i = 0; i < N; ++i) dw[i] = db[i] = 0.0f;
  if constexpr (kKeep) {
    if (row < a.M) load(row);
    load_params(a.weight, w_f32, col, left, 1.0f, w);
  }
  for (int slot = 0; row < a.M; row += step, slot ^= 1) {
    const float rstd = load_f32(a.rstd + row), mean = a.mean ? load_f32(a.mean + row) : 0.0f;
    if constexpr (!kKeep) {
      load(row);
      load_params(a.weight, w_f32, col, left, 1.0f, w);
    }
    float xh[N], g[N], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {  // (dy is 0 where there is no column)
      xh[i] = (value_of(x[i], codes || x_f32) - mean) * rstd;
      g[i] = value_of(dy[i], dy_f32);
      dw[i] = fmaf(g[i], xh[i], dw[i]);
      db[i] += g[i];
      g[i] *= w[i];
      s1 += g[i];
      s2 = fmaf(g[i], xh[i], s2);
    }
    if constexpr (kKeep) {
      if (row + step < a.M) load(row + step);
    }
    row_sums(part, slot, group, W, s1, s2);
    s1 = a.mean ? s1 * per_k : 0.0f;
    s2 *= per_k;
#pragma unroll
    for (int i = 0; i < N; ++i) g[i] = fmaf(-xh[i], s2, g[i] - s1) * rstd;
    store_values(static_cast<char*>(a.dx) + (row * K + col) * (dx_f32 ? 4 : 2), dx_f32, left, g);
  }
  if (!a.dweight && !a.dbias) return;
  const int groups = blockDim.x / T;
  float* sm = reinterpret_cast<float*>(ring_shared);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    for_values<N>(left, [&](int i) { sm[(k * groups + group) * K + col + i * 32] = k ? db[i] : dw[i]; });
  }
  join_shares(a, sm, groups);
}

// Adds up the CTAs' shares of a parameter's gradient (blockIdx.y: which): 32 columns a CTA, the shares over 16
// warps, ten of a warp's on their way together. About 3 us, of its launch and two round trips; lanes of 2 or 4
// columns gain 0.6 us of 7.5 on 64 shares of 8192 columns and lose 0.3 of 4.9 on 2048.
__global__ void __launch_bounds__(512) norm_reduce_kernel(NormArgs a, int parts) {
  __shared__ float sum[16][33];
  pdl_launch_dependents();
  pdl_wait();
  float* to = blockIdx.y ? a.dbias : a.dweight;
  if (!to) return;
  constexpr int kAhead = 10;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, K = (int)a.K, col = (int)blockIdx.x * 32 + lane;
  const float* from = a.workspace + (int64_t)blockIdx.y * parts * K + col;
  float s = 0.0f;
  if (col < K) {
    for (int p0 = warp; p0 < parts; p0 += 16 * kAhead) {
      float v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        v[i] = p0 + 16 * i < parts ? load_f32(from + (int64_t)(p0 + 16 * i) * K) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) s += v[i];
    }
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < K) {
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += sum[i][lane];
    to[col] = s;
  }
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Groups of a CTA of `most` threads that rows of W warps and their shared memory leave room for: `fixed` bytes
// once and `stage` bytes per group for each of `stages` rows on their way (most of at most kMaxStages).
struct Groups {
  int count, stages;
  size_t smem;
};
Groups fit_groups(int most, int W, size_t fixed, size_t stage) {
  Groups g{most / 32 / W, 0, 0};
  while (g.count > 1 && fixed + g.count * stage > kNormSmem) --g.count;
  if (fixed + g.count * stage > kNormSmem) return Groups{0, 0, 0};
  g.stages = stage ? (int)((kNormSmem - fixed) / (g.count * stage)) : 0;
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  g.smem = fixed + g.count * stage * g.stages;
  return g;
}

// Few rows go to as many CTAs as there are: `count` groups of a CTA, or as many as M rows need at `slots` a round
// (gradients of 64 rows of 1024 8.0 -> 5.0 us, of 8192 9.7 -> 7.7).
int spread(int count, int64_t M, int64_t slots) {
  const int64_t need = (M + slots - 1) / slots;
  return need < count ? (int)need : count;
}

template <bool XF32, int P, int R, bool QUANT>
cudaError_t run_norm(const NormArgs& a, cudaStream_t stream) {
  const int W = (int)((a.K + P * 256 - 1) / (P * 256));
  const auto kernel =
      a.K % (P * 256) == 0 ? &norm_kernel<XF32, P, R, QUANT, true> : &norm_kernel<XF32, P, R, QUANT, false>;
  // Rows that are all resident at once, at most 8 an SM, go by the kernel without shared memory for rows and
  // parameters (into bf16: 1 x 8192 3.5 -> 2.5 us, 300 x 8192 4.6 -> 4.2, but 600 x 8192 6.3 -> 7.6; 1200 x 1024 3.3 ->
  // 2.9, 2400 x 1024 4.2 -> 4.5).
  const auto row = &norm_row_kernel<XF32, P, QUANT>;
  if (a.M <= resident_ctas(reinterpret_cast<const void*>(row), 32 * W, 0, 8)) {
    return launch_pdl(row, dim3((unsigned)a.M), dim3(32 * W), 0, stream, a);
  }
  const Groups g = fit_groups(kNormThreads, W, (size_t)64 * W * ParamRuns<P>::kBytes,
                              (size_t)32 * W * R * P * 8 * (XF32 ? 4 : 2));
  // two rows of more than 14336 columns of fp32 do not fit beside their parameters
  if constexpr (R > 1 && P == 4 && XF32) {
    if (!g.count) return run_norm<XF32, P, 1, QUANT>(a, stream);
  }
  if (!g.count) return cudaErrorInvalidConfiguration;
  const int64_t slots = resident_ctas(reinterpret_cast<const void*>(kernel), 32 * W * g.count, g.smem, 1);
  if (slots <= 0) return cudaErrorInvalidConfiguration;
  const int count = spread(g.count, a.M, R * slots);
  const int64_t ctas = (a.M + count * R - 1) / (count * R);
  return launch_pdl(kernel, dim3((unsigned)(ctas < slots ? ctas : slots)), dim3(32 * W * count), g.smem, stream, a,
                    W, g.stages);
}
// Rows of up to 512 columns are one warp's with one or two runs per lane; longer ones a group's with four.
template <bool XF32, bool QUANT>
cudaError_t run_norm(const NormArgs& a, cudaStream_t stream) {
  if (a.K <= 256) return run_norm<XF32, 1, 2, QUANT>(a, stream);
  return a.K <= 512 ? run_norm<XF32, 2, 2, QUANT>(a, stream) : run_norm<XF32, 4, 2, QUANT>(a, stream);
}

cudaError_t run_any(void (*kernel)(NormArgs, int), const NormArgs& a, int W, cudaStream_t stream) {
  const int most = W >= 16 ? 1 : 16 / W;
  const int64_t slots = resident_ctas(reinterpret_cast<const void*>(kernel), 32 * W * most, 0, 0);
  if (slots <= 0) return cudaErrorInvalidConfiguration;
  const int count = spread(most, a.M, slots);
  const int64_t ctas = (a.M + count - 1) / count;
  return launch_pdl(kernel, dim3((unsigned)(ctas < slots ? ctas : slots)), dim3(32 * W * count), 0, stream, a, W);
}

template <bool XF32>
cudaError_t pick_norm(const NormArgs& a, bool vec, cudaStream_t stream) {
  if (a.codes) return run_norm<XF32, true>(a, stream);
  if (vec) return run_norm<XF32, false>(a, stream);
  const int W = (int)((a.K + 511) / 512);
  return run_any(W <= 16 ? &norm_any_kernel<XF32, 512> : &norm_any_kernel<XF32, 1024>, a, W, stream);
}

// `cols` columns of a row per warp; bytes of shared memory per thread of a group once, and per thread and stage.
// single: the kernel for no more rows than CTAs, or null.
using BackwardKernel = void (*)(NormArgs, int, int);
cudaError_t run_backward(BackwardKernel kernel, BackwardKernel single, int fixed, int stage, const NormArgs& a,
                         int cols, cudaStream_t stream) {
  const int W = (int)((a.K + cols - 1) / cols);
  Groups g = fit_groups(kNormThreads, W, (size_t)fixed * 32 * W, (size_t)stage * 32 * W);
  if (!g.count) return cudaErrorInvalidConfiguration;
  const bool params = a.dweight || a.dbias;
  if (params && g.smem < (size_t)g.count * a.K * 8) g.smem = (size_t)g.count * a.K * 8;  // the groups' shares
  int64_t slots = resident_ctas(reinterpret_cast<const void*>(kernel), 32 * W * g.count, g.smem, 1);
  if (single && a.M <= slots) {
    kernel = single;
    slots = resident_ctas(reinterpret_cast<const void*>(kernel), 32 * W * g.count, g.smem, 1);
  }
  if (slots <= 0) return cudaErrorInvalidConfiguration;
  const int count = spread(g.count, a.M, slots);
  int64_t ctas = (a.M + count - 1) / count;
  if (ctas > slots) ctas = slots;
  if (params && ctas > kMaxParts) ctas = kMaxParts;
  const cudaError_t err =
      launch_pdl(kernel, dim3((unsigned)ctas), dim3(32 * W * count), g.smem, stream, a, W, g.stages);
  if (err != cudaSuccess || !params || ctas == 1) return err;
  return launch_pdl(&norm_reduce_kernel, dim3((unsigned)((a.K + 31) / 32), 2), dim3(512), 0, stream, a,
                    (int)ctas);
}

template <int XT, bool DYF32>
cudaError_t run_ring(const NormArgs& a, cudaStream_t stream) {
  using Ring = NormRing<XT, DYF32>;
  return run_backward(a.K % 1024 == 0 ? &norm_backward_kernel<XT, DYF32, kFullCols>
                                      : &norm_backward_kernel<XT, DYF32, kAnyCols>,
                      &norm_backward_kernel<XT, DYF32, kSingleRows>, Ring::kWeights, Ring::kStage, a, 1024, stream);
}

cudaError_t pick_ring(const NormArgs& a, cudaStream_t stream) {
  const bool dy_f32 = a.y_type == kTypeFp32;
  if (a.x_type == kTypeBf16) {
    return dy_f32 ? run_ring<kTypeBf16, true>(a, stream) : run_ring<kTypeBf16, false>(a, stream);
  }
  if (a.x_type == kTypeFp32) {
    return dy_f32 ? run_ring<kTypeFp32, true>(a, stream) : run_ring<kTypeFp32, false>(a, stream);
  }
  return dy_f32 ? run_ring<kTypeB128, true>(a, stream) : run_ring<kTypeB128, false>(a, stream);
}

}  // namespace

int64_t norm_workspace_floats(int64_t M, int64_t K) { return 2 * (M < kMaxParts ? M : kMaxParts) * K; }

cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream) {
  const bool vec = a.codes || (a.K % 8 == 0 && aligned_to(a.x, 32) && aligned_to(a.y, 32) &&
                               aligned_to(a.weight, 32) && aligned_to(a.bias, 32));
  return a.x_type == kTypeFp32 ? pick_norm<true>(a, vec, stream) : pick_norm<false>(a, vec, stream);
}

cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t stream) {
  const bool vec = a.K % 8 == 0 && aligned_to(a.x, 16) && aligned_to(a.y, 16) && aligned_to(a.dx, 16) &&
                   aligned_to(a.weight, 32);
  if (vec) return pick_ring(a, stream);
  return a.K <= 8192 ? run_backward(&norm_backward_any_kernel<16>, nullptr, 0, 0, a, 512, stream)
                     : run_backward(&norm_backward_any_kernel<32>, nullptr, 0, 0, a, 1024, stream);
}

}  // namespace mxq
