// mx_combine.cu -- joining the experts' outputs: out[t] = sum_j w[t, j] y[slot[t, j]], and its
// gradient dy[slot] = w dout[t], dw[t, j] = <dout[t], y[slot]>. A slot of -1 (no expert) takes and
// gives nothing. Sums are in fp32 in the order of j; each output is rounded to bf16 once.
// Without weights (all ones) the forward is the gradient of gathering rows by token.
//
// Bound by memory: every chosen row is read once (16-byte loads, up to eight rows in flight per
// thread), every output row written once. The backward walks tokens, not rows, so that dout is
// read once and not k times. 16384 tokens with 8 rows of 2048 each: 96 us (6.3 TB/s), the gradients
// 190 us (6.0 TB/s).
//
// Rows of dy that no slot names have a gradient of zero. Which these are, the walk over tokens does not
// see: it leaves the number of the choice at its row's place in a workspace, and a second kernel takes a
// row for named where the choice noted there does name it, which needs no workspace cleared before. That
// costs a launch and the reads of the workspace and the choices (131072 rows, none of them zeroed: 2.5 us).
#include "mx_device.cuh"
#include "mx_expert.h"
#include "mx_launch.h"

namespace mxq {

namespace {

constexpr int kCombineThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// Written once, not read again here: evict-first (324 -> 287 us for forward and backward of 16384
// tokens, 8 rows of 2048 each).
__device__ __forceinline__ void store4(void* p, const uint32_t* r) {
  asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

// One item = eight columns of one token; KU choices are loaded together.
template <int KU>
__global__ void __launch_bounds__(kCombineThreads, 3) combine_kernel(CombineArgs a, int64_t chunks,
                                                                  int64_t items) {
  pdl_launch_dependents();
  pdl_wait();
  const uint16_t* y = static_cast<const uint16_t*>(a.y);
  for (int64_t it = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x; it < items;
       it += (int64_t)gridDim.x * kCombineThreads) {
    const int64_t t = it / chunks, col = it % chunks * 8;
    float acc[8] = {};
    for (int j0 = 0; j0 < a.k; j0 += KU) {
      uint32_t v[KU][4];
      float w[KU];
      int32_t row[KU];  // -1: none
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        row[u] = j0 + u < a.k ? load_s32(a.slots + t * a.k + j0 + u) : -1;
        if (row[u] >= a.R) row[u] = -1;
      }
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        if (row[u] >= 0) load16B(y + row[u] * a.N + col, v[u]);
      }
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        w[u] = j0 + u < a.k && a.weights ? load_f32(a.weights + t * a.k + j0 + u) : 1.0f;
      }
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        if (row[u] < 0) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[2 * i] = fmaf(w[u], bf16_lo(v[u][i]), acc[2 * i]);
          acc[2 * i + 1] = fmaf(w[u], bf16_hi(v[u][i]), acc[2 * i + 1]);
        }
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16(acc[2 * i], acc[2 * i + 1]);
    store4(static_cast<uint16_t*>(a.out) + t * a.N + col, o);
  }
}

// One CTA per token; choices in groups of KU whose inner products a thread keeps in registers.
template <int KU>
__global__ void __launch_bounds__(kCombineThreads) combine_backward_kernel(CombineArgs a,
                                                                           int64_t chunks) {
  __shared__ float part[kCombineThreads / 32][KU];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t = blockIdx.x;
  const uint16_t* y = static_cast<const uint16_t*>(a.y);
  const uint16_t* dout = static_cast<const uint16_t*>(a.dout) + t * a.N;
  uint16_t* dy = static_cast<uint16_t*>(a.dy);
  for (int j0 = 0; j0 < a.k; j0 += KU) {
    int64_t row[KU];
    float w[KU], dot[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      row[u] = j0 + u < a.k ? load_s32(a.slots + t * a.k + j0 + u) : -1;
      w[u] = j0 + u < a.k && a.weights ? load_f32(a.weights + t * a.k + j0 + u) : 1.0f;
      dot[u] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      if (row[u] >= a.R) row[u] = -1;
      if (a.owner && tid == 0 && row[u] >= 0) a.owner[row[u]] = (int32_t)(t * a.k + j0 + u);
    }
    for (int64_t c = tid; c < chunks; c += kCombineThreads) {
      uint32_t d[4], v[KU][4];
      load16B(dout + c * 8, d);
      if (a.dweights) {
#pragma unroll
        for (int u = 0; u < KU; ++u) {
          if (row[u] >= 0) load16B(y + row[u] * a.N + c * 8, v[u]);
        }
      }
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(d[i]);
        f[2 * i + 1] = bf16_hi(d[i]);
      }
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        if (row[u] < 0) continue;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i] = pack_bf16(w[u] * f[2 * i], w[u] * f[2 * i + 1]);
          if (a.dweights) {
            dot[u] = fmaf(f[2 * i], bf16_lo(v[u][i]), dot[u]);
            dot[u] = fmaf(f[2 * i + 1], bf16_hi(v[u][i]), dot[u]);
          }
        }
        store4(dy + row[u] * a.N + c * 8, o);
      }
    }
    if (!a.dweights) continue;
#pragma unroll
    for (int u = 0; u < KU; ++u) {
#pragma unroll
      for (int s = 16; s; s >>= 1) dot[u] += __shfl_xor_sync(0xFFFFFFFFu, dot[u], s);
      if (lane == 0) part[warp][u] = dot[u];
    }
    __syncthreads();
    if (tid < KU && j0 + tid < a.k) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < kCombineThreads / 32; ++i) sum += part[i][tid];
      a.dweights[t * a.k + j0 + tid] = sum;
    }
    __syncthreads();
  }
}

// Zeros to the rows of dy whose owner is no choice that names them. A warp looks at 32 rows.
__global__ void __launch_bounds__(kCombineThreads) zero_unnamed_kernel(CombineArgs a, int64_t chunks) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t r0 = ((int64_t)blockIdx.x * kCombineThreads + threadIdx.x) - lane;
  const int64_t n = a.T * a.k, r = r0 + lane;
  bool named = true;
  if (r < a.R) {
    const int32_t o = load_s32(a.owner + r);
    named = o >= 0 && o < n && load_s32(a.slots + o) == r;
  }
  uint32_t left = __ballot_sync(0xFFFFFFFFu, !named);
  const uint32_t zeros[4] = {0u, 0u, 0u, 0u};
  while (left) {
    uint16_t* row = static_cast<uint16_t*>(a.dy) + (r0 + __ffs(left) - 1) * a.N;
    for (int64_t c = lane; c < chunks; c += 32) store4(row + c * 8, zeros);
    left &= left - 1u;
  }
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream) {
  const int64_t chunks = a.N / 8, items = a.T * chunks;
  const int64_t ctas = (items + kCombineThreads - 1) / kCombineThreads;
  const dim3 grid((unsigned)(ctas < (1 << 20) ? ctas : (1 << 20)));
  if (a.k <= 2) {
    return launch_pdl(&combine_kernel<2>, grid, dim3(kCombineThreads), 0, stream, a, chunks, items);
  }
  if (a.k <= 4) {
    return launch_pdl(&combine_kernel<4>, grid, dim3(kCombineThreads), 0, stream, a, chunks, items);
  }
  return launch_pdl(&combine_kernel<8>, grid, dim3(kCombineThreads), 0, stream, a, chunks, items);
}

cudaError_t launch_combine_backward(const CombineArgs& a, cudaStream_t stream) {
  const int64_t chunks = a.N / 8;
  const dim3 grid((unsigned)a.T), block(kCombineThreads);
  if (a.T > 0) {
    const cudaError_t err =
        a.k <= 2   ? launch_pdl(&combine_backward_kernel<2>, grid, block, 0, stream, a, chunks)
        : a.k <= 4 ? launch_pdl(&combine_backward_kernel<4>, grid, block, 0, stream, a, chunks)
                   : launch_pdl(&combine_backward_kernel<8>, grid, block, 0, stream, a, chunks);
    if (err != cudaSuccess) return err;
  }
  if (!a.owner || a.R == 0 || a.N == 0) return cudaSuccess;
  return launch_pdl(&zero_unnamed_kernel,
                    dim3((unsigned)((a.R + kCombineThreads - 1) / kCombineThreads)), block, 0, stream, a,
                    chunks);
}

}  // namespace mxq
