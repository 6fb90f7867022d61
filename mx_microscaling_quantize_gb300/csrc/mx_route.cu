// mx_route.cu -- routing of tokens to experts: scores, choice, weights, the gradient of the
// logits, and the plan that orders the chosen (token, expert) pairs by expert.
#include "mx_device.cuh"
#include "mx_expert.h"
#include "mx_launch.h"

namespace mxq {

namespace {

constexpr int kRouteWarps = 4;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if (BF16) return __uint_as_float(load_u16(static_cast<const uint16_t*>(p) + i) << 16);
  return load_f32(static_cast<const float*>(p) + i);
}

// Unsigned order of choice scores: excluded (-inf) 0, NaN next, then every number in its order.
__device__ __forceinline__ uint32_t order_key(float c) {
  const uint32_t u = __float_as_uint(__fadd_rn(c, 0.0f));  // -0 counts as +0
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0x007FFFFFu;
  if (u == 0xFF800000u) return 0u;
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {  // of a key that is a number's
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// Scores of one token, V experts per lane (expert 32 i + lane): sigmoid, or exp(l - max) with the
// sum in *total.
template <int V, bool BF16, bool SIGMOID>
__device__ __forceinline__ void token_scores(const void* logits, int64_t t, int E, float (&l)[V],
                                             float (&s)[V], float* total) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 32 * i + lane;
    l[i] = e < E ? load_logit<BF16>(logits, t * E + e) : -INFINITY;
  }
  if (SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l[i])));
    *total = 1.0f;
    return;
  }
  float m = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    m = fmaxf(m, l[i]);
    nan |= l[i] != l[i];
  }
  m = warp_max(m);
  if (m == -INFINITY) m = 0.0f;  // nothing to choose: every score is exp(-inf) = 0
  if (__any_sync(0xFFFFFFFFu, nan)) m = __uint_as_float(0x7FC00000u);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s[i] = expf(__fsub_rn(l[i], m));
    if (32 * i + lane >= E) s[i] = 0.0f;
    sum += s[i];
  }
  *total = warp_sum(sum);
}

// One warp per token. With s the scores (softmax numerators exp(l - max), or sigmoids), the
// choice c is s, or s + bias (then of the normalised softmax), and -inf where l is: such an
// expert is never chosen. Without a bias the softmax's denominator cannot change the order, so
// the choice uses the numerators and does not depend on the order of a sum.
// Groups: lane g sums group g's two largest choices (from shared memory, each lane of a
// group's share starting at another place so that the 32 lanes meet 32 banks), ranks itself
// among the groups, and a ballot names the kept ones.
// Top k: keys are unsigned images of the choices; each round is one warp-wide maximum and one
// minimum of the index among the lanes that hold it, so ties go to the lowest index, and only
// the winning lane searches its own values again.
template <int V, bool BF16, bool SIGMOID, bool GROUPS>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a, int group_size,
                                                                 uint32_t group_magic, int lanes) {
  __shared__ float score_row[kRouteWarps][V * 32];
  __shared__ float choice_row[GROUPS ? kRouteWarps : 1][GROUPS ? V * 32 : 1];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  float l[V], s[V], total;
  token_scores<V, BF16, SIGMOID>(a.logits, t, a.E, l, s, &total);
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 32 * i + lane;
    float c = s[i];
    if (a.bias && e < a.E) {
      c = __fadd_rn(SIGMOID ? c : __fdiv_rn(c, total), load_f32(a.bias + e));
    }
    if (e >= a.E || l[i] == -INFINITY) c = -INFINITY;
    key[i] = order_key(c);
    score_row[warp][e] = s[i];
    if (GROUPS) choice_row[warp][e] = c;
  }
  __syncwarp();
  if (GROUPS) {
    // lanes per group: `lanes` (a power of two, groups * lanes <= 32)
    const int g = lane / lanes, sub = lane % lanes;
    uint32_t k0 = 0u, k1 = 0u;  // keys of the two largest
    if (g < a.groups) {
      const int steps = (group_size + lanes - 1) / lanes;
      for (int it = 0; it < steps; ++it) {
        int at = it + g;
        while (at >= steps) at -= steps;
        const int j = at * lanes + sub;
        if (j < group_size) {
          const uint32_t q = order_key(choice_row[warp][g * group_size + j]);
          k1 = max(k1, min(k0, q));
          k0 = max(k0, q);
        }
      }
    }
    for (int d = 1; d < lanes; d <<= 1) {
      const uint32_t o0 = __shfl_xor_sync(0xFFFFFFFFu, k0, d);
      const uint32_t o1 = __shfl_xor_sync(0xFFFFFFFFu, k1, d);
      k1 = max(min(k0, o0), max(k1, o1));
      k0 = max(k0, o0);
    }
    // the group's score: its largest choice plus its second one where there is one
    uint32_t gk = k0;
    if (k0 > 0x007FFFFFu && k1 != 0u) {
      gk = order_key(k1 == 0x007FFFFFu ? __uint_as_float(0x7FC00000u)
                                       : __fadd_rn(key_value(k0), key_value(k1)));
    }
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
      const uint32_t other = __shfl_sync(0xFFFFFFFFu, gk, h * lanes);
      rank += other > gk || (other == gk && h < g);
    }
    const uint32_t kept = __ballot_sync(0xFFFFFFFFu, g < a.groups && rank < a.top_groups);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 32 * i + lane;
      // e / group_size: exact for e < 1024 with magic = ceil(2^32 / group_size)
      const int ge = group_size == 1 ? e : (int)__umulhi((uint32_t)e, group_magic);
      if (e < a.E && !((kept >> (ge * lanes)) & 1u)) key[i] = 0u;
    }
  }
  uint32_t best = 0u, best_e = 0u;
  auto search = [&]() {
    best = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (key[i] > best) {
        best = key[i];
        best_e = 32 * i + lane;
      }
    }
  };
  search();
  int32_t expert = -1;  // lane j: the j-th choice
  for (int j = 0; j < a.k; ++j) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    if (top == 0u) break;
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, best == top ? best_e : 0xFFFFFFFFu);
    if (lane == j) expert = (int32_t)e;
    if ((int)(e & 31u) == lane) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i == (int)(e >> 5)) key[i] = 0u;
      }
      search();
    }
  }
  float w = 0.0f;
  if (expert >= 0) {
    w = score_row[warp][expert];
    if (!SIGMOID) w = __fdiv_rn(w, total);
  }
  if (a.renormalize) {
    const float P = warp_sum(w);
    w = P == 0.0f ? 0.0f : __fdiv_rn(w, P);
  }
  if (lane < a.k) {
    a.experts[t * a.k + lane] = expert;
    a.weights[t * a.k + lane] = w * a.scale;
  }
}

// Gradient of the logits. With p the scores of the chosen experts and g the gradient of their
// weights w = scale p (/ P if renormalised, P = sum p):
//   dp_j = scale (g_j - sum_i g_i p_i / P) / P, or scale g_j;
//   sigmoid: dl = dp s (1 - s), nothing for the others;
//   softmax: dl_i = s_i (dp_i - sum_j dp_j s_j), every logit.
// A choice of -1 (no expert) takes and gives nothing. The scores are computed again from the
// logits: reading them back would cost what the logits cost.
template <int V, bool BF16, bool SIGMOID>
__global__ void __launch_bounds__(kRouteWarps * 32) route_backward_kernel(RouteArgs a) {
  __shared__ float score_row[kRouteWarps][V * 32];
  __shared__ float grad_row[kRouteWarps][V * 32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  float l[V], s[V], total;
  token_scores<V, BF16, SIGMOID>(a.logits, t, a.E, l, s, &total);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!SIGMOID) s[i] = total == 0.0f ? 0.0f : __fdiv_rn(s[i], total);
    score_row[warp][32 * i + lane] = s[i];
    grad_row[warp][32 * i + lane] = 0.0f;
  }
  __syncwarp();
  int32_t expert = -1;
  float g = 0.0f, p = 0.0f;
  if (lane < a.k) {
    expert = a.chosen[t * a.k + lane];
    if (expert >= a.E) expert = -1;
  }
  if (expert >= 0) {
    g = a.scale * a.grad_weights[t * a.k + lane];
    p = score_row[warp][expert];
  }
  if (a.renormalize) {
    const float P = warp_sum(p);
    const float along = warp_sum(g * p);
    g = P == 0.0f ? 0.0f : (g - along / P) / P;
  }
  const float through = warp_sum(expert >= 0 ? g * p : 0.0f);
  // an expert named twice (no call of the router does that) adds both
  if (expert >= 0) atomicAdd(&grad_row[warp][expert], g);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 32 * i + lane;
    if (e >= a.E) continue;
    const float d = grad_row[warp][e];
    float dl;
    if (SIGMOID) {
      dl = d * s[i] * (1.0f - s[i]);
    } else {
      dl = s[i] * (d - through);
    }
    if (BF16) {
      uint16_t h;
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(dl));
      static_cast<uint16_t*>(a.grad_logits)[t * a.E + e] = h;
    } else {
      static_cast<float*>(a.grad_logits)[t * a.E + e] = dl;
    }
  }
}

// ------------------------------------------------------------------------------------------
// plan: a stable counting sort of the n = T * k choices by expert
// ------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanMinChunk = 4096, kPlanMaxChunks = 512;

int64_t plan_chunk(int64_t n) {
  int64_t c = (n + kPlanMaxChunks - 1) / kPlanMaxChunks;
  c = (c + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
  return c < kPlanMinChunk ? kPlanMinChunk : c;
}

__device__ __forceinline__ int plan_expert(const PlanArgs& a, int64_t i) {
  const int e = a.experts[i];
  return e >= 0 && e < a.E ? e : -1;
}

// Choices of each expert in each chunk of the list.
__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(PlanArgs a, int64_t chunk) {
  extern __shared__ int32_t count[];
  pdl_launch_dependents();
  pdl_wait();
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) count[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * chunk, hi = min(lo + chunk, a.n);
  for (int64_t i = lo + threadIdx.x; i < hi; i += kPlanThreads) {
    const int e = plan_expert(a, i);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kPlanThreads) {
    a.workspace[blockIdx.x * (int64_t)a.E + e] = count[e];
  }
}

// Exclusive prefix over v[0 .. E) of shared memory by the whole CTA (E <= 2 * kPlanThreads);
// returns the total.
__device__ __forceinline__ int64_t block_scan(int64_t* v, int E, int64_t* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t x0 = 2 * tid < E ? v[2 * tid] : 0, x1 = 2 * tid + 1 < E ? v[2 * tid + 1] : 0;
  int64_t sum = x0 + x1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
    if (lane >= d) sum += up;
  }
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
  }
  before += sum - x0 - x1;
  if (2 * tid < E) v[2 * tid] = before;
  if (2 * tid + 1 < E) v[2 * tid + 1] = before + x0;
  __syncthreads();
  return total;
}

// One CTA per chunk: where each expert's rows start (the counts of all chunks, summed by every
// CTA: a few KB from L2, cheaper than a launch between), how many of them come before this
// chunk, then the chunk's own choices in order: warp w walks its 1/16 of the chunk 32 at a time,
// equal experts of the 32 found with match, so that a row's place is the number of equal experts
// before it and the result does not depend on timing.
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(PlanArgs a, int64_t chunk,
                                                                  int chunks) {
  extern __shared__ __align__(8) uint8_t smem[];
  int64_t* base = reinterpret_cast<int64_t*>(smem);                    // [E]
  int32_t* next = reinterpret_cast<int32_t*>(base + a.E);              // [kPlanWarps][E]
  __shared__ int64_t warp_sums[kPlanWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t lo = blockIdx.x * chunk, hi = min(lo + chunk, a.n);
  const int64_t span = chunk / kPlanWarps;  // a multiple of 32
  const int64_t wlo = min(lo + warp * span, hi), whi = min(wlo + span, hi);
  for (int i = tid; i < kPlanWarps * a.E; i += kPlanThreads) next[i] = 0;
  __syncthreads();
  for (int64_t i = wlo + lane; i < whi; i += 32) {
    const int e = plan_expert(a, i);
    if (e >= 0) atomicAdd(&next[warp * a.E + e], 1);
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += kPlanThreads) {
    int64_t before = 0, total = 0;
    if (chunks > 1) {
      for (int c = 0; c < chunks; ++c) {
        const int32_t v = a.workspace[c * (int64_t)a.E + e];
        total += v;
        if (c < (int)blockIdx.x) before += v;
      }
    }
    int32_t run = (int32_t)before;  // this chunk's first row of the expert, then each warp's
#pragma unroll
    for (int w = 0; w < kPlanWarps; ++w) {
      const int32_t v = next[w * a.E + e];
      next[w * a.E + e] = run;
      run += v;
    }
    base[e] = chunks > 1 ? total : run;
  }
  __syncthreads();
  const int64_t made = block_scan(base, a.E, warp_sums);
  if (blockIdx.x == 0) {
    for (int e = tid; e < a.E; e += kPlanThreads) a.offsets[e] = base[e];
    if (tid == 0) a.offsets[a.E] = made;
  }
  for (int64_t i0 = wlo; i0 < whi; i0 += 32) {
    const int64_t i = i0 + lane;
    const int e = i < whi ? plan_expert(a, i) : -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    int64_t row = -1;
    if (e >= 0) {
      int32_t* n = &next[warp * a.E + e];
      row = base[e] + *n + __popc(same & ((1u << lane) - 1u));
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) next[warp * a.E + e] += __popc(same);
    __syncwarp();
    if (i < whi) {
      a.slots[i] = (int32_t)row;
      if (row >= 0) a.tokens[row] = (int32_t)(i / a.k);
    }
  }
  for (int64_t i = max(lo, made) + tid; i < hi; i += kPlanThreads) a.tokens[i] = -1;
}

template <int V, bool BF16, bool SIGMOID>
cudaError_t route_groups(const RouteArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.T + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
  if (a.groups == 1 || a.top_groups == a.groups) {
    return launch_pdl(&route_kernel<V, BF16, SIGMOID, false>, grid, block, 0, stream, a, a.E, 0u, 1);
  }
  const int size = a.E / a.groups;
  const uint32_t magic = size == 1 ? 0u : (uint32_t)(((1ull << 32) + size - 1) / size);
  int lanes = 32;
  while (lanes * a.groups > 32) lanes >>= 1;
  return launch_pdl(&route_kernel<V, BF16, SIGMOID, true>, grid, block, 0, stream, a, size, magic,
                    lanes);
}

template <int V, bool BF16, bool SIGMOID>
cudaError_t route_one(const RouteArgs& a, bool backward, cudaStream_t stream) {
  if (!backward) return route_groups<V, BF16, SIGMOID>(a, stream);
  const dim3 grid((unsigned)((a.T + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
  return launch_pdl(&route_backward_kernel<V, BF16, SIGMOID>, grid, block, 0, stream, a);
}

template <int V>
cudaError_t route_v(const RouteArgs& a, bool backward, cudaStream_t stream) {
  if (a.bf16) {
    return a.sigmoid ? route_one<V, true, true>(a, backward, stream)
                     : route_one<V, true, false>(a, backward, stream);
  }
  return a.sigmoid ? route_one<V, false, true>(a, backward, stream)
                   : route_one<V, false, false>(a, backward, stream);
}

cudaError_t route_any(const RouteArgs& a, bool backward, cudaStream_t stream) {
  const int v = (a.E + 31) / 32;
  if (v <= 1) return route_v<1>(a, backward, stream);
  if (v <= 2) return route_v<2>(a, backward, stream);
  if (v <= 4) return route_v<4>(a, backward, stream);
  if (v <= 8) return route_v<8>(a, backward, stream);
  if (v <= 16) return route_v<16>(a, backward, stream);
  return route_v<32>(a, backward, stream);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  return route_any(a, false, stream);
}

cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t stream) {
  return route_any(a, true, stream);
}

int64_t plan_workspace_ints(int64_t n, int E) {
  const int64_t chunks = (n + plan_chunk(n) - 1) / plan_chunk(n);
  return chunks > 1 ? chunks * E : 0;
}

cudaError_t launch_plan(const PlanArgs& a, cudaStream_t stream) {
  const int64_t chunk = plan_chunk(a.n);
  const int chunks = a.n == 0 ? 1 : (int)((a.n + chunk - 1) / chunk);
  if (chunks > 1) {
    const cudaError_t err = launch_pdl(&plan_count_kernel, dim3(chunks), dim3(kPlanThreads),
                                       a.E * sizeof(int32_t), stream, a, chunk);
    if (err != cudaSuccess) return err;
  }
  const size_t smem = a.E * (sizeof(int64_t) + kPlanWarps * sizeof(int32_t));
  // the dynamic shared-memory limit is raised once, for the largest E
  constexpr size_t kMaxSmem = 1024 * (sizeof(int64_t) + kPlanWarps * sizeof(int32_t));
  if (resident_ctas(reinterpret_cast<const void*>(&plan_place_kernel), kPlanThreads, kMaxSmem, 0) <=
      0) {
    return cudaErrorInvalidConfiguration;
  }
  return launch_pdl(&plan_place_kernel, dim3(chunks), dim3(kPlanThreads), smem, stream, a, chunk,
                    chunks);
}

}  // namespace mxq
