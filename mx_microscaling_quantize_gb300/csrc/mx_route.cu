// mx_route.cu -- routing of tokens to experts: scores, choice, weights, the gradient of the
// logits, and the plan that orders the chosen (token, expert) pairs by expert.
#include <cmath>

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

// Lane l holds experts V l .. V l + V - 1: a lane's values are one run of memory, a group of experts is
// a run of lanes, and the lowest lane of several has the lowest index.
template <int V, bool BF16>
__device__ __forceinline__ void load_logits(const void* logits, int64_t t, int E, bool wide,
                                            float (&l)[V]) {
  const int e0 = (threadIdx.x & 31) * V;
  if constexpr (V >= 4) {
    if (wide && e0 + V <= E) {  // rows of whole 16-byte pieces
      if constexpr (BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(logits) + t * E + e0;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          uint32_t w0, w1;
          asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "l"(p + i));
          l[i] = bf16_lo(w0);
          l[i + 1] = bf16_hi(w0);
          l[i + 2] = bf16_lo(w1);
          l[i + 3] = bf16_hi(w1);
        }
      } else {
        const float* p = static_cast<const float*>(logits) + t * E + e0;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const uint4 w = load_v4(p + i);
          l[i] = __uint_as_float(w.x);
          l[i + 1] = __uint_as_float(w.y);
          l[i + 2] = __uint_as_float(w.z);
          l[i + 3] = __uint_as_float(w.w);
        }
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    l[i] = e0 + i < E ? load_logit<BF16>(logits, t * E + e0 + i) : -INFINITY;
  }
}

// The reciprocal rounded to nearest is the quotient 1 / (1 + exp(-l)) rounded to nearest.
__device__ __forceinline__ float sigmoid(float l) { return __frcp_rn(__fadd_rn(1.0f, expf(-l))); }

// Scores of one token before the division: exp(l - max) with the sum in *total and the maximum in *top.
template <int V>
__device__ __forceinline__ void softmax_scores(const float (&l)[V], float (&s)[V], float* total,
                                               float* top) {
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
    s[i] = expf(__fsub_rn(l[i], m));  // past E: of -inf, 0 (NaN where m, and so the sum, is)
    sum += s[i];
  }
  *total = warp_sum(sum);
  *top = m;
}

// The two largest keys of two pairs.
__device__ __forceinline__ void merge_two(uint32_t& k0, uint32_t& k1, uint32_t o0, uint32_t o1) {
  k1 = max(min(k0, o0), max(k1, o1));
  k0 = max(k0, o0);
}

enum RouteGroups { kNoGroups = 0, kLaneGroups = 1, kAnyGroups = 2 };

// One warp per token. With s the scores (softmax numerators exp(l - max), or sigmoids), the
// choice c is s, or s + bias (then of the normalised softmax), and -inf where l is: such an
// expert is never chosen. Without a bias the softmax's denominator cannot change the order, so
// the choice uses the numerators and does not depend on the order of a sum.
// Groups: where a group is a whole run of lanes (kLaneGroups) the two largest choices of each come
// from the lanes' own and shuffles; otherwise from shared memory, each lane of a group's share
// starting at another place so that the 32 lanes meet 32 banks. Each group's first lane ranks it
// among the groups, and a ballot names the kept ones.
// Top k: keys are unsigned images of the choices; each round is one warp-wide maximum, a ballot whose
// lowest lane holds the lowest index, and the winning lane's step to its next best: its second, which
// it knows, and only after that a search among its own values.
// 16384 tokens of 256 experts in groups 17.5 us, without 14.0; their 19 MB would take 3. The time goes with
// the instructions this form issues: 1020 of a warp per token in groups, 760 without, in 81 % and 75 % of
// the schedulers' cycles, most of them for one result that 32 lanes work out together.
template <int V, bool BF16, bool SIGMOID, int GROUPS>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a, int group_size,
                                                                 uint32_t group_magic, int lanes,
                                                                 bool wide, bool wide_bias) {
  __shared__ __align__(16) float score_row[kRouteWarps][V * 32];
  __shared__ float choice_row[GROUPS == kAnyGroups ? kRouteWarps : 1][GROUPS == kAnyGroups ? V * 32 : 1];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * V;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  float l[V], s[V], total;
  load_logits<V, BF16>(a.logits, t, a.E, wide, l);
  if (SIGMOID) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = sigmoid(l[i]);
    total = 1.0f;
  } else {
    float top;
    softmax_scores(l, s, &total, &top);
  }
  if constexpr (V >= 4) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      *reinterpret_cast<float4*>(&score_row[warp][e0 + i]) =
          make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) score_row[warp][e0 + i] = s[i];
  }
  float choice[V];
#pragma unroll
  for (int i = 0; i < V; ++i) choice[i] = s[i];
  if (a.bias) {
    float b[V];
    load_logits<V, false>(a.bias, 0, a.E, wide_bias, b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      choice[i] = __fadd_rn(SIGMOID ? s[i] : __fdiv_rn(s[i], total), b[i]);
    }
  }
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float c = l[i] == -INFINITY ? -INFINITY : choice[i];  // (past E too)
    key[i] = order_key(c);
    if (GROUPS == kAnyGroups) choice_row[warp][e0 + i] = c;
  }
  __syncwarp();
  // the lane's two largest keys, the earlier of equal ones first; `taken` are left out
  uint32_t best = 0u, best_i = 0u, second = 0u, second_i = 0u, taken = 0u;
  auto search = [&]() {
    best = second = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t q = (taken >> i) & 1u ? 0u : key[i];
      if (q > best) {
        second = best;
        second_i = best_i;
        best = q;
        best_i = i;
      } else if (q > second) {
        second = q;
        second_i = i;
      }
    }
  };
  if (GROUPS != kAnyGroups) search();
  if (GROUPS != kNoGroups) {
    // lanes per group: `lanes`, a power of two, groups * lanes <= 32
    const int g = lane / lanes, sub = lane % lanes;
    uint32_t k0 = 0u, k1 = 0u;  // keys of the two largest
    if (GROUPS == kLaneGroups) {
      k0 = best;
      k1 = second;
    } else if (g < a.groups) {
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
      merge_two(k0, k1, o0, o1);
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
    const bool keep = g < a.groups && rank < a.top_groups;
    if (GROUPS == kLaneGroups) {
      if (!keep) best = second = 0u;  // the lane never wins
    } else {
      const uint32_t kept = __ballot_sync(0xFFFFFFFFu, keep);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = e0 + i;
        // e / group_size: exact for e < 1024 with magic = ceil(2^32 / group_size)
        const int ge = group_size == 1 ? e : (int)__umulhi((uint32_t)e, group_magic);
        if (e < a.E && !((kept >> (ge * lanes)) & 1u)) key[i] = 0u;
      }
    }
  }
  if (GROUPS == kAnyGroups) search();
  bool fresh = true;  // `second` is the lane's next best
  int32_t expert = -1;  // lane j: the j-th choice
  for (int j = 0; j < a.k; ++j) {
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    if (top == 0u) break;
    const int who = __ffs(__ballot_sync(0xFFFFFFFFu, best == top)) - 1;
    const int e = __shfl_sync(0xFFFFFFFFu, e0 + (int)best_i, who);
    if (lane == j) expert = e;
    if (lane == who) {
      taken |= 1u << best_i;
      if (fresh) {
        best = second;
        best_i = second_i;
      } else {
        search();
      }
      fresh = !fresh;
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
//   sigmoid: dl = dp s (1 - s), nothing for the others; 1 - s is the sigmoid of -l (from s itself nothing
//   would be left of it where the router is sure: s is 1 in fp32 from l = 17 on);
//   softmax: dl_i = s_i (dp_i - sum_j dp_j s_j), every logit.
// Where the router is sure of its choice, both differences are far below their terms, so they are taken
// between the gradients, term by term: dp_j = scale sum_i p_i (g_j - g_i) / P^2, and for a chosen expert
// dp_i - sum_j dp_j s_j = dp_i r + sum_j s_j (dp_i - dp_j) over the chosen j, r the scores not chosen
// (renormalised, sum_j dp_j s_j is nothing but its own rounding).
// A choice of -1 (no expert) takes and gives nothing. The scores are computed again from the
// logits: reading them back would cost what the logits cost. The row is written as if nothing had been
// chosen (d = 0), then lane j its choice's element over it, whose score it has from its own logit: no
// row of scores or gradients is kept beside the registers (with such rows in shared memory 4096 tokens of
// 512 experts took more than twice as long). 4096 tokens of 512 experts in bf16, 8 chosen: 6.4 us, of which
// the differences are 0.5; 4097 of 64, 6 chosen: 3.4; 1000 of 1024 in fp32: 7.6.
template <bool BF16>
__device__ __forceinline__ void store_grad(void* p, int64_t at, float v) {
  if (BF16) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
    static_cast<uint16_t*>(p)[at] = h;
  } else {
    static_cast<float*>(p)[at] = v;
  }
}
template <int V, bool BF16, bool SIGMOID>
__global__ void __launch_bounds__(kRouteWarps * 32) route_backward_kernel(RouteArgs a, bool wide) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * V;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  float l[V];
  if (!SIGMOID) load_logits<V, BF16>(a.logits, t, a.E, wide, l);  // asked for before the choice's
  int32_t expert = -1;
  float g = 0.0f, p = 0.0f, chosen = 0.0f;  // gradient, score and logit of the lane's choice
  if (lane < a.k) {
    expert = load_s32(a.chosen + t * a.k + lane);
    g = load_f32(a.grad_weights + t * a.k + lane);
    if (expert >= a.E || expert < 0) expert = -1;
  }
  if (expert >= 0) {
    chosen = load_logit<BF16>(a.logits, t * a.E + expert);
  } else {
    g = 0.0f;
  }
  float dl[V];
  if (SIGMOID) {
    if (expert >= 0) p = sigmoid(chosen);
  } else {
    float total, m;
    softmax_scores(l, dl, &total, &m);
#pragma unroll
    for (int i = 0; i < V; ++i) dl[i] = total == 0.0f ? 0.0f : __fdiv_rn(dl[i], total);
    if (expert >= 0) p = total == 0.0f ? 0.0f : __fdiv_rn(expf(__fsub_rn(chosen, m)), total);
  }
  if (a.renormalize) {
    const float P = warp_sum(p);
    const float share = P == 0.0f ? 0.0f : p / P;
    float sum = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      sum += __shfl_sync(0xFFFFFFFFu, share, j) * (g - __shfl_sync(0xFFFFFFFFu, g, j));
    }
    g = expert < 0 || P == 0.0f ? 0.0f : sum / P;
  }
  const float through = a.scale * warp_sum(expert >= 0 ? g * p : 0.0f);
  // an expert named twice (no call of the router does that) adds both, in order; its first lane writes
  float d = g;
  bool first = expert >= 0;
  const uint32_t same = __match_any_sync(0xFFFFFFFFu, expert);
  if (__any_sync(0xFFFFFFFFu, first && (same & (same - 1u)))) {
    d = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      const float other = __shfl_sync(0xFFFFFFFFu, g, j);
      if ((same >> j) & 1u) d += other;
    }
    first = first && lane == __ffs(same) - 1;
  }
  float own = a.scale * d;  // the gradient of the choice's logit over its p
  if (SIGMOID) {
    own *= sigmoid(-chosen);
  } else if (a.renormalize) {
    own -= through;
  } else {
    float rest = 0.0f, sum = 0.0f;  // of the scores not chosen; of the differences to the chosen ones
    uint32_t mine = 0u;             // the lane's experts that are chosen
    const float mass = first ? p : 0.0f;
    for (int j = 0; j < a.k; ++j) {
      const uint32_t at = (uint32_t)(__shfl_sync(0xFFFFFFFFu, expert, j) - e0);
      if (at < (uint32_t)V) mine |= 1u << at;
      sum += __shfl_sync(0xFFFFFFFFu, mass, j) * (d - __shfl_sync(0xFFFFFFFFu, d, j));
    }
#pragma unroll
    for (int i = 0; i < V; ++i) rest += (mine >> i) & 1u ? 0.0f : dl[i];
    own = a.scale * (d * warp_sum(rest) + sum);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) dl[i] = SIGMOID ? 0.0f : dl[i] * (0.0f - through);
  bool whole = false;
  if constexpr (V >= 4) {
    whole = wide && e0 + V <= a.E;
    if (whole) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        if constexpr (BF16) {
          uint32_t w0, w1;
          asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(w0) : "f"(dl[i]), "f"(dl[i + 1]));
          asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(w1) : "f"(dl[i + 2]), "f"(dl[i + 3]));
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.grad_logits) + t * a.E + e0 + i) =
              make_uint2(w0, w1);
        } else {
          *reinterpret_cast<float4*>(static_cast<float*>(a.grad_logits) + t * a.E + e0 + i) =
              make_float4(dl[i], dl[i + 1], dl[i + 2], dl[i + 3]);
        }
      }
    }
  }
  if (!whole) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (e0 + i < a.E) store_grad<BF16>(a.grad_logits, t * a.E + e0 + i, dl[i]);
    }
  }
  __syncwarp();  // the row comes before its choices
  if (first) {
    store_grad<BF16>(a.grad_logits, t * a.E + expert, p * own);
  }
}

// ------------------------------------------------------------------------------------------
// plan: a stable counting sort of the n = T * k choices by expert
// ------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;
constexpr int kPlanOneChunk = 1024, kPlanMaxChunks = 512;

// One CTA and one launch up to kPlanOneChunk choices (1024 choices: 3.9 us, in two launches 4.8; 2048:
// 5.5 us in two). Beyond, the walk of a chunk (0.45 us per 512 choices) and every CTA's sums over all
// chunks' counts grow against each other, least together where a chunk is some multiple of sqrt(n):
// 131072 choices of 256 experts in chunks of 512, 1024, 2048 and 3072 take 19.3, 14.2, 9.7 and 10.9 us,
// 4096 choices in chunks of 512, 1024 and 2048 5.0, 6.0 and 7.2.
int64_t plan_chunk(int64_t n) {
  if (n <= kPlanOneChunk) return n <= kPlanThreads ? kPlanThreads : kPlanOneChunk;
  int64_t c = (int64_t)(5.5 * std::sqrt((double)n));
  if (c < (n + kPlanMaxChunks - 1) / kPlanMaxChunks) c = (n + kPlanMaxChunks - 1) / kPlanMaxChunks;
  return (c + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
}

__device__ __forceinline__ int plan_expert(const PlanArgs& a, int64_t i) {
  const int e = load_s32(a.experts + i);
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
// before it and the result does not depend on timing. 131072 choices of 256 experts: 9.7 us for both
// launches, of which their start and the chunks' serial walks are most (2.6 MB move).
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
#pragma unroll 8
      for (int c = 0; c < chunks; ++c) {
        const int32_t v = load_s32(a.workspace + c * (int64_t)a.E + e);
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

template <int V, bool BF16, bool SIGMOID, int GROUPS>
cudaError_t route_launch(const RouteArgs& a, int size, uint32_t magic, int lanes, bool wide,
                         cudaStream_t stream) {
  // One token per warp and then the warp ends: resident warps that walk the tokens, the next logits
  // already asked for, measured slower (21 against 18 us for 16384 x 256), their registers costing
  // more resident warps than the loads cost time.
  return launch_pdl(&route_kernel<V, BF16, SIGMOID, GROUPS>,
                    dim3((unsigned)((a.T + kRouteWarps - 1) / kRouteWarps)), dim3(kRouteWarps * 32), 0,
                    stream, a, size, magic, lanes, wide,
                    a.E % 4 == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0);
}

template <int V, bool BF16, bool SIGMOID>
cudaError_t route_groups(const RouteArgs& a, bool wide, cudaStream_t stream) {
  if (a.groups == 1 || a.top_groups == a.groups) {
    return route_launch<V, BF16, SIGMOID, kNoGroups>(a, a.E, 0u, 1, wide, stream);
  }
  const int size = a.E / a.groups;
  const uint32_t magic = size == 1 ? 0u : (uint32_t)(((1ull << 32) + size - 1) / size);
  if (size % V == 0 && ((size / V) & (size / V - 1)) == 0) {
    return route_launch<V, BF16, SIGMOID, kLaneGroups>(a, size, magic, size / V, wide, stream);
  }
  int lanes = 32;
  while (lanes * a.groups > 32) lanes >>= 1;
  return route_launch<V, BF16, SIGMOID, kAnyGroups>(a, size, magic, lanes, wide, stream);
}

template <int V, bool BF16, bool SIGMOID>
cudaError_t route_one(const RouteArgs& a, bool backward, cudaStream_t stream) {
  // four values are loaded (and stored) together where every row allows it
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.grad_logits);
  const bool wide = a.E % 4 == 0 && at % (BF16 ? 8 : 16) == 0;
  if (!backward) return route_groups<V, BF16, SIGMOID>(a, wide, stream);
  const dim3 grid((unsigned)((a.T + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
  return launch_pdl(&route_backward_kernel<V, BF16, SIGMOID>, grid, block, 0, stream, a, wide);
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
