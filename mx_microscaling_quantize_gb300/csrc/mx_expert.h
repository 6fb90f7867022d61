// mx_expert.h -- host-side launch interface of the expert-layer kernels (routing, 8-bit operands
// with a scale per block of 128, their products, combination of the experts' outputs).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace mxq {

constexpr int kB128 = 128;           // elements along the contraction under one scale
constexpr float kB128AmaxFloor = 7.888609052210118e-31f;  // 2^-100

struct RouteArgs {
  const void* logits;   // [T, E], bf16 or fp32
  const float* bias;    // [E] or null
  int64_t T;
  int E, k;
  int groups, top_groups;
  bool sigmoid, renormalize, bf16;
  float scale;
  int32_t* experts;     // [T, k]
  float* weights;       // [T, k]
  const float* grad_weights;  // backward: [T, k]
  const int32_t* chosen;      // backward: [T, k]
  void* grad_logits;          // backward: [T, E], as logits
};
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t stream);

struct PlanArgs {
  const int32_t* experts;  // [n]
  int64_t n;               // T * k
  int k, E;
  int64_t* offsets;        // [E + 1]
  int32_t* tokens;         // [n]
  int32_t* slots;          // [n]
  int32_t* workspace;      // plan_workspace_ints
};
int64_t plan_workspace_ints(int64_t n, int E);
cudaError_t launch_plan(const PlanArgs& a, cudaStream_t stream);

struct B128QuantArgs {
  const void* x;           // bf16 [batch, M, K]
  const int32_t* index;    // rows / cols: source row of each of R rows (< 0: zeros), or null
  int64_t batch, M, K, R;
  const int64_t* offsets;  // cols: [E + 1] or null (one run of R rows)
  int E;
  int64_t blocks;          // cols: 128-row blocks of the output
  uint8_t* codes;
  float* scales;
  uint8_t* codes_t;        // blocks: the transposed operand, or null
  float* scales_t;
};
cudaError_t launch_b128_rows(const B128QuantArgs& a, cudaStream_t stream);
cudaError_t launch_b128_cols(const B128QuantArgs& a, cudaStream_t stream);
cudaError_t launch_b128_blocks(const B128QuantArgs& a, cudaStream_t stream);

enum B128Mode { kB128Dense = 0, kB128Grouped = 1, kB128Wgrad = 2 };

struct B128GemmArgs {
  const void* a_codes;    // dense [M, K]; grouped [M, K] rows by expert; wgrad [M, K = R]
  const float* a_scales;  // [ceil(K / 128), M]
  const void* b_codes;    // dense [N, K]; grouped [E, N, K]; wgrad [N, K = R]
  const float* b_scales;  // blocks [E, ceil(N / 128), ceil(K / 128)] or rows [ceil(K / 128), N]
  void* c;                // dense / grouped [M, N]; wgrad [E, M, N]
  int64_t M, N, K;
  const int64_t* offsets; // [E + 1]; rows of a by expert (wgrad: rows before padding)
  int64_t rows_total;     // wgrad: largest offset
  int E;
  bool b_rows;            // b_scales in the rows form
  bool out_f32;
  unsigned int* err;
  unsigned long long wait_limit_ns;
};
cudaError_t launch_b128_gemm(int mode, const B128GemmArgs& a, cudaStream_t stream);

struct CombineArgs {
  const void* y;          // bf16 [R, N]
  const int32_t* slots;   // [T, k]
  const float* weights;   // [T, k] or null
  const void* dout;       // backward: bf16 [T, N]
  int64_t T, R, N;
  int k;
  void* out;              // forward: bf16 [T, N]
  void* dy;               // backward: bf16 [R, N]
  float* dweights;        // backward: [T, k] or null
  int32_t* owner;         // backward: workspace [R], then rows of dy that no slot names become zeros; or null
};
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream);
cudaError_t launch_combine_backward(const CombineArgs& a, cudaStream_t stream);

}  // namespace mxq
