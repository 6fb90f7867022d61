// mx_train.h -- host-side launch interface of the kernels between the products of an 8-bit training
// step: layer norm, activation, and what is made of activation checkpoints (E4M3 codes with a scale
// per block of 128).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace mxq {

// element types as the kernels know them (the header's MX_TYPE_*)
constexpr int kTypeBf16 = 0, kTypeFp32 = 1, kTypeB128 = 2;

constexpr int64_t kNormMaxCols = 16384;

struct NormArgs {
  const void* x;        // [M, K] of x_type (backward: kTypeB128 too)
  const float* x_scales;  // backward, kTypeB128: [ceil(K / 128), M]
  const void* weight;   // [K] of w_type, or null (ones)
  const void* bias;     // [K] of w_type, or null (zeros)
  int x_type, w_type, y_type, dx_type;
  int64_t M, K;
  float eps;
  bool center;          // forward: subtract the mean
  void* y;              // forward: [M, K] of y_type; backward: dy, the gradient of it
  uint8_t* codes;       // forward into 8 bits: [M, K], y is null
  float* scales;        // [ceil(K / 128), M]
  uint8_t* x_codes;     // forward: checkpoint of x, or null
  float* x_scales_out;
  float* mean;          // forward: [M] or null; backward: read, null where not centred
  float* rstd;          // forward: [M] or null; backward: read
  void* dx;             // backward: [M, K] of dx_type
  float* dweight;       // backward: [K] or null
  float* dbias;         // backward: [K] or null
  float* workspace;     // backward: norm_workspace_floats
  unsigned int* err;    // device error word
  unsigned long long wait_limit_ns;  // of each wait for a row
};
cudaError_t launch_norm(const NormArgs& a, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormArgs& a, cudaStream_t stream);
int64_t norm_workspace_floats(int64_t M, int64_t K);

struct ActArgs {
  const void* u;        // [R, U] (U = 2 H when gated, else H): bf16, or codes with u_scales
  const float* u_scales;
  const void* dh;       // backward: bf16 [R, H]
  int64_t R, H;
  int kind;             // MX_ACT_*
  bool gated;
  uint8_t* codes;       // forward: h [R, H]; backward: du [R, U], or null
  float* scales;
  uint8_t* u_codes;     // forward: checkpoint of u, or null
  float* u_scales_out;
  void* du;             // backward: bf16 [R, U], or null
};
cudaError_t launch_activation(const ActArgs& a, cudaStream_t stream);
cudaError_t launch_activation_backward(const ActArgs& a, cudaStream_t stream);

struct DequantB128Args {
  const uint8_t* codes;   // [M, K]
  const float* scales;    // [ceil(K / 128), M]
  const int32_t* index;   // [R] or null
  int64_t M, K, R;
  void* y;                // [R, K]
  bool f32;
};
cudaError_t launch_b128_dequant(const DequantB128Args& a, cudaStream_t stream);

}  // namespace mxq
