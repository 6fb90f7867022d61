// mx_train_api.cu -- the extern "C" entry points of what stands between the products of an 8-bit training
// step (layer norm, activation, activation checkpoints), declared in include/mxq.h: host-side validation
// and launch selection. No allocation, no synchronization, no device reads.
#include <climits>
#include <cstdint>

#include "mx_expert.h"
#include "mx_launch.h"
#include "mx_train.h"
#include "mxq.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// The status of a launch. What is kept per device is made on the host's heap: no exception of it leaves
// a C entry.
template <typename F>
mx_status launched(F&& launch) {
  try {
    return launch() == cudaSuccess ? MX_OK : MX_ERR_CUDA;
  } catch (...) {
    return MX_ERR_CUDA;
  }
}

bool sizes_ok(int64_t M, int64_t K) {
  return M >= 0 && K >= 0 && M <= INT32_MAX && K <= INT32_MAX &&
         (K == 0 || M <= (int64_t(1) << 40) / K);
}
bool float_type(int t) { return t == MX_TYPE_BF16 || t == MX_TYPE_FP32; }
uintptr_t size_of(int t) { return t == MX_TYPE_FP32 ? 4 : t == MX_TYPE_BF16 ? 2 : 1; }

constexpr unsigned long long kWaitNs = 2000000000ull;

mx_status run_norm(cudaError_t (*launch)(const mxq::NormArgs&, cudaStream_t), mxq::NormArgs& a,
                   unsigned long long limit_ns, void* stream) {
  a.wait_limit_ns = limit_ns;
  return launched([&] {
    const cudaError_t err = mxq::device_error_word(&a.err);
    return err != cudaSuccess ? err : launch(a, as_stream(stream));
  });
}

// fp32 results of a call whose sums are empty: n zeros in each of a and b (or null)
mx_status zeros(float* a, float* b, int64_t n, void* stream) {
  cudaError_t err = cudaSuccess;
  if (n == 0) return MX_OK;
  if (a) err = cudaMemsetAsync(a, 0, (size_t)n * 4, as_stream(stream));
  if (b && err == cudaSuccess) err = cudaMemsetAsync(b, 0, (size_t)n * 4, as_stream(stream));
  return err == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

mx_status check_norm(int64_t M, int64_t K) {
  return sizes_ok(M, K) && K <= mxq::kNormMaxCols ? MX_OK : MX_ERR_SHAPE;
}

mx_status layer_norm(const void* x, int x_type, const void* weight, const void* bias, int w_type, int64_t M,
                     int64_t K, float eps, int center, void* y, int y_type, float* mean, float* rstd,
                     unsigned long long limit_ns, void* stream) {
  const mx_status st = check_norm(M, K);
  if (st != MX_OK) return st;
  if (!float_type(x_type) || !float_type(w_type) || !float_type(y_type)) return MX_ERR_UNSUPPORTED;
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return MX_ERR_ALIGN;
  if (M == 0 || K == 0) return zeros(mean, rstd, M, stream);
  if (!x || !y) return MX_ERR_NULL;
  if (!aligned(x, size_of(x_type)) || !aligned(y, size_of(y_type)) || !aligned(weight, size_of(w_type)) ||
      !aligned(bias, size_of(w_type))) {
    return MX_ERR_ALIGN;
  }
  mxq::NormArgs a{};
  a.x = x;
  a.x_type = x_type;
  a.weight = weight;
  a.bias = bias;
  a.w_type = w_type;
  a.M = M;
  a.K = K;
  a.eps = eps;
  a.center = center != 0;
  a.y = y;
  a.y_type = y_type;
  a.mean = mean;
  a.rstd = rstd;
  return run_norm(&mxq::launch_norm, a, limit_ns, stream);
}

mx_status layer_norm_backward(const void* dy, int dy_type, const void* x, int x_type, const float* x_scales,
                              const float* mean, const float* rstd, const void* weight, int w_type, int64_t M,
                              int64_t K, void* dx, int dx_type, float* dweight, float* dbias, void* workspace,
                              unsigned long long limit_ns, void* stream) {
  const mx_status st = check_norm(M, K);
  if (st != MX_OK) return st;
  if (!float_type(dy_type) || !float_type(w_type) || !float_type(dx_type) ||
      (!float_type(x_type) && x_type != MX_TYPE_E4M3_B128)) {
    return MX_ERR_UNSUPPORTED;
  }
  if (x_type == MX_TYPE_E4M3_B128 && K % 32 != 0) return MX_ERR_SHAPE;
  if (K == 0) return MX_OK;
  if (!aligned(dweight, 4) || !aligned(dbias, 4)) return MX_ERR_ALIGN;
  if (M == 0) return zeros(dweight, dbias, K, stream);
  if (!dy || !x || !rstd || !dx || (x_type == MX_TYPE_E4M3_B128 && !x_scales)) return MX_ERR_NULL;
  if ((dweight || dbias) && !workspace) return MX_ERR_NULL;
  if (!aligned(dy, size_of(dy_type)) || !aligned(x, size_of(x_type)) || !aligned(dx, size_of(dx_type)) ||
      !aligned(weight, size_of(w_type)) || !aligned(x_scales, 4) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(workspace, 4)) {
    return MX_ERR_ALIGN;
  }
  mxq::NormArgs a{};
  a.x = x;
  a.x_type = x_type;
  a.x_scales = x_scales;
  a.weight = weight;
  a.w_type = w_type;
  a.M = M;
  a.K = K;
  a.y = const_cast<void*>(dy);
  a.y_type = dy_type;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dx = dx;
  a.dx_type = dx_type;
  a.dweight = dweight;
  a.dbias = dbias;
  a.workspace = static_cast<float*>(workspace);
  return run_norm(&mxq::launch_norm_backward, a, limit_ns, stream);
}

// Activations: R rows of H outputs, `parts` inputs each; whole blocks where two parts have codes of their
// own.
mx_status check_activation(int64_t R, int64_t H, int kind, int gated, bool codes_of_u) {
  if (kind != MX_ACT_SILU && kind != MX_ACT_GELU && kind != MX_ACT_GELU_TANH) return MX_ERR_UNSUPPORTED;
  if (!sizes_ok(R, H) || H > (1 << 27) || !sizes_ok(R, 2 * H)) return MX_ERR_SHAPE;
  return H % (gated && codes_of_u ? 128 : 32) == 0 ? MX_OK : MX_ERR_SHAPE;
}

}  // namespace

extern "C" {

mx_status mx_layer_norm(const void* x, int x_type, const void* weight, const void* bias, int w_type,
                        int64_t M, int64_t K, float eps, int center, void* y, int y_type, float* mean,
                        float* rstd, void* stream) {
  return layer_norm(x, x_type, weight, bias, w_type, M, K, eps, center, y, y_type, mean, rstd, kWaitNs, stream);
}

mx_status mx_selftest_layer_norm_give_up(const void* x, int64_t M, int64_t K, void* y, int64_t limit_ns,
                                         void* stream) {
  if (limit_ns <= 0 || limit_ns > 100000000 || M == 0 || K == 0) return MX_ERR_SHAPE;
  return layer_norm(x, MX_TYPE_BF16, nullptr, nullptr, MX_TYPE_FP32, M, K, 1e-5f, 1, y, MX_TYPE_BF16, nullptr,
                    nullptr, (unsigned long long)limit_ns, stream);
}

mx_status mx_layer_norm_b128(const void* x, int x_type, const void* weight, const void* bias, int w_type,
                             int64_t M, int64_t K, float eps, int center, void* codes, float* scales,
                             void* x_codes, float* x_scales, float* mean, float* rstd, void* stream) {
  const mx_status st = check_norm(M, K);
  if (st != MX_OK) return st;
  if (K % 32 != 0) return MX_ERR_SHAPE;
  if (!float_type(x_type) || !float_type(w_type)) return MX_ERR_UNSUPPORTED;
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return MX_ERR_ALIGN;
  if (M == 0 || K == 0) return zeros(mean, rstd, M, stream);
  if (!x || !codes || !scales || (x_codes == nullptr) != (x_scales == nullptr)) return MX_ERR_NULL;
  if (!aligned(x, 32) || !aligned(codes, 32) || !aligned(scales, 4) || !aligned(x_codes, 32) ||
      !aligned(x_scales, 4) || !aligned(weight, 32) || !aligned(bias, 32)) {
    return MX_ERR_ALIGN;
  }
  mxq::NormArgs a{};
  a.x = x;
  a.x_type = x_type;
  a.weight = weight;
  a.bias = bias;
  a.w_type = w_type;
  a.M = M;
  a.K = K;
  a.eps = eps;
  a.center = center != 0;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.x_codes = static_cast<uint8_t*>(x_codes);
  a.x_scales_out = x_scales;
  a.mean = mean;
  a.rstd = rstd;
  return run_norm(&mxq::launch_norm, a, kWaitNs, stream);
}

mx_status mx_layer_norm_backward_workspace(int64_t M, int64_t K, int64_t* bytes) {
  if (!bytes) return MX_ERR_NULL;
  const mx_status st = check_norm(M, K);
  if (st != MX_OK) return st;
  *bytes = mxq::norm_workspace_floats(M, K) * 4;
  return MX_OK;
}

mx_status mx_layer_norm_backward(const void* dy, int dy_type, const void* x, int x_type,
                                 const float* x_scales, const float* mean, const float* rstd,
                                 const void* weight, int w_type, int64_t M, int64_t K, void* dx,
                                 int dx_type, float* dweight, float* dbias, void* workspace,
                                 void* stream) {
  return layer_norm_backward(dy, dy_type, x, x_type, x_scales, mean, rstd, weight, w_type, M, K, dx, dx_type,
                             dweight, dbias, workspace, kWaitNs, stream);
}

mx_status mx_selftest_layer_norm_backward_give_up(const void* dy, const void* x, int x_type,
                                                  const float* x_scales, const float* mean,
                                                  const float* rstd, int64_t M, int64_t K, void* dx,
                                                  int64_t limit_ns, void* stream) {
  if (limit_ns <= 0 || limit_ns > 100000000 || M == 0 || K == 0) return MX_ERR_SHAPE;
  return layer_norm_backward(dy, MX_TYPE_BF16, x, x_type, x_scales, mean, rstd, nullptr, MX_TYPE_FP32, M, K, dx,
                             MX_TYPE_BF16, nullptr, nullptr, nullptr, (unsigned long long)limit_ns, stream);
}

mx_status mx_activation_b128(const void* u, int64_t R, int64_t H, int kind, int gated, void* codes,
                             float* scales, void* u_codes, float* u_scales, void* stream) {
  const mx_status st = check_activation(R, H, kind, gated, u_codes != nullptr);
  if (st != MX_OK) return st;
  if (R == 0 || H == 0) return MX_OK;
  if (!u || !codes || !scales || (u_codes == nullptr) != (u_scales == nullptr)) return MX_ERR_NULL;
  if (!aligned(u, 32) || !aligned(codes, 32) || !aligned(scales, 4) || !aligned(u_codes, 32) ||
      !aligned(u_scales, 4)) {
    return MX_ERR_ALIGN;
  }
  mxq::ActArgs a{};
  a.u = u;
  a.R = R;
  a.H = H;
  a.kind = kind;
  a.gated = gated != 0;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.u_codes = static_cast<uint8_t*>(u_codes);
  a.u_scales_out = u_scales;
  return launched([&] { return mxq::launch_activation(a, as_stream(stream)); });
}

mx_status mx_activation_backward(const void* dh, const void* u, int u_type, const float* u_scales,
                                 int64_t R, int64_t H, int kind, int gated, void* du, void* du_codes,
                                 float* du_scales, void* stream) {
  if (u_type != MX_TYPE_BF16 && u_type != MX_TYPE_E4M3_B128) return MX_ERR_UNSUPPORTED;
  const bool checkpoint = u_type == MX_TYPE_E4M3_B128;
  const mx_status st = check_activation(R, H, kind, gated, checkpoint || du_codes);
  if (st != MX_OK) return st;
  if (R == 0 || H == 0) return MX_OK;
  if (!dh || !u || (checkpoint && !u_scales) || (!du && !du_codes) ||
      (du_codes == nullptr) != (du_scales == nullptr)) {
    return MX_ERR_NULL;
  }
  if (!aligned(dh, 32) || !aligned(u, 32) || !aligned(u_scales, 4) || !aligned(du, 32) ||
      !aligned(du_codes, 32) || !aligned(du_scales, 4)) {
    return MX_ERR_ALIGN;
  }
  mxq::ActArgs a{};
  a.u = u;
  a.u_scales = checkpoint ? u_scales : nullptr;
  a.dh = dh;
  a.R = R;
  a.H = H;
  a.kind = kind;
  a.gated = gated != 0;
  a.codes = static_cast<uint8_t*>(du_codes);
  a.scales = du_scales;
  a.du = du;
  return launched([&] { return mxq::launch_activation_backward(a, as_stream(stream)); });
}

mx_status mx_requantize_b128_cols(const void* codes, const float* scales, int64_t M, int64_t K,
                                  const int32_t* index, int64_t R, const int64_t* row_offsets, int E,
                                  void* out_codes, float* out_scales, void* stream) {
  if (!sizes_ok(M, K) || !sizes_ok(R, K) || K % 32 != 0) return MX_ERR_SHAPE;
  if (!index && R != M && R != 0) return MX_ERR_SHAPE;
  if (!row_offsets && E != 1) return MX_ERR_SHAPE;
  int64_t rows = 0;
  const mx_status st = mx_b128_padded_rows(R, E, &rows);
  if (st != MX_OK) return st;
  if (rows == 0 || K == 0) return MX_OK;
  if ((M > 0 && (!codes || !scales)) || !out_codes || !out_scales) return MX_ERR_NULL;
  if (!aligned(codes, 32) || !aligned(scales, 4) || !aligned(out_codes, 32) || !aligned(out_scales, 4) ||
      !aligned(index, 4) || !aligned(row_offsets, 8)) {
    return MX_ERR_ALIGN;
  }
  mxq::B128QuantArgs a{};
  a.x = codes;
  a.x_scales = scales;
  a.index = index;
  a.batch = 1;
  a.M = M;
  a.K = K;
  a.R = R;
  a.offsets = row_offsets;
  a.E = E;
  a.blocks = rows / 128;
  a.codes = static_cast<uint8_t*>(out_codes);
  a.scales = out_scales;
  return launched([&] { return mxq::launch_b128_recols(a, as_stream(stream)); });
}

mx_status mx_dequantize_b128_rows(const void* codes, const float* scales, int64_t M, int64_t K,
                                  const int32_t* index, int64_t R, void* y, int y_type, void* stream) {
  if (!sizes_ok(M, K) || !sizes_ok(R, K) || K % 32 != 0) return MX_ERR_SHAPE;
  if (!index && R != M && R != 0) return MX_ERR_SHAPE;
  if (!float_type(y_type)) return MX_ERR_UNSUPPORTED;
  if (R == 0 || K == 0) return MX_OK;
  if ((M > 0 && (!codes || !scales)) || !y) return MX_ERR_NULL;
  if (!aligned(codes, 32) || !aligned(scales, 4) || !aligned(index, 4) || !aligned(y, 32)) {
    return MX_ERR_ALIGN;
  }
  mxq::DequantB128Args a{};
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = scales;
  a.index = index;
  a.M = M;
  a.K = K;
  a.R = R;
  a.y = y;
  a.f32 = y_type == MX_TYPE_FP32;
  return launched([&] { return mxq::launch_b128_dequant(a, as_stream(stream)); });
}

}  // extern "C"
