// mx_expert_api.cu -- the extern "C" entry points of the expert layer declared in include/mxq.h
// (routing, operands with a scale per block of 128, their products, combination): host-side
// validation and launch selection. No allocation, no synchronization, no device reads.
#include <climits>
#include <cstdint>

#include "mx_expert.h"
#include "mx_launch.h"
#include "mxq.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
mx_status from_cuda(cudaError_t err) { return err == cudaSuccess ? MX_OK : MX_ERR_CUDA; }
cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// The status of a launch. What is kept per device is made on the host's heap: no exception of it leaves
// a C entry.
template <typename F>
mx_status launched(F&& launch) {
  try {
    return from_cuda(launch());
  } catch (...) {
    return MX_ERR_CUDA;
  }
}

// rows and columns of one operand or matrix: non-negative, 32-bit, their product far from overflow
bool sizes_ok(int64_t M, int64_t K) {
  return M >= 0 && K >= 0 && M <= INT32_MAX && K <= INT32_MAX &&
         (K == 0 || M <= (int64_t(1) << 40) / K);
}

mx_status check_route(int64_t T, int E, int k, int logits_type, int score) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 32 || k > E) return MX_ERR_SHAPE;
  if (T > INT32_MAX / k) return MX_ERR_SHAPE;  // rows are 32-bit
  if (logits_type != MX_TYPE_BF16 && logits_type != MX_TYPE_FP32) return MX_ERR_UNSUPPORTED;
  if (score != MX_SCORE_SOFTMAX && score != MX_SCORE_SIGMOID) return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

mx_status check_b128_gemm(int64_t M, int64_t N, int64_t K, int c_type) {
  if (!sizes_ok(M, K) || !sizes_ok(N, K) || !sizes_ok(M, N)) return MX_ERR_SHAPE;
  if (K % 32 != 0 || N % 8 != 0) return MX_ERR_SHAPE;
  if (c_type != MX_TYPE_BF16 && c_type != MX_TYPE_FP32) return MX_ERR_UNSUPPORTED;
  return MX_OK;
}

mx_status check_b128_pointers(const void* a_codes, const float* a_scales, const void* b_codes,
                              const float* b_scales, const void* c) {
  if (!a_codes || !a_scales || !b_codes || !b_scales || !c) return MX_ERR_NULL;
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(c, 16)) return MX_ERR_ALIGN;
  if (!aligned(a_scales, 4) || !aligned(b_scales, 4)) return MX_ERR_ALIGN;
  return MX_OK;
}

mx_status run_gemm(int mode, mxq::B128GemmArgs& g, unsigned long long limit_ns, void* stream) {
  g.wait_limit_ns = limit_ns;
  return launched([&] {
    const cudaError_t err = mxq::device_error_word(&g.err);
    return err != cudaSuccess ? err : mxq::launch_b128_gemm(mode, g, as_stream(stream));
  });
}

constexpr unsigned long long kWaitNs = 2000000000ull;

mx_status dense(const void* a_codes, const float* a_scales, const void* b_codes,
                const float* b_scales, int64_t M, int64_t N, int64_t K, int b_form, int c_type,
                void* c, unsigned long long limit_ns, void* stream) {
  mx_status st = check_b128_gemm(M, N, K, c_type);
  if (st != MX_OK) return st;
  if (b_form != MX_B128_BLOCKS && b_form != MX_B128_ROWS) return MX_ERR_UNSUPPORTED;
  if (K == 0) return MX_ERR_SHAPE;
  if (M == 0 || N == 0) return MX_OK;
  st = check_b128_pointers(a_codes, a_scales, b_codes, b_scales, c);
  if (st != MX_OK) return st;
  mxq::B128GemmArgs g{};
  g.a_codes = a_codes;
  g.a_scales = a_scales;
  g.b_codes = b_codes;
  g.b_scales = b_scales;
  g.c = c;
  g.M = M;
  g.N = N;
  g.K = K;
  g.E = 1;
  g.b_rows = b_form == MX_B128_ROWS;
  g.out_f32 = c_type == MX_TYPE_FP32;
  return run_gemm(mxq::kB128Dense, g, limit_ns, stream);
}

mx_status grouped(const void* a_codes, const float* a_scales, const void* b_codes,
                  const float* b_scales, const int64_t* row_offsets, int E, int64_t M_total, int64_t N,
                  int64_t K, int c_type, void* c, unsigned long long limit_ns, void* stream) {
  mx_status st = check_b128_gemm(M_total, N, K, c_type);
  if (st != MX_OK) return st;
  if (E < 1 || E > 1024 || N > INT32_MAX / E || K == 0) return MX_ERR_SHAPE;
  if (M_total == 0 || N == 0) return MX_OK;
  if (!row_offsets) return MX_ERR_NULL;
  st = check_b128_pointers(a_codes, a_scales, b_codes, b_scales, c);
  if (st != MX_OK) return st;
  if (!aligned(row_offsets, 8)) return MX_ERR_ALIGN;
  mxq::B128GemmArgs g{};
  g.a_codes = a_codes;
  g.a_scales = a_scales;
  g.b_codes = b_codes;
  g.b_scales = b_scales;
  g.c = c;
  g.M = M_total;
  g.N = N;
  g.K = K;
  g.offsets = row_offsets;
  g.E = E;
  g.out_f32 = c_type == MX_TYPE_FP32;
  return run_gemm(mxq::kB128Grouped, g, limit_ns, stream);
}

}  // namespace

extern "C" {

mx_status mx_route(const void* logits, int logits_type, const float* bias, int64_t T, int E, int k,
                   int score, int groups, int top_groups, int renormalize, float scale,
                   int32_t* experts, float* weights, void* stream) {
  mx_status st = check_route(T, E, k, logits_type, score);
  if (st != MX_OK) return st;
  if (groups < 1 || groups > 32 || E % groups != 0) return MX_ERR_SHAPE;
  if (top_groups < 1 || top_groups > groups || k > E / groups * top_groups) return MX_ERR_SHAPE;
  if (T == 0) return MX_OK;
  if (!logits || !experts || !weights) return MX_ERR_NULL;
  if (!aligned(logits, logits_type == MX_TYPE_BF16 ? 2 : 4) || !aligned(bias, 4) ||
      !aligned(experts, 4) || !aligned(weights, 4)) {
    return MX_ERR_ALIGN;
  }
  mxq::RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.T = T;
  a.E = E;
  a.k = k;
  a.groups = groups;
  a.top_groups = top_groups;
  a.sigmoid = score == MX_SCORE_SIGMOID;
  a.renormalize = renormalize != 0;
  a.bf16 = logits_type == MX_TYPE_BF16;
  a.scale = scale;
  a.experts = experts;
  a.weights = weights;
  return launched([&] { return mxq::launch_route(a, as_stream(stream)); });
}

mx_status mx_route_backward(const float* grad_weights, const void* logits, int logits_type,
                            const int32_t* experts, int64_t T, int E, int k, int score,
                            int renormalize, float scale, void* grad_logits, void* stream) {
  mx_status st = check_route(T, E, k, logits_type, score);
  if (st != MX_OK) return st;
  if (T == 0) return MX_OK;
  if (!grad_weights || !logits || !experts || !grad_logits) return MX_ERR_NULL;
  const uintptr_t el = logits_type == MX_TYPE_BF16 ? 2 : 4;
  if (!aligned(logits, el) || !aligned(grad_logits, el) || !aligned(grad_weights, 4) ||
      !aligned(experts, 4)) {
    return MX_ERR_ALIGN;
  }
  mxq::RouteArgs a{};
  a.logits = logits;
  a.T = T;
  a.E = E;
  a.k = k;
  a.sigmoid = score == MX_SCORE_SIGMOID;
  a.renormalize = renormalize != 0;
  a.bf16 = logits_type == MX_TYPE_BF16;
  a.scale = scale;
  a.grad_weights = grad_weights;
  a.chosen = experts;
  a.grad_logits = grad_logits;
  return launched([&] { return mxq::launch_route_backward(a, as_stream(stream)); });
}

mx_status mx_route_plan_workspace(int64_t T, int k, int E, int64_t* bytes) {
  if (!bytes) return MX_ERR_NULL;
  if (T < 0 || k < 1 || E < 1 || E > 1024 || T > INT32_MAX / k) return MX_ERR_SHAPE;
  *bytes = mxq::plan_workspace_ints(T * k, E) * 4;
  return MX_OK;
}

mx_status mx_route_plan(const int32_t* experts, int64_t T, int k, int E, int64_t* row_offsets,
                        int32_t* tokens, int32_t* slots, void* workspace, void* stream) {
  int64_t bytes = 0;
  const mx_status st = mx_route_plan_workspace(T, k, E, &bytes);
  if (st != MX_OK) return st;
  if (!row_offsets) return MX_ERR_NULL;
  if (T > 0 && (!experts || !tokens || !slots)) return MX_ERR_NULL;
  if (bytes > 0 && !workspace) return MX_ERR_NULL;
  if (!aligned(row_offsets, 8) || !aligned(experts, 4) || !aligned(tokens, 4) ||
      !aligned(slots, 4) || !aligned(workspace, 4)) {
    return MX_ERR_ALIGN;
  }
  mxq::PlanArgs a{};
  a.experts = experts;
  a.n = T * k;
  a.k = k;
  a.E = E;
  a.offsets = row_offsets;
  a.tokens = tokens;
  a.slots = slots;
  a.workspace = static_cast<int32_t*>(workspace);
  return launched([&] { return mxq::launch_plan(a, as_stream(stream)); });
}

mx_status mx_b128_padded_rows(int64_t R, int E, int64_t* rows) {
  if (!rows) return MX_ERR_NULL;
  if (R < 0 || E < 1 || E > 1024) return MX_ERR_SHAPE;
  if (R > INT32_MAX - 128 * int64_t(1025)) return MX_ERR_SHAPE;
  *rows = (R + 127 * (int64_t)E) / 128 * 128;
  return MX_OK;
}

mx_status mx_quantize_b128_rows(const void* x, int64_t M, int64_t K, const int32_t* index, int64_t R,
                                void* codes, float* scales, void* stream) {
  if (!sizes_ok(M, K) || !sizes_ok(R, K) || K % 32 != 0) return MX_ERR_SHAPE;
  if (!index && R != M && R != 0) return MX_ERR_SHAPE;
  if (R == 0 || K == 0) return MX_OK;
  if ((M > 0 && !x) || !codes || !scales) return MX_ERR_NULL;
  if (!aligned(x, 32) || !aligned(codes, 32) || !aligned(scales, 4) || !aligned(index, 4)) {
    return MX_ERR_ALIGN;
  }
  mxq::B128QuantArgs a{};
  a.x = x;
  a.index = index;
  a.batch = 1;
  a.M = M;
  a.K = K;
  a.R = R;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  return launched([&] { return mxq::launch_b128_rows(a, as_stream(stream)); });
}

mx_status mx_quantize_b128_cols(const void* x, int64_t M, int64_t K, const int32_t* index, int64_t R,
                                const int64_t* row_offsets, int E, void* codes, float* scales,
                                void* stream) {
  if (!sizes_ok(M, K) || !sizes_ok(R, K) || K % 32 != 0) return MX_ERR_SHAPE;
  if (!index && R != M && R != 0) return MX_ERR_SHAPE;
  if (!row_offsets && E != 1) return MX_ERR_SHAPE;
  int64_t rows = 0;
  const mx_status st = mx_b128_padded_rows(R, E, &rows);
  if (st != MX_OK) return st;
  if (rows == 0 || K == 0) return MX_OK;
  if ((M > 0 && !x) || !codes || !scales) return MX_ERR_NULL;
  if (!aligned(x, 32) || !aligned(codes, 32) || !aligned(scales, 4) || !aligned(index, 4) ||
      !aligned(row_offsets, 8)) {
    return MX_ERR_ALIGN;
  }
  mxq::B128QuantArgs a{};
  a.x = x;
  a.index = index;
  a.batch = 1;
  a.M = M;
  a.K = K;
  a.R = R;
  a.offsets = row_offsets;
  a.E = E;
  a.blocks = rows / 128;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  return launched([&] { return mxq::launch_b128_cols(a, as_stream(stream)); });
}

mx_status mx_quantize_b128_blocks(const void* x, int64_t batch, int64_t M, int64_t K, void* codes,
                                  float* scales, void* codes_t, float* scales_t, void* stream) {
  if (batch < 0 || batch > 65535 || !sizes_ok(M, K) || K % 32 != 0) return MX_ERR_SHAPE;
  if (batch > 0 && M * K > (int64_t(1) << 40) / batch) return MX_ERR_SHAPE;
  if (ceil_div(M, 128) * ceil_div(K, 128) > INT32_MAX) return MX_ERR_SHAPE;
  if (batch == 0 || M == 0 || K == 0) return MX_OK;
  if (!x || !codes || !scales || (codes_t == nullptr) != (scales_t == nullptr)) return MX_ERR_NULL;
  if (!aligned(x, 32) || !aligned(codes, 32) || !aligned(scales, 4) || !aligned(codes_t, 32) ||
      !aligned(scales_t, 4)) {
    return MX_ERR_ALIGN;
  }
  mxq::B128QuantArgs a{};
  a.x = x;
  a.batch = batch;
  a.M = M;
  a.K = K;
  a.R = M;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = scales;
  a.codes_t = static_cast<uint8_t*>(codes_t);
  a.scales_t = scales_t;
  return launched([&] { return mxq::launch_b128_blocks(a, as_stream(stream)); });
}

mx_status mx_gemm_b128(const void* a_codes, const float* a_scales, const void* b_codes,
                       const float* b_scales, int64_t M, int64_t N, int64_t K, int b_form,
                       int c_type, void* c, void* stream) {
  return dense(a_codes, a_scales, b_codes, b_scales, M, N, K, b_form, c_type, c, kWaitNs, stream);
}

mx_status mx_selftest_gemm_b128_give_up(const void* a_codes, const float* a_scales,
                                        const void* b_codes, const float* b_scales, int64_t M,
                                        int64_t N, int64_t K, int b_form, void* c, int64_t limit_ns,
                                        void* stream) {
  if (limit_ns <= 0 || limit_ns > 100000000) return MX_ERR_SHAPE;
  if (M == 0 || N == 0) return MX_ERR_SHAPE;  // a launch is the point
  return dense(a_codes, a_scales, b_codes, b_scales, M, N, K, b_form, MX_TYPE_BF16, c,
               (unsigned long long)limit_ns, stream);
}

mx_status mx_gemm_b128_grouped(const void* a_codes, const float* a_scales, const void* b_codes,
                               const float* b_scales, const int64_t* row_offsets, int E,
                               int64_t M_total, int64_t N, int64_t K, int c_type, void* c,
                               void* stream) {
  return grouped(a_codes, a_scales, b_codes, b_scales, row_offsets, E, M_total, N, K, c_type, c, kWaitNs,
                 stream);
}

mx_status mx_selftest_gemm_b128_grouped_give_up(const void* a_codes, const float* a_scales,
                                                const void* b_codes, const float* b_scales,
                                                const int64_t* row_offsets, int E, int64_t M_total,
                                                int64_t N, int64_t K, void* c, int64_t limit_ns,
                                                void* stream) {
  if (limit_ns <= 0 || limit_ns > 100000000) return MX_ERR_SHAPE;
  if (M_total == 0 || N == 0) return MX_ERR_SHAPE;  // a launch is the point
  return grouped(a_codes, a_scales, b_codes, b_scales, row_offsets, E, M_total, N, K, MX_TYPE_BF16, c,
                 (unsigned long long)limit_ns, stream);
}

mx_status mx_gemm_b128_grouped_wgrad(const void* a_codes, const float* a_scales,
                                     const void* b_codes, const float* b_scales,
                                     const int64_t* row_offsets, int E, int64_t M, int64_t N,
                                     int64_t R_padded, int c_type, void* c, void* stream) {
  mx_status st = check_b128_gemm(M, N, R_padded, c_type);
  if (st != MX_OK) return st;
  if (E < 1 || E > 1024 || R_padded % 128 != 0) return MX_ERR_SHAPE;
  if (M > 0 && N > 0 && M * N > (int64_t(1) << 40) / E) return MX_ERR_SHAPE;
  if (M == 0 || N == 0) return MX_OK;
  if (R_padded == 0) {  // no rows at all: every sum is empty
    if (!c) return MX_ERR_NULL;
    if (!aligned(c, 16)) return MX_ERR_ALIGN;
    return from_cuda(cudaMemsetAsync(c, 0, (size_t)(M * N * E) * (c_type == MX_TYPE_FP32 ? 4 : 2),
                                     as_stream(stream)));
  }
  if (!row_offsets) return MX_ERR_NULL;
  st = check_b128_pointers(a_codes, a_scales, b_codes, b_scales, c);
  if (st != MX_OK) return st;
  if (!aligned(row_offsets, 8)) return MX_ERR_ALIGN;
  mxq::B128GemmArgs g{};
  g.a_codes = a_codes;
  g.a_scales = a_scales;
  g.b_codes = b_codes;
  g.b_scales = b_scales;
  g.c = c;
  g.M = M;
  g.N = N;
  g.K = R_padded;
  g.offsets = row_offsets;
  g.rows_total = R_padded;
  g.E = E;
  g.b_rows = true;
  g.out_f32 = c_type == MX_TYPE_FP32;
  return run_gemm(mxq::kB128Wgrad, g, kWaitNs, stream);
}

namespace {
mx_status check_combine(int64_t T, int k, int64_t R, int64_t N) {
  if (T < 0 || k < 1 || k > 64 || R < 0 || N < 0 || N % 8 != 0) return MX_ERR_SHAPE;
  if (T > INT32_MAX / k || R > INT32_MAX || N > INT32_MAX) return MX_ERR_SHAPE;
  if (N > 0 && (T * k > (int64_t(1) << 40) / N || R > (int64_t(1) << 40) / N)) return MX_ERR_SHAPE;
  return MX_OK;
}
}  // namespace

mx_status mx_combine(const void* y, const int32_t* slots, const float* weights, int64_t T, int k,
                     int64_t R, int64_t N, void* out, void* stream) {
  const mx_status st = check_combine(T, k, R, N);
  if (st != MX_OK) return st;
  if (T == 0 || N == 0) return MX_OK;
  if ((R > 0 && !y) || !slots || !out) return MX_ERR_NULL;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(slots, 4) || !aligned(weights, 4)) {
    return MX_ERR_ALIGN;
  }
  mxq::CombineArgs a{};
  a.y = y;
  a.slots = slots;
  a.weights = weights;
  a.T = T;
  a.R = R;
  a.N = N;
  a.k = k;
  a.out = out;
  return launched([&] { return mxq::launch_combine(a, as_stream(stream)); });
}

namespace {
mx_status combine_backward(const void* dout, const void* y, const int32_t* slots, const float* weights,
                           int64_t T, int k, int64_t R, int64_t N, void* dy, float* dweights,
                           int32_t* owner, void* stream) {
  if (T > 0 && (!slots || (N > 0 && (!dout || (R > 0 && !dy) || (R > 0 && dweights && !y))))) {
    return MX_ERR_NULL;
  }
  if (!aligned(y, 16) || !aligned(dout, 16) || !aligned(dy, 16) || !aligned(slots, 4) ||
      !aligned(weights, 4) || !aligned(dweights, 4) || !aligned(owner, 4)) {
    return MX_ERR_ALIGN;
  }
  mxq::CombineArgs a{};
  a.y = y;
  a.slots = slots;
  a.weights = weights;
  a.dout = dout;
  a.T = T;
  a.R = R;
  a.N = N;
  a.k = k;
  a.dy = dy;
  a.dweights = dweights;
  a.owner = owner;
  return launched([&] { return mxq::launch_combine_backward(a, as_stream(stream)); });
}
}  // namespace

mx_status mx_combine_backward(const void* dout, const void* y, const int32_t* slots,
                              const float* weights, int64_t T, int k, int64_t R, int64_t N,
                              void* dy, float* dweights, void* stream) {
  const mx_status st = check_combine(T, k, R, N);
  if (st != MX_OK) return st;
  if (T == 0) return MX_OK;
  return combine_backward(dout, y, slots, weights, T, k, R, N, dy, dweights, nullptr, stream);
}

mx_status mx_combine_backward_whole(const void* dout, const void* y, const int32_t* slots,
                                    const float* weights, int64_t T, int k, int64_t R, int64_t N,
                                    void* dy, float* dweights, void* workspace, void* stream) {
  const mx_status st = check_combine(T, k, R, N);
  if (st != MX_OK) return st;
  if (R > 0 && N > 0 && (!dy || !workspace)) return MX_ERR_NULL;
  return combine_backward(dout, y, slots, weights, T, k, R, N, dy, dweights,
                          R > 0 && N > 0 ? static_cast<int32_t*>(workspace) : nullptr, stream);
}

}  // extern "C"
