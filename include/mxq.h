/*
 * mxq.h -- C ABI of libmxq: OCP-MX block quantization (MXFP4 / MXFP8) on one GB300 GPU.
 *
 * What the library computes (sources are the pages this library restates):
 *  - "[Transform] [Quantization] Add QuTLASS support to vLLM" (vllm PR 24440), feature list:
 *    abs-max block scales ("Multiple quantization schemes ... Abs-Max"), the MXFP4 format,
 *    "Fused transform + quantization + scale computation", rotation matrices "loaded at
 *    runtime, allowing any transformation", rotation sizes 16/32/64/128; review thread on
 *    vllm/_custom_ops.py (`fusedQuantizeMx(a, b, ...)` returning packed E2M1 codes and E8M0
 *    scales of shape `padded_rows x padded_cols`) and on vllm/qutlass_utils/utils.py
 *    (`to_blocked`: the blocked scale layout block-scaled GEMMs consume).
 *  - "use cute-dsl to speedup mxfp QDQ" (intel/neural-compressor PR 2548), Description:
 *    MXFP4 / MXFP8 QDQ on contiguous input, group size 32, K divisible by 32, CUDA-Graph use.
 *  - prhub summary of vllm PR 47229, code snippet of mxfp8_utils.py: MXFP8 (E4M3) quantize
 *    with MXFP8_BLOCK_SIZE = 32 returning codes and scales, scales viewed as [M, K/32] when not
 *    swizzled, or in the swizzled layout when `is_sf_swizzled_layout`.
 *
 * Arithmetic (the pages name the formats but print no formula; this is the OCP MX reading):
 *  For every block of 32 consecutive elements along K of a bf16 row-major [M, K] matrix:
 *    amax = max |v_i|;  s = clamp(floor(log2 amax) - emax, -127, 127)  (emax = 2 for E2M1,
 *    8 for E4M3; an all-zero block gets s = -127);  E8M0 scale byte = s + 127;
 *    code_i = v_i / 2^s rounded to nearest-even on the element grid, saturating at the largest
 *    finite magnitude (6 for E2M1, 448 for E4M3), sign kept (also for zero);
 *    QDQ output_i = bf16_round_nearest_even(decode(code_i) * 2^s).
 *  A block holding a NaN or an infinity gets scale byte 0xFF; its codes are 0x7F (E4M3) or
 *  0x0 (E2M1) and its QDQ outputs are the bf16 NaN 0x7FC0.
 *
 * Conventions for every entry point:
 *  - Pointers named x, y, codes, scales, H, row_offsets are DEVICE memory owned by the caller;
 *    the library never allocates, frees or synchronizes, and never reads device memory on the
 *    host. Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default stream) and is
 *    asynchronous.
 *  - Validation happens on the host before any launch; on error nothing is launched and the
 *    status says why. After the launch, a launch failure maps to MX_ERR_CUDA.
 *  - x, y and codes must be 32-byte aligned, H and swizzled scales 16-byte aligned; rows
 *    are contiguous.
 *  - M == 0 or K == 0 is a valid empty call: nothing is launched, MX_OK is returned.
 *  - Layouts: E4M3 codes are [M, K] bytes (float8_e4m3fn). E2M1 codes are [M, K/2] bytes, two
 *    codes per byte, the lower K index in the low nibble. Linear scales are [M, K/32] bytes,
 *    row-major. Swizzled scales are [ceil(M/128)*128, ceil(K/128)*4] bytes: the scale matrix is
 *    padded with zero bytes and cut into 128x4 tiles of 512 bytes, stored row-block-major; scale
 *    (r, c) of a tile sits at byte (r % 32) * 16 + (r / 32) * 4 + c. Every byte, pads
 *    included, is written by each call.
 */
#ifndef MXQ_H
#define MXQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int mx_status;

/* status codes */
#define MX_OK 0
#define MX_ERR_NULL 1        /* a required pointer is NULL */
#define MX_ERR_SHAPE 2       /* negative size, K % 32 != 0, K % g != 0, bad expert count */
#define MX_ERR_ALIGN 3       /* misaligned pointer (x, y, codes: 32 B; H, scales: 16 B) */
#define MX_ERR_UNSUPPORTED 4 /* unknown format / layout / rounding, group != 32, bad g */
#define MX_ERR_CUDA 5        /* the CUDA runtime reported an error at launch */

/* element formats */
#define MX_FMT_E2M1 1 /* MXFP4: 1 sign, 2 exponent, 1 mantissa bit */
#define MX_FMT_E4M3 2 /* MXFP8: 1 sign, 4 exponent, 3 mantissa bits ("fn": max 448, no Inf) */

/* scale layouts */
#define MX_SCALES_LINEAR 0   /* [M, K/32] row-major */
#define MX_SCALES_SWIZZLED 1 /* 128x4 blocked tiles, padded (see above) */

/*
 * Rounding schemes (argument `rounding`): how the block scale is chosen. The elements are always
 * rounded to nearest even with saturation under the chosen scale.
 *  MX_ROUND_RNE: the abs-max scale above (the QuTLASS feature list's "Abs-Max" scheme).
 *  MX_ROUND_QUEST: the Quartet / "Quest-like" scale (QuTLASS feature list: "Multiple
 *    quantization schemes ... Quartet (i.e., Quest-like)"; the review thread on
 *    vllm/_custom_ops.py names its call fusedQuantizeMxQuest(a, b, xh_e2m1, xh_e8m0)). MXFP4
 *    (MX_FMT_E2M1) only; not for grouped calls. The pages print no rule; the reading is the
 *    rule above with the block's clip point c in place of amax:
 *      c = alpha * sqrt(sum_i v_i^2 / 32),  s = clamp(floor(log2 c) - 2, -127, 127),
 *    alpha = 2.922475, the ratio of clip point to standard deviation that minimises the mean
 *    squared error of the E2M1 grid (its largest value 6 at the clip point) on a normally
 *    distributed input; values above 6 * 2^s saturate (the clipping). An all-zero block gets
 *    byte 0, a block with a NaN or an infinity 0xFF as above. The sum of squares is formed in
 *    fp32 after an exact power-of-two scaling (no overflow or underflow for any finite input),
 *    so s can differ from the real-number rule only where c lies within about 2^-20 relative of
 *    a power of two.
 */
#define MX_ROUND_RNE 0
#define MX_ROUND_QUEST 1

/*
 * Rotation kinds (argument rot_kind of the rotating calls; ignored where H is NULL).
 *  MX_ROT_DENSE: H is any bf16 [g, g] matrix; the product runs on the tensor cores (calls
 *    with at most 16 rows and M * g <= 512: fp32 FMAs).
 *  MX_ROT_HADAMARD: the caller states that H = c * S_g, where S_g is the Sylvester Hadamard
 *    matrix of order g (S_1 = [1], S_2n = [[S_n, S_n], [S_n, -S_n]], entry (i, j) =
 *    (-1)^popcount(i & j)) and c = H[0][0], e.g. the normalized hadamard(g) * g^-0.5 rounded
 *    to bf16. For g <= 64 the product is then a fast Walsh-Hadamard transform in registers
 *    (log2 g butterfly stages in fp32, then a multiplication by c) on the streaming kernel.
 *    Every CTA checks the statement on the bit patterns of H on the device; where it does not
 *    hold the call computes sum_i x_i H[i][j] with fp32 FMAs instead, so the results are
 *    correct for any H (only slower). For g = 128 the call runs as MX_ROT_DENSE (faster
 *    there).
 *  MX_ROT_AUTO: the same statement as MX_ROT_HADAMARD; the library takes whichever of the two
 *    kernels measured faster on GB300 for the call: the fp32-FMA kernel for decode-sized calls
 *    (M <= 16, M * g <= 512) and the tensor cores for g = 128; otherwise the Walsh-Hadamard
 *    kernel below 4096 rows, and from 4096 rows the tensor cores for 4-bit codes (MXFP4, NVFP4)
 *    and for MXFP8 codes or QDQ outputs while M * K <= 3 * 2^25, the Walsh-Hadamard kernel above.
 *    mx_rotate_debug treats it as MX_ROT_HADAMARD.
 * The kinds compute the same rotation up to fp32 rounding (well inside the 1e-5 normwise
 * tolerance of the rotated path).
 */
#define MX_ROT_DENSE 0
#define MX_ROT_HADAMARD 1
#define MX_ROT_AUTO 2

/* Text of a status code (static storage). */
const char* mx_status_string(mx_status status);

/*
 * Shape of the scale matrix for an [M, K] input: linear [M, K/32]; swizzled
 * [ceil(M/128)*128, ceil(K/128)*4]. Host only, launches nothing.
 * Errors: MX_ERR_NULL (rows or cols NULL), MX_ERR_SHAPE (M < 0, K < 0, K % 32),
 * MX_ERR_UNSUPPORTED (group != 32, unknown layout).
 */
mx_status mx_scales_shape(int64_t M, int64_t K, int group, int layout, int64_t* rows,
                          int64_t* cols);

/*
 * Block quantize (pages: fusedQuantizeMx without the rotation; mxfp8_quantize).
 * x: bf16 [M, K]. codes: see layouts. scales: per `layout`. fmt: MX_FMT_*. group: must be 32.
 * rounding: MX_ROUND_RNE, or MX_ROUND_QUEST with MX_FMT_E2M1. Errors: see conventions.
 */
mx_status mx_quantize(const void* x, int64_t M, int64_t K, int fmt, int group, int layout,
                      int rounding, void* codes, void* scales, void* stream);

/*
 * QDQ: quantize then dequantize, bf16 in, bf16 out (pages: mxfp4_qdq / mxfp8_qdq).
 * If H is not NULL, every g-element chunk along K is first rotated, y_chunk = x_chunk * H
 * (H: bf16 [g, g] row-major device matrix, g in {16, 32, 64, 128}, K % g == 0, rot_kind an
 * MX_ROT_* value), and the rotated values are quantized; the output stays in the rotated
 * basis. If H is NULL, g and rot_kind are ignored. y: bf16 [M, K], must not overlap x.
 * rounding as in mx_quantize.
 */
mx_status mx_qdq(const void* x, int64_t M, int64_t K, int fmt, int group, int rounding,
                 const void* H, int g, int rot_kind, void* y, void* stream);

/*
 * Dequantize stored MX data to bf16 (pages: the QuTLASS review thread on vLLM's MXFP4 test,
 * which dequantizes packed E2M1 codes with their E8M0 scales, `_dq_fp4(b_e2m1, b_e8m0, ...)`,
 * before a reference matmul; the dequantize half of mxfp4_qdq / mxfp8_qdq).
 * y_i = bf16_round_nearest_even(decode(code_i) * 2^(scale_byte - 127)) for every element, so
 * mx_dequantize(mx_quantize(x)) == mx_qdq(x) bit for bit. Any code and scale byte is accepted:
 * scale byte 0xFF (E8M0 NaN) and E4M3 codes S.1111.111 give the bf16 NaN 0x7FC0, products
 * above the bf16 range give +-Inf, tiny products round to bf16 subnormals or signed zero.
 * codes: E2M1 [M, K/2] or E4M3 [M, K] bytes (32-byte aligned), laid out as mx_quantize writes
 * them. scales: linear [M, K/32] or swizzled (16-byte aligned) as returned by
 * mx_scales_shape(); pad bytes are not read. y: bf16 [M, K] (32-byte aligned), must not
 * overlap the inputs. Errors: see conventions.
 */
mx_status mx_dequantize(const void* codes, const void* scales, int64_t M, int64_t K, int fmt,
                        int group, int layout, void* y, void* stream);

/*
 * Fused rotate + quantize (pages: fusedQuantizeMx(a, b) with b the runtime-loaded rotation).
 * y_chunk = x_chunk * H for every g-chunk along K (bf16 products, fp32 accumulation; see
 * MX_ROT_* for how), then the block quantization above on the fp32 rotated values.
 * H: bf16 [g, g] row-major, g in {16, 32, 64, 128}, K % g == 0. rot_kind: MX_ROT_*. Other
 * arguments as mx_quantize.
 */
mx_status mx_rotate_quantize(const void* x, int64_t M, int64_t K, const void* H, int g,
                             int rot_kind, int fmt, int group, int layout, int rounding,
                             void* codes, void* scales, void* stream);

/*
 * Scale-matrix shape for a grouped call with E experts and M_total rows: linear
 * [M_total, K/32]; swizzled [R, ceil(K/128)*4] with R = floor((M_total + 127*E) / 128) * 128,
 * an upper bound of sum_e ceil(n_e/128)*128 valid for any split of M_total rows.
 */
mx_status mx_grouped_scales_shape(int64_t M_total, int E, int64_t K, int group, int layout,
                                  int64_t* rows, int64_t* cols);

/*
 * Grouped (MoE expert) quantize. Rows [row_offsets[e], row_offsets[e+1]) of x belong to
 * expert e (row_offsets: DEVICE int64 [E+1], row_offsets[0] = 0, row_offsets[E] = M_total,
 * non-decreasing). Codes stay contiguous as for mx_quantize on the whole x. Linear scales are
 * [M_total, K/32]: the call is then mx_quantize on the whole x and does not read row_offsets.
 * Swizzled scales give each expert its own run of 128-row tiles: expert e's
 * rows start at padded row P_e = sum_{e' < e} ceil(n_e'/128) * 128; the buffer has
 * mx_grouped_scales_shape() rows and all of it is written (rows past the last expert: zero).
 * 1 <= E <= 1024. Offsets that break the contract give unspecified values but every access
 * stays inside x, codes and scales. rounding: MX_ROUND_RNE (MX_ROUND_QUEST: MX_ERR_UNSUPPORTED).
 */
mx_status mx_quantize_grouped(const void* x, const int64_t* row_offsets, int E, int64_t M_total,
                              int64_t K, int fmt, int group, int layout, int rounding,
                              void* codes, void* scales, void* stream);

/*
 * NVFP4 (pages: the QuTLASS feature list, "Support for both NVFP4 and MXFP4", and its review
 * thread on benchmarks/kernels/bench_nvfp4_qutlass.py: fusedQuantizeNv(a, H, global_scale)
 * returning E2M1 codes and blocked scales viewed as [-1, K/16]). E2M1 codes in blocks of 16
 * along K, one E4M3 scale byte per block, under a per-tensor fp32 global scale gs. The pages
 * print no scale rule; the reading is the usual two-level one, every step one fp32 operation
 * rounded to nearest even, in this order, per block with abs-max amax:
 *   s_f = amax * (gs / 6);  scale byte = E4M3(s_f), saturating at 448;
 *   enc = gs / decode(scale);  code_i = E2M1(v_i * enc)  (enc = 0 when decode(scale) == 0);
 *   QDQ: y_i = bf16(decode(code_i) * (decode(scale) / gs))  (0 factor likewise).
 * A block holding a NaN or an infinity gets scale byte 0x7F, codes 0 and QDQ outputs 0x7FC0.
 * With H (bf16 [g, g], g in {16, 32, 64, 128}, K % g == 0) every g-chunk is first rotated,
 * y_chunk = x_chunk * H (fp32 accumulation; rot_kind as in mx_rotate_quantize, ignored without
 * H), as in mx_rotate_quantize.
 * global_scale: DEVICE pointer to one fp32 value, 4-byte aligned, read by the kernel (so it may
 * come from an earlier kernel on the same stream); it must be positive and finite, and
 * gs / 2^-9 must not overflow fp32 (gs < 1.7e38 * 2^-9), else results are unspecified.
 * K % 32 == 0. Codes: [M, K/2] bytes (32-byte aligned), the lower K index in the low nibble.
 * Scales: linear [M, K/16] (2-byte aligned) or swizzled [ceil(M/128)*128, ceil(K/64)*4]
 * (16-byte aligned; 128x4 tiles as for the MX scales, pads zero), see mx_nvfp4_scales_shape.
 */
mx_status mx_nvfp4_scales_shape(int64_t M, int64_t K, int layout, int64_t* rows, int64_t* cols);

mx_status mx_quantize_nvfp4(const void* x, int64_t M, int64_t K, const void* H, int g,
                            int rot_kind, const float* global_scale, int layout, void* codes,
                            void* scales, void* stream);

/* NVFP4 QDQ (see above): bf16 y [M, K], 32-byte aligned, must not overlap x. */
mx_status mx_qdq_nvfp4(const void* x, int64_t M, int64_t K, const void* H, int g, int rot_kind,
                       const float* global_scale, void* y, void* stream);

/*
 * Grouped (MoE expert) NVFP4 quantize: rows [row_offsets[e], row_offsets[e+1]) of x are expert
 * e's input and are quantized as by mx_quantize_nvfp4 (no rotation) under that expert's own
 * global scale global_scales[e] (DEVICE fp32 [E], 4-byte aligned, each positive and finite;
 * pass E equal values for one shared scale). row_offsets: DEVICE int64 [E+1] with the contract
 * of mx_quantize_grouped. Codes stay contiguous [M_total, K/2]. Linear scales are
 * [M_total, K/16] (2-byte aligned); swizzled scales give each expert its own run of 128-row
 * tiles starting at padded row P_e = sum_{e' < e} ceil(n_e'/128) * 128, in a buffer of
 * mx_nvfp4_grouped_scales_shape() bytes that is written whole (pads zero; 16-byte aligned).
 * 1 <= E <= 1024, K % 32 == 0.
 */
mx_status mx_nvfp4_grouped_scales_shape(int64_t M_total, int E, int64_t K, int layout,
                                        int64_t* rows, int64_t* cols);

mx_status mx_quantize_nvfp4_grouped(const void* x, const int64_t* row_offsets, int E,
                                    int64_t M_total, int64_t K, const float* global_scales,
                                    int layout, void* codes, void* scales, void* stream);

/*
 * NVFP4 dequantize (the dequantize half of NVFP4 QDQ; see the NVFP4 reading above):
 * y_i = bf16(decode(code_i) * (decode(scale) / gs)) with each 16-element block's E4M3 scale
 * byte decoded as a signed E4M3 value (0 factor when it decodes to zero), every step one fp32
 * operation rounded to nearest even, so mx_dequantize_nvfp4(mx_quantize_nvfp4(x)) ==
 * mx_qdq_nvfp4(x) bit for bit (same H, same gs). Scale bytes 0x7F / 0xFF (the E4M3 NaN) give
 * 0x7FC0 for their block. codes: [M, K/2] bytes (32-byte aligned). scales: linear [M, K/16]
 * (2-byte aligned) or swizzled as mx_nvfp4_scales_shape() (16-byte aligned; pads not read).
 * global_scale: DEVICE pointer to one positive finite fp32 value (4-byte aligned). y: bf16
 * [M, K] (32-byte aligned), must not overlap the inputs. K % 32 == 0. Errors: see conventions.
 */
mx_status mx_dequantize_nvfp4(const void* codes, const void* scales, int64_t M, int64_t K,
                              const float* global_scale, int layout, void* y, void* stream);

/*
 * Block-scaled GEMM consumer (pages: the QuTLASS review thread on vLLM's MXFP4 test, which runs
 * matmul_mxf4_bf16_tn(a_e2m1, b_e2m1, a_e8m0, b_e8m0, alpha) on the quantizer's outputs and
 * compares it with the matmul of the dequantized operands `_dq_fp4(...)`):
 *   C[i][j] = alpha * sum_k dequant(A)[i][k] * dequant(B)[j][k]   ("TN": both K-major),
 * dequant as in mx_dequantize (decode(code) * 2^(scale_byte - 127) rounded to bf16 once: exact
 * for every E2M1 value and for E4M3 unless below the bf16 range), products exact, sums in fp32
 * on the tensor cores, C rounded to bf16 once. A: codes [M, K/2] (E2M1) or [M, K] (E4M3) with
 * scales [M, K/32] (linear) or the 128x4 blocked layout of mx_scales_shape(M, K) (swizzled), as
 * mx_quantize writes them; B likewise with N rows; both in the same fmt and layout. C: bf16
 * [M, N] row-major, must not overlap the inputs. K % 64 == 0 (K > 0), N % 8 == 0; codes and C
 * 16-byte aligned, linear scales 2-byte aligned, swizzled scales 16-byte aligned. A scale byte
 * 0xFF makes its 32 values NaN.
 * M <= 8,388,480 (65,535 tiles of 128 rows). M == 0 or N == 0 is a no-op returning MX_OK.
 * Errors: see conventions; K not a positive multiple of 64, N % 8 or M too large ->
 * MX_ERR_SHAPE.
 */
mx_status mx_gemm(const void* a_codes, const void* a_scales, const void* b_codes,
                  const void* b_scales, int64_t M, int64_t N, int64_t K, int fmt, int group,
                  int layout, float alpha, void* c, void* stream);

/* ------------------------------------------------------------------------------------------
 * Expert layers: routing tokens to experts, 8-bit operands with one scale per block of 128, the
 * products of such operands (dense, by expert, and for weight gradients) and the combination of
 * the experts' outputs. The conventions at the top of this file hold; alignment is stated per
 * call. These have no counterpart on the pages; mx_quantize_grouped takes the row_offsets of
 * mx_route_plan too.
 * ------------------------------------------------------------------------------------------ */

/* element types of logits and of products */
#define MX_TYPE_BF16 0
#define MX_TYPE_FP32 1

/* scores of mx_route */
#define MX_SCORE_SOFTMAX 0
#define MX_SCORE_SIGMOID 1

/*
 * Routing. For each of T tokens with logits l [T, E] (MX_TYPE_BF16 or MX_TYPE_FP32):
 *   s = softmax(l) or sigmoid(l) over the E experts, in fp32;
 *   choice c = s + bias (bias: DEVICE fp32 [E] or NULL; it takes part in the choice only); without
 *   a bias the softmax choice is exp(l - max l), which orders the experts as s does;
 *   an expert whose l (or c) is -inf is never chosen;
 *   groups > 1: the E experts form `groups` equal runs, a run's score is the sum of its two
 *   largest c (of its only one where it has one), and only the top_groups best runs stay;
 *   experts[t, :] = the k experts of largest c, descending; ties go to the lowest index (runs
 *   likewise), a NaN ranks below every number; -1 where none is left;
 *   weights[t, j] = scale * s[experts[t, j]] (/ the sum of the k scores when renormalize != 0; 0
 *   where that sum is 0), 0 where experts[t, j] = -1.
 * A NaN logit makes its token's softmax NaN. 1 <= E <= 1024, 1 <= k <= min(E, 32), 1 <= groups
 * <= 32, E % groups == 0, k <= top_groups * E / groups, T * k < 2^31. experts: int32 [T, k],
 * weights: fp32 [T, k]. Alignment: that of the elements.
 */
mx_status mx_route(const void* logits, int logits_type, const float* bias, int64_t T, int E, int k,
                   int score, int groups, int top_groups, int renormalize, float scale,
                   int32_t* experts, float* weights, void* stream);

/*
 * Gradient of the logits through the weights of mx_route (the choice is taken as fixed; the bias
 * has none). grad_weights: fp32 [T, k]; experts: as mx_route wrote them; grad_logits: [T, E] of
 * the logits' type, written whole. With p the chosen scores, P their sum and g = grad_weights:
 * dp_j = scale * (g_j - sum_i g_i p_i / P) / P when renormalize != 0, else scale * g_j; then
 * s_i (1 - s_i) dp_i (sigmoid) or s_i (dp_i - sum_j dp_j s_j) (softmax).
 */
mx_status mx_route_backward(const float* grad_weights, const void* logits, int logits_type,
                            const int32_t* experts, int64_t T, int E, int k, int score,
                            int renormalize, float scale, void* grad_logits, void* stream);

/*
 * Plan of the expert rows: the T * k choices ordered by expert, and by (token, j) within one.
 * row_offsets: int64 [E + 1], expert e owns rows [row_offsets[e], row_offsets[e + 1]);
 * tokens: int32 [T * k], the token of each row, -1 from row_offsets[E] on; slots: int32 [T, k], the
 * row of each choice, -1 for a choice of -1 (anything outside [0, E) counts as none). workspace:
 * device memory of mx_route_plan_workspace() bytes (may be NULL when that is 0), 4-byte aligned.
 */
mx_status mx_route_plan_workspace(int64_t T, int k, int E, int64_t* bytes);

mx_status mx_route_plan(const int32_t* experts, int64_t T, int k, int E, int64_t* row_offsets,
                        int32_t* tokens, int32_t* slots, void* workspace, void* stream);

/*
 * E4M3 operands with one fp32 scale per block of 128 along the contraction. For a block with
 * abs-max A: a = max(A, 2^-100), r = 448 / a, scale = a / 448, code_i = E4M3(x_i * r), every step
 * one fp32 operation rounded to nearest even, codes saturating at 448; a block with a NaN or an
 * infinity has scale NaN and codes 0x7F. x is bf16 (32-byte aligned, K % 32 == 0), codes are
 * 32-byte and scales 4-byte aligned. A last block may be shorter than 128.
 *
 * rows: 1 x 128 blocks along K of R rows. index (DEVICE int32 [R]) names the row of x [M, K] that
 * each of them is (an entry outside [0, M) gives a row of zeros); index NULL: R = M, row for row, or R = 0.
 *   codes [R, K]; scales [ceil(K / 128), R].
 * cols: 128 x 1 blocks along the rows, written transposed, for products that contract over the
 * rows of x. Rows as above; row_offsets (DEVICE int64 [E + 1]) makes each expert's rows start a
 * new block, filled up with zeros; NULL with E = 1: one run of R rows.
 *   codes [K, P], scales [P / 128, K], P = mx_b128_padded_rows(R, E) = floor((R + 127 E) / 128) * 128;
 *   expert e's columns start at the sum of its predecessors' row counts, each rounded up to 128;
 *   what lies past the last expert's is not written.
 * blocks: 128 x 128 squares of each of `batch` matrices [M, K] (M * K rows following one another).
 *   codes [batch, M, K], scales [batch, ceil(M / 128), ceil(K / 128)], and unless NULL the
 *   transposed operand: codes_t [batch, K, M], scales_t [batch, ceil(K / 128), ceil(M / 128)]
 *   (five times slower where M is no multiple of 16, whose columns are then written byte by byte).
 */
mx_status mx_b128_padded_rows(int64_t R, int E, int64_t* rows);

mx_status mx_quantize_b128_rows(const void* x, int64_t M, int64_t K, const int32_t* index, int64_t R,
                                void* codes, float* scales, void* stream);

mx_status mx_quantize_b128_cols(const void* x, int64_t M, int64_t K, const int32_t* index, int64_t R,
                                const int64_t* row_offsets, int E, void* codes, float* scales,
                                void* stream);

mx_status mx_quantize_b128_blocks(const void* x, int64_t batch, int64_t M, int64_t K, void* codes,
                                  float* scales, void* codes_t, float* scales_t, void* stream);

/* forms of B's scales in mx_gemm_b128 */
#define MX_B128_BLOCKS 0 /* [ceil(N / 128), ceil(K / 128)]: mx_quantize_b128_blocks */
#define MX_B128_ROWS 1   /* [ceil(K / 128), N]: mx_quantize_b128_rows or _cols */

/*
 * Products of such operands: C[i][j] = sum over blocks b of sa[b, i] sb[b, j] times the sum over
 * the block of a[i][k] b[j][k]; products and sums in fp32 on the tensor cores, C rounded once to
 * c_type (MX_TYPE_BF16 or MX_TYPE_FP32). Codes [rows, K], both K-major; A's scales in the rows
 * form. K % 32 == 0, N % 8 == 0; codes and C 16-byte aligned.
 * The factor sa[b, i] sb[b, j] is one fp32 product, taken first: where it is 2^128 or more (blocks whose
 * abs-maxes multiply to some 2^145) the entry is infinite or NaN whatever the sum, and below 2^-126 the
 * factor loses bits, an error of at most 2^-125 per block.
 *
 * mx_gemm_b128: A [M, K], B [N, K], B's scales in b_form; C [M, N]. K > 0.
 * mx_gemm_b128_grouped: rows [row_offsets[e], row_offsets[e + 1]) of A times B[e] [N, K] (B's
 *   scales in the blocks form, [E, ceil(N / 128), ceil(K / 128)]); rows of C [M_total, N] from
 *   row_offsets[E] on are not written. E * N < 2^31.
 * mx_gemm_b128_grouped_wgrad: A [M, R_padded] and B [N, R_padded] as mx_quantize_b128_cols writes
 *   them for the same row_offsets, scales in the rows form; C [E, M, N], C[e] contracts over expert
 *   e's rows and is 0 where it has none. R_padded % 128 == 0.
 * row_offsets: DEVICE int64 [E + 1], 0 first, non-decreasing, 1 <= E <= 1024. Offsets that break
 * that give unspecified values but every access stays inside the buffers.
 */
mx_status mx_gemm_b128(const void* a_codes, const float* a_scales, const void* b_codes,
                       const float* b_scales, int64_t M, int64_t N, int64_t K, int b_form,
                       int c_type, void* c, void* stream);

mx_status mx_gemm_b128_grouped(const void* a_codes, const float* a_scales, const void* b_codes,
                               const float* b_scales, const int64_t* row_offsets, int E,
                               int64_t M_total, int64_t N, int64_t K, int c_type, void* c,
                               void* stream);

mx_status mx_gemm_b128_grouped_wgrad(const void* a_codes, const float* a_scales,
                                     const void* b_codes, const float* b_scales,
                                     const int64_t* row_offsets, int E, int64_t M, int64_t N,
                                     int64_t R_padded, int c_type, void* c, void* stream);

/*
 * Combination of expert rows: out[t] = sum over j of weights[t, j] * y[slots[t, j]] (fp32, in the
 * order of j, rounded to bf16 once); weights NULL: all ones, the gradient of gathering rows by
 * token. A slot outside [0, R) adds nothing. y: bf16 [R, N], out: bf16 [T, N], 16-byte aligned,
 * N % 8 == 0; slots: int32 [T, k], weights: fp32 [T, k], 1 <= k <= 64.
 * Backward: dy[slots[t, j]] = weights[t, j] * dout[t] (rows of dy that no slot names are not
 * written; every row may be named once), dweights[t, j] = <dout[t], y[slots[t, j]]> (fp32, 0 for a
 * slot that is none). dweights NULL: not wanted, y is then not read.
 * mx_combine_backward_whole also writes the rows of dy that no slot names: zeros, their gradient.
 * workspace: device memory of 4 * R bytes, 4-byte aligned.
 */
mx_status mx_combine(const void* y, const int32_t* slots, const float* weights, int64_t T, int k,
                     int64_t R, int64_t N, void* out, void* stream);

mx_status mx_combine_backward(const void* dout, const void* y, const int32_t* slots,
                              const float* weights, int64_t T, int k, int64_t R, int64_t N,
                              void* dy, float* dweights, void* stream);

mx_status mx_combine_backward_whole(const void* dout, const void* y, const int32_t* slots,
                                    const float* weights, int64_t T, int k, int64_t R, int64_t N,
                                    void* dy, float* dweights, void* workspace, void* stream);

/* ------------------------------------------------------------------------------------------
 * Between the products of an 8-bit training step: layer norm and activation whose output is an
 * operand of the next product, activation checkpoints in 8 bits, and what the backward pass makes of
 * them. A checkpoint is E4M3 codes [M, K] with scales [ceil(K / 128), M] as mx_quantize_b128_rows
 * writes them; it stands for the values code * scale, one fp32 product each (a block with a NaN or an
 * infinity: NaN). The conventions at the top of this file hold; alignment is stated per call; no output
 * may overlap an input or another output. These have no counterpart on the pages.
 * ------------------------------------------------------------------------------------------ */

/* a checkpoint, where a call takes one in place of bf16 or fp32 */
#define MX_TYPE_E4M3_B128 2

/*
 * Layer norm of the M rows of x [M, K] (x_type: MX_TYPE_BF16 or MX_TYPE_FP32):
 *   mean = sum_i x_i / K (0 when center == 0: the root-mean-square form),
 *   rstd = 1 / sqrt(sum_i (x_i - mean)^2 / K + eps),  y_i = (x_i - mean) rstd weight_i + bias_i.
 * In fp32, the variance from the differences to the mean; y rounded once. weight, bias: [K] of w_type,
 * NULL for ones and zeros (w_type is then not used, but must be valid). mean, rstd: fp32 [M] or NULL,
 * what mx_layer_norm_backward takes (zeros when K == 0). K <= 16384.
 *
 * mx_layer_norm: y [M, K] of y_type. Alignment: that of the elements; all four on 32 bytes with
 *   K % 8 == 0 take wide loads.
 * mx_layer_norm_b128: y as the operand that mx_quantize_b128_rows makes of the unrounded y: codes
 *   [M, K], scales [ceil(K / 128), M]. x_codes, x_scales: unless NULL, a checkpoint of x. K % 32 == 0;
 *   x, codes, weight and bias 32-byte aligned.
 */
mx_status mx_layer_norm(const void* x, int x_type, const void* weight, const void* bias, int w_type,
                        int64_t M, int64_t K, float eps, int center, void* y, int y_type, float* mean,
                        float* rstd, void* stream);

mx_status mx_layer_norm_b128(const void* x, int x_type, const void* weight, const void* bias, int w_type,
                             int64_t M, int64_t K, float eps, int center, void* codes, float* scales,
                             void* x_codes, float* x_scales, float* mean, float* rstd, void* stream);

/*
 * Gradients of mx_layer_norm. dy [M, K] of dy_type; x as the forward call read it (bf16 or fp32), or a
 * checkpoint of it (MX_TYPE_E4M3_B128 with x_scales, K % 32 == 0); mean, rstd: as the forward call wrote
 * them (mean NULL: not centred). With xhat_i = (x_i - mean) rstd and g_i = dy_i weight_i:
 *   dx_i = rstd (g_i - sum g / K - xhat_i sum(g xhat) / K), the second term only when centred,
 *   dweight_i = sum over the rows of dy_i xhat_i,  dbias_i = sum over the rows of dy_i,
 * dx of dx_type, dweight and dbias fp32 [K] or NULL (not wanted; zeros when M == 0). A checkpoint's value
 * may be rounded with what is done to it (code * (scale rstd) - mean rstd), not on its own first; mean rstd
 * must then be finite in fp32. Sums in fp32, in an order that the sizes, types, alignment and device alone
 * decide. workspace: device memory of
 * mx_layer_norm_backward_workspace() bytes, 4-byte aligned (NULL will do without dweight and dbias); two
 * calls that may run at the same time need one each. Alignment: that of the elements; dy, x and dx on 16
 * bytes and weight on 32 with K % 8 == 0 take wide loads.
 */
mx_status mx_layer_norm_backward_workspace(int64_t M, int64_t K, int64_t* bytes);

mx_status mx_layer_norm_backward(const void* dy, int dy_type, const void* x, int x_type,
                                 const float* x_scales, const float* mean, const float* rstd,
                                 const void* weight, int w_type, int64_t M, int64_t K, void* dx,
                                 int dx_type, float* dweight, float* dbias, void* workspace,
                                 void* stream);

/* activations: x s(x) with s the logistic function; x Phi(x); x s(2 z), z = sqrt(2 / pi) (x + 0.044715 x^3) */
#define MX_ACT_SILU 0
#define MX_ACT_GELU 1
#define MX_ACT_GELU_TANH 2

/*
 * Activation of R rows into the operand of the next product. gated != 0: u is [R, 2 H] = [gate | up],
 * h = f(gate) * up; else u is [R, H], h = f(u). u: bf16; h in fp32, then codes [R, H] and scales
 * [ceil(H / 128), R] as mx_quantize_b128_rows makes them of the unrounded h. u_codes, u_scales: unless
 * NULL, a checkpoint of u (what mx_quantize_b128_rows makes of it). H % 32 == 0, H <= 2^27; gated with a
 * checkpoint H % 128 == 0. u and codes 32-byte aligned.
 *
 * Backward: dh bf16 [R, H]; u bf16 or a checkpoint (u_type MX_TYPE_E4M3_B128 with u_scales). du, bf16
 * like u, is dh up f'(gate) | dh f(gate), or dh f'(u); du_codes, du_scales: the operand that
 * mx_quantize_b128_rows makes of the unrounded du, for the product that goes on backward. Either may be
 * NULL, not both. H % 32 == 0; gated with a checkpoint or an operand H % 128 == 0. All but the scales
 * 32-byte aligned.
 */
mx_status mx_activation_b128(const void* u, int64_t R, int64_t H, int kind, int gated, void* codes,
                             float* scales, void* u_codes, float* u_scales, void* stream);

mx_status mx_activation_backward(const void* dh, const void* u, int u_type, const float* u_scales,
                                 int64_t R, int64_t H, int kind, int gated, void* du, void* du_codes,
                                 float* du_scales, void* stream);

/*
 * mx_quantize_b128_cols of the values of a checkpoint (codes [M, K], scales [ceil(K / 128), M]): the
 * operand of the weights' gradient, without bf16 rows. index, R, row_offsets, E and the results as
 * there. codes and out_codes 32-byte aligned.
 */
mx_status mx_requantize_b128_cols(const void* codes, const float* scales, int64_t M, int64_t K,
                                  const int32_t* index, int64_t R, const int64_t* row_offsets, int E,
                                  void* out_codes, float* out_scales, void* stream);

/*
 * Values of a checkpoint (rows `index` of it, as in mx_quantize_b128_rows): y [R, K] of y_type
 * (MX_TYPE_BF16, rounded once, or MX_TYPE_FP32). codes and y 32-byte aligned, K % 32 == 0.
 */
mx_status mx_dequantize_b128_rows(const void* codes, const float* scales, int64_t M, int64_t K,
                                  const int32_t* index, int64_t R, void* y, int y_type, void* stream);

/*
 * Diagnostics: the rotated values y = x_chunk * H exactly as mx_rotate_quantize computes them
 * before quantization with the same rot_kind (same device code), written as fp32 [M, K] to
 * y_f32 (device, 32-byte aligned).
 */
mx_status mx_rotate_debug(const void* x, int64_t M, int64_t K, const void* H, int g, int rot_kind,
                          float* y_f32, void* stream);

/*
 * Device-side error word of the current device: bit 0 set if a kernel gave up waiting for
 * its tensor-core work to complete (a bounded wait ran out; its outputs are then invalid).
 * Synchronizes the device, returns the word in *flags and clears it.
 */
mx_status mx_device_errors(int* flags);

/*
 * Failure-detection self-test (no counterpart on the pages): launches one thread that waits on
 * an mbarrier nothing ever arrives at, with the same bounded-wait routine the tensor-core
 * kernel uses for every wait, given up after limit_ns nanoseconds (1 .. 100,000,000). The wait
 * gives up, sets bit 0 of the device error word (read it with mx_device_errors) and the kernel
 * returns; the context stays usable. Errors: MX_ERR_SHAPE (limit out of range), MX_ERR_CUDA.
 */
mx_status mx_selftest_bounded_wait(int64_t limit_ns, void* stream);

/*
 * Give-up self-test of the tensor-core rotation kernel (no counterpart on the pages): the call
 * mx_rotate_quantize(x, M, K, H, g, MX_FMT_E2M1, 32, MX_SCALES_SWIZZLED, MX_ROUND_RNE, codes,
 * scales, stream) makes, with every mbarrier wait of the kernel limited to limit_ns
 * nanoseconds (1 .. 100,000,000) instead of 2 s, so that waits run out while the pipeline is
 * busy. A role whose wait ran out stops issuing work, and the kernel still waits for its loads,
 * MMAs and stores in flight before it frees tensor memory and exits: the call ends, the device
 * error word reports the give-up (mx_device_errors) and the context stays usable. codes and
 * scales then hold unspecified bytes. Shapes as mx_rotate_quantize, except that calls the
 * few-row kernel would take (M <= 16 and M * g <= 512) and empty calls are MX_ERR_SHAPE.
 * Errors: MX_ERR_SHAPE (limit or shape), MX_ERR_NULL, MX_ERR_ALIGN, MX_ERR_UNSUPPORTED (g),
 * MX_ERR_CUDA.
 */
mx_status mx_selftest_rotate_give_up(const void* x, int64_t M, int64_t K, const void* H, int g,
                                     void* codes, void* scales, int64_t limit_ns, void* stream);

/*
 * Give-up self-test of the GEMM kernel (no counterpart on the pages): the call
 * mx_gemm(a_codes, a_scales, b_codes, b_scales, M, N, K, fmt, 32, layout, 1.0f, c, stream)
 * makes, with every pipeline wait of the kernel limited to limit_ns nanoseconds
 * (1 .. 100,000,000) instead of 2 s. A role whose wait ran out stops issuing work; the loads in
 * flight and the MMAs issued are still waited for (2 s) before the kernel frees its tensor
 * memory and exits: the call ends, the device error word reports the give-up
 * (mx_device_errors) and the context stays usable. c then holds unspecified bytes. Shapes and
 * errors as mx_gemm, except that M == 0 or N == 0 is MX_ERR_SHAPE.
 */
mx_status mx_selftest_gemm_give_up(const void* a_codes, const void* a_scales, const void* b_codes,
                                   const void* b_scales, int64_t M, int64_t N, int64_t K, int fmt,
                                   int layout, void* c, int64_t limit_ns, void* stream);

/*
 * The same self-test of the product of operands with a scale per block of 128: mx_gemm_b128 with
 * a bf16 C and every pipeline wait limited to limit_ns; and mx_gemm_b128_grouped likewise. Drains are
 * limited to 2 s. Few tokens run the swapped shape, M = N = 2048 CTA pairs (both forms of B's scales);
 * by expert, experts of more than 128 rows pairs, the others single CTAs.
 */
mx_status mx_selftest_gemm_b128_give_up(const void* a_codes, const float* a_scales,
                                        const void* b_codes, const float* b_scales, int64_t M,
                                        int64_t N, int64_t K, int b_form, void* c, int64_t limit_ns,
                                        void* stream);

mx_status mx_selftest_gemm_b128_grouped_give_up(const void* a_codes, const float* a_scales,
                                                const void* b_codes, const float* b_scales,
                                                const int64_t* row_offsets, int E, int64_t M_total,
                                                int64_t N, int64_t K, void* c, int64_t limit_ns,
                                                void* stream);

/*
 * The same self-test of the layer norm's kernels, whose waits are for rows on their way to shared memory:
 * mx_layer_norm of bf16 rows into bf16, and mx_layer_norm_backward from bf16 dy and bf16 or checkpointed
 * rows (x_type) into a bf16 dx, every wait limited to limit_ns; what a wait that ran out had asked for is
 * waited for once more, 2 s at most, before the kernel ends. Rows that allow no wide loads run without such
 * waits, and as few rows of mx_layer_norm as are resident at once: 8 a multiprocessor up to 1024 columns, 2
 * of 8192, 1 of 16384. y and dx then hold unspecified values. Errors as those calls, and MX_ERR_SHAPE for a
 * limit out of range, M == 0 and K == 0.
 */
mx_status mx_selftest_layer_norm_give_up(const void* x, int64_t M, int64_t K, void* y, int64_t limit_ns,
                                         void* stream);

mx_status mx_selftest_layer_norm_backward_give_up(const void* dy, const void* x, int x_type,
                                                  const float* x_scales, const float* mean,
                                                  const float* rstd, int64_t M, int64_t K, void* dx,
                                                  int64_t limit_ns, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_H */
