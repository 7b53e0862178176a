/*
 * Routing and FP4 products around the experts forward of moe_experts.h: C ABI.
 *
 *   - the router's choice of experts with its weights (the topk_idx and topk_w
 *     of moe_experts_forward and moe_sort_tokens), and its gradient;
 *   - quantization to the FP4 format of the weights, and back;
 *   - products of many tokens with FP4 weights and FP4 activations.
 *
 * The conventions of moe_block.h hold.
 */
#ifndef BSMOE_MOE_ROUTE_FP4_H_
#define BSMOE_MOE_ROUTE_FP4_H_

#include "moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------- routing ------
 * Scores s[t, e]: softmax of a token's logits over the experts, or the sigmoid of
 * each. An expert is available to a token if its logit and, where one is given,
 * its bias are more than -inf and no NaN. The K best available experts, best first,
 * ties to the lowest index, go to topk_idx [T, K]; where fewer are available the
 * last slots get -1 and weight 0. Best: by s + bias where bias (f32 [E]) is given, as
 * the scores compare before any rounding (evaluated in 64 bits where fp32 does not
 * settle it), else by the logits. With num_groups > 1 the experts form groups of
 * E / num_groups neighbours, and the choice is among those of the top_groups groups
 * of the largest value: the sum of the group's two largest s + bias (MOE_GROUP_TOP2;
 * the largest alone where one expert is available) or the largest (MOE_GROUP_MAX);
 * ties to the lowest group. topk_w [T, K] = scale * s (without bias) of the chosen,
 * divided by their sum first with renormalize.
 * A NaN among a token's logits makes its weights NaN (the choice is that without the
 * experts of such logits). So does +inf under softmax, which then has no scores: where
 * scores decide (a bias, or groups by their two best) the choice is that without its
 * expert, where logits alone do it is the largest.
 * mean_scores f32 [E] (may be null): mean over the tokens of
 * s[t, e] / (sum over e of s[t, e]); a token without logits above -inf counts 0.
 *
 * Shapes: 1 <= E <= 512, 1 <= K <= 32, 0 <= T * K <= 2^26, num_groups <= 32
 * divides E, 1 <= top_groups <= num_groups, K <= top_groups * (E / num_groups).
 * logits: dtype [T, E], row stride ld_logits. Sums have a fixed order.
 */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;
typedef enum { MOE_GROUP_TOP2 = 0, MOE_GROUP_MAX = 1 } moe_group_score;

/* Bytes of workspace of moe_route_tokens with mean_scores; 0 for an unsupported E. */
size_t moe_route_workspace_bytes(int E);

/* workspace (256-byte aligned) is needed with mean_scores only. */
moe_status moe_route_tokens(int dtype, const void* logits, int64_t ld_logits, const float* bias, int T, int E, int K,
                            int score, int num_groups, int top_groups, int group_score, int renormalize, float scale,
                            int32_t* topk_idx, float* topk_w, float* mean_scores, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * Gradient of moe_route_tokens for the choice topk_idx: d_logits dtype [T, E],
 * contiguous, from d_topk_w f32 [T, K] and d_mean_scores f32 [E] (null: none).
 * Slots with an id outside [0, E) count for nothing. The choice itself and the
 * bias have no gradient.
 */
moe_status moe_route_tokens_backward(int dtype, const float* d_topk_w, const float* d_mean_scores, const void* logits,
                                     int64_t ld_logits, const int32_t* topk_idx, int T, int E, int K, int score,
                                     int renormalize, float scale, void* d_logits, void* stream);

/* ------------------------------------------------- the FP4 format --------
 * Rows of C elements (a multiple of 32, 32 <= C <= 2^20) as e2m1 codes u8 [R, C / 2]
 * (low nibble = even index) and UE8M0 scales u8 [R, C / 32], the layout of
 * MOE_W_FP4 weights and of MOE_Q_FP4. Per block of 32: n = min{n >= -127: amax <=
 * 6 * 2^n} (0 for a block of zeros), scale byte n + 127, code = x * 2^-n rounded to
 * the nearest e2m1 value, ties to even. A block that holds a NaN or an infinity
 * gets scale byte 255 and zero codes: all of it reads as NaN.
 */
/* x dtype [R, C] (row stride ld_x); codes 16-byte aligned, contiguous like scale. */
moe_status moe_quantize_fp4(int dtype, const void* x, int64_t ld_x, int R, int C, void* codes, void* scale,
                            void* stream);
/* out dtype [R, C] = code * 2^(scale - 127), rounded to dtype; contiguous. */
moe_status moe_dequantize_fp4(int dtype, const void* codes, const void* scale, int R, int C, void* out, void* stream);

/* --------------------------- FP4 x FP4 products of many tokens -----------
 * y[t, n] = sum over k of dq(x)[t, k] * dq(W)[n, k] on the tensor cores, with x
 * quantized as moe_quantize_fp4 does, fp32 sums and one rounding. W: codes u8
 * [N, K / 2] and scale u8 [N, K / 32] (255 = NaN). K a multiple of 32, 32 <= K <= 32768;
 * 1 <= N <= 2^20; 0 <= T <= 2^20. swiglu as in moe_matvec.
 */
/* Bytes of the kernel-layout weights; 0 for an unsupported shape. */
size_t moe_matmul_fp4_prepared_bytes(int N, int K, int swiglu);

/* One-shot layout of checkpoint weights; prepared is 256-byte aligned. */
moe_status moe_matmul_fp4_prepare(int N, int K, int swiglu, const void* codes, const void* scale, void* prepared,
                                  size_t prepared_bytes, void* stream);

/* Bytes of workspace for up to T_max tokens; 0 for an unsupported T_max or K. */
size_t moe_matmul_fp4_workspace_bytes(int T_max, int K);

/*
 * x bf16 or fp16 [T, K] (row stride ld_x) -> y of the same type [T, N], or
 * [T, N / 2] with swiglu. The workspace (256-byte aligned) starts with the status
 * word that moe_get_device_status reads (MOE_DEV_TIMEOUT: y is invalid) and must
 * not be used by another call until this one has finished on `stream`; a call without
 * tokens touches nothing. Above 8 tokens it is two launches, the quantization and the
 * product. A token's row has the same bits in any batch of up to 128 tokens that is on
 * the same side of 8, and in any larger batch.
 */
moe_status moe_matmul_fp4(int N, int K, int swiglu, float swiglu_limit, const void* prepared, int dtype, const void* x,
                          int64_t ld_x, int T, void* workspace, size_t workspace_bytes, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSMOE_MOE_ROUTE_FP4_H_ */
