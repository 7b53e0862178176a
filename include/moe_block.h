/*
 * Operators around the experts forward of moe_experts.h: C ABI.
 *
 *   - tokens sorted by expert and back, with the routing weights applied on
 *     either way, and the gradients (for training the experts, and for
 *     grouped products other than the quantized ones of moe_experts.h);
 *   - the norms before and after a block, fused with the block's gate, the
 *     residual scale and the next block's norm, and their gradients;
 *   - matrix-vector products with 4-bit weights and group scales (dense
 *     layers, a shared expert, an output head at decode).
 *
 * The conventions of moe_experts.h hold: device pointers of the calling
 * thread's current device, an asynchronous call on `stream`, nothing
 * allocated, a non-MOE_OK status means that nothing was enqueued, calls from
 * several host threads and for several devices do not disturb each other, element
 * types named by a moe_dtype argument and otherwise not checked. Row strides
 * (ld_*) count elements, from 0 (the same row for every token, inputs only)
 * up; the elements of a row are contiguous. Any alignment of at least the
 * element size is taken; 16-byte aligned pointers and row strides run the
 * vectorized kernels. Outputs are contiguous and must not overlap inputs.
 */
#ifndef BSMOE_MOE_BLOCK_H_
#define BSMOE_MOE_BLOCK_H_

#include "moe_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_BF16 = 0, MOE_FP16 = 1, MOE_FP32 = 2 } moe_dtype;

/* ---------------------------------------------------- tokens by expert ---
 * Slot s = t * K + k holds the pair of token t and its k-th expert. Slots of
 * one expert form a group, in ascending s; groups stand in expert order, each
 * starting at a multiple of row_align. A slot with id -1 is skipped and has
 * no row; an id outside [-1, E) is treated as skipped and raises
 * MOE_DEV_BAD_EXPERT_ID in the plan's status word.
 *
 * Shapes: 1 <= E <= 512, 1 <= K <= 32, 1 <= row_align <= 256,
 * 0 <= T * K <= 2^26, 1 <= H <= 65536.
 */

/*
 * Byte offsets inside a sort plan (all int32):
 *   status u32 (moe_get_device_status works on the plan's start);
 *   counts [E]; offsets [E + 1] (first row of each group; offsets[E] = rows
 *   in use, padding included); inv [T * K] (slot -> row, -1 if skipped);
 *   row_slot [M] (row -> slot, -1 for padding rows and rows past offsets[E]).
 * M = row_capacity = floor((S + min(E, S) * (row_align - 1)) / row_align) *
 * row_align with S = T * K: the most rows that any routing of T tokens takes.
 */
typedef struct {
  size_t total_bytes;
  size_t status, counts, offsets, inv, row_slot;
  int32_t row_capacity;
} moe_sort_layout;

/* MOE_ERR_INVALID_ARG for a null layout, MOE_ERR_UNSUPPORTED_SHAPE. */
moe_status moe_query_sort_layout(int T, int E, int K, int row_align, moe_sort_layout* layout);

/*
 * topk_idx i32 [T, K] contiguous -> plan (256-byte aligned device memory of
 * total_bytes). T = 0 writes an empty plan.
 */
moe_status moe_sort_tokens(const int32_t* topk_idx, int T, int E, int K, int row_align, void* plan,
                           size_t plan_bytes, void* stream);

/*
 * rows[inv[t, k]] = w[t, k] * hidden[t], one rounding to dtype; every other
 * of the M rows is zero. topk_w f32 [T, K] or null (rows are copies).
 * hidden dtype [T, H] (row stride ld_hidden), rows dtype [M, H].
 */
moe_status moe_permute_tokens(int dtype, const void* hidden, int64_t ld_hidden, const float* topk_w,
                              const void* plan, size_t plan_bytes, int T, int H, int E, int K, int row_align,
                              void* rows, void* stream);

/*
 * Gradient of moe_permute_tokens: d_hidden[t] = sum over k (ascending, fp32)
 * of w[t, k] * d_rows[inv[t, k]], and with topk_w
 * d_topk_w[t, k] = <hidden[t], d_rows[inv[t, k]]> (0 for skipped slots).
 * Without topk_w, hidden and d_topk_w are not used (null).
 */
moe_status moe_permute_tokens_backward(int dtype, const void* d_rows, int64_t ld_rows, const void* hidden,
                                       int64_t ld_hidden, const float* topk_w, const void* plan, size_t plan_bytes,
                                       int T, int H, int E, int K, int row_align, void* d_hidden, float* d_topk_w,
                                       void* stream);

/*
 * out[t] = sum over k (ascending, fp32) of w[t, k] * rows[inv[t, k]] (w = 1
 * without topk_w), one rounding to dtype; a token without rows gives zeros.
 * Rows that belong to no slot are never read.
 */
moe_status moe_unpermute_tokens(int dtype, const void* rows, int64_t ld_rows, const float* topk_w,
                                const void* plan, size_t plan_bytes, int T, int H, int E, int K, int row_align,
                                void* out, void* stream);

/*
 * Gradient of moe_unpermute_tokens: d_rows[inv[t, k]] = w[t, k] * d_out[t],
 * every other row zero, and with topk_w
 * d_topk_w[t, k] = <d_out[t], rows[inv[t, k]]> (0 for skipped slots).
 * Without topk_w, rows and d_topk_w are not used (null).
 */
moe_status moe_unpermute_tokens_backward(int dtype, const void* d_out, int64_t ld_out, const void* rows,
                                         int64_t ld_rows, const float* topk_w, const void* plan, size_t plan_bytes,
                                         int T, int H, int E, int K, int row_align, void* d_rows, float* d_topk_w,
                                         void* stream);

/* -------------------------------------------- norms around a block -------
 * N(v; w) = v * rsqrt(mean(v^2) + eps) * (w + w_offset), w = 1 - w_offset
 * where no weight is given. All arithmetic in fp32, one rounding per output.
 * 1 <= H <= 16384, T >= 0. x, h, gradients, gate: dtype. Norm weights: dtype
 * or f32 (weight_f32 = 1); their gradients have the weights' type.
 */
typedef enum {
  MOE_GATE_NONE = 0,
  MOE_GATE_CHANNEL = 1, /* gate [H] */
  MOE_GATE_TOKEN = 2,   /* gate [T] */
  MOE_GATE_ELEMENT = 3  /* gate [T, H], row stride ld_gate */
} moe_gate_kind;
typedef enum { MOE_GATE_LINEAR = 0, MOE_GATE_SIGMOID = 1, MOE_GATE_TANH = 2 } moe_gate_act;

/* y = N(x; weight). weight may be null. */
moe_status moe_norm_before(int dtype, const void* x, int64_t ld_x, const void* weight, int weight_f32,
                           float w_offset, float eps, int T, int H, void* y, void* stream);

/* Bytes of workspace of the two gradients below; 0 for an unsupported H. */
size_t moe_norm_backward_workspace_bytes(int H);

/*
 * dx = gradient of N at x for dy, plus dr where it is given (the gradient
 * that reaches x another way, the residual's); d_weight = sum over tokens of
 * dy * x * rsqrt(...) (null without weight). Sums over tokens have a fixed
 * order: the same call gives the same bits.
 */
moe_status moe_norm_before_backward(int dtype, const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                                    const void* dr, int64_t ld_dr, const void* weight, int weight_f32,
                                    float w_offset, float eps, int T, int H, void* dx, void* d_weight,
                                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * r = beta * x + alpha * g * z with z = N(h; weight) (norm = 1) or h
 * (norm = 0) and g = act(gate), and where y is not null
 * y = N(r; next_weight) of the unrounded r (next_eps; the same w_offset).
 */
moe_status moe_norm_after(int dtype, const void* x, int64_t ld_x, const void* h, int64_t ld_h, int norm,
                          const void* weight, const void* next_weight, int weight_f32, float w_offset,
                          int gate_kind, int gate_act, const void* gate, int64_t ld_gate, float alpha, float beta,
                          float eps, float next_eps, int T, int H, void* r, void* y, void* stream);

/*
 * Gradient of moe_norm_after. dr: gradient of r; dy (null without the next
 * norm): gradient of y, with the forward's r. With G = dr + (gradient of N at
 * r for dy):
 *   dx = beta * G (dx may be null), dh, d_weight (null without weight),
 *   d_gate of the gate's shape and type, contiguous (null without gate),
 *   d_next_weight (null without next_weight).
 */
moe_status moe_norm_after_backward(int dtype, const void* dr, int64_t ld_dr, const void* dy, int64_t ld_dy,
                                   const void* h, int64_t ld_h, const void* r, int64_t ld_r, int norm,
                                   const void* weight, const void* next_weight, int weight_f32, float w_offset,
                                   int gate_kind, int gate_act, const void* gate, int64_t ld_gate, float alpha,
                                   float beta, float eps, float next_eps, int T, int H, void* dx, void* dh,
                                   void* d_weight, void* d_gate, void* d_next_weight, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* ------------------------------------- products with 4-bit weights -------
 * y[t, n] = sum over k of x[t, k] * W[n, k], sums in fp32, one rounding. Every
 * finite x counts in full, whatever else its row holds.
 *   MOE_Q_FP4:  the weights of MOE_W_FP4: codes u8 [N, K / 2] (e2m1, low
 *               nibble = even k), scale u8 [N, K / 32] (UE8M0; 255 = NaN);
 *   MOE_Q_INT4: codes u8 [N, K / 2] (0..15, low nibble = even k),
 *               W = (code - zero) * scale, scale bf16 or fp16
 *               [N, ceil(K / group)], zero u8 (0..15) of the same shape, or
 *               null for 8; group 32, 64 or 128.
 * K a multiple of 32, 32 <= K <= 32768; 1 <= N <= 2^20.
 * swiglu: rows [0, N/2) are gate, [N/2, N) up (N even), and
 *   y[t, n] = silu(min(gate, L)) * clamp(up, -L, L), n < N / 2
 *   (unclamped for a limit that is NaN or not positive).
 */
typedef enum { MOE_Q_FP4 = 0, MOE_Q_INT4 = 1 } moe_qfmt;

/* Bytes of the kernel-layout weights; 0 for an unsupported shape. */
size_t moe_matvec_prepared_bytes(int qfmt, int N, int K, int group, int swiglu);

/* One-shot layout of checkpoint weights for moe_matvec; prepared is 256-byte
 * aligned. scale_dtype: MOE_BF16 or MOE_FP16 (MOE_Q_INT4 only). */
moe_status moe_matvec_prepare(int qfmt, int N, int K, int group, int swiglu, const void* codes, const void* scale,
                              int scale_dtype, const void* zero, void* prepared, size_t prepared_bytes,
                              void* stream);

/* x bf16 or fp16 [T, K] (row stride ld_x) -> y of the same type [T, N], or
 * [T, N / 2] with swiglu. Meant for few tokens: the weights are read once per
 * 16 tokens (fewer where x would not fit into shared memory). The kernel starts
 * reading `prepared` while the kernel in front of it on the stream ends. That is
 * safe behind moe_matvec_prepare and any copy; a kernel of the caller's that writes
 * prepared weights itself must not be the last operation in front of the call (an
 * event, a memset or a kernel launched without programmatic serialization in
 * between is enough). */
moe_status moe_matvec(int qfmt, int N, int K, int group, int swiglu, float swiglu_limit, int scale_dtype,
                      const void* prepared, int dtype, const void* x, int64_t ld_x, int T, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSMOE_MOE_BLOCK_H_ */
