// Internal declarations of the operators around the experts forward
// (include/moe_block.h): what the C entry points share with the kernels.
#pragma once
#include "../device_check.h"
#include "../moe_internal.cuh"
#include "moe_route_fp4.h"
#include "vec_io.cuh"

namespace bsmoe {

constexpr int kMaxRowAlign = 256;
constexpr int kMaxRowWidth = 65536;   // permute / unpermute
constexpr int kMaxNormWidth = 16384;  // norms

// Dynamic shared memory that a launch of `kernel` may ask for. The limit belongs to
// the kernel, not to the launch: every call sets the same one, so that another
// host thread's call cannot lower it between the two.
constexpr int kMaxDynSmem = 226 * 1024;  // beside at most 1 KB of static shared memory
template <typename K>
cudaError_t allow_smem(K* kernel, size_t smem, int most = kMaxDynSmem) {
  if (smem > static_cast<size_t>(most)) return cudaErrorInvalidValue;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
}

// The sort plan as the kernels see it.
struct SortPlan {
  uint32_t* status;
  int32_t *counts, *offsets, *inv, *row_slot;
  int T, E, K, S, M, align;
};

bool sort_layout(int T, int E, int K, int row_align, moe_sort_layout* out);
cudaError_t launch_sort(const int32_t* topk_idx, const SortPlan& p, cudaStream_t st);

// rows[inv[t, k]] = w[t, k] * x[t] (w null: copies), zeros in the other rows;
// with dots, dots[t, k] = <x[t], other[inv[t, k]]>.
struct PlaceArgs {
  const void* x;
  int64_t ld_x;
  const void* other;
  int64_t ld_other;
  const float* w;
  void* rows;
  float* dots;
  int H;
  SortPlan p;
};
cudaError_t launch_place(int dtype, const PlaceArgs& a, cudaStream_t st);

// out[t] = sum over k of w[t, k] * rows[inv[t, k]] (w null: 1); with dots,
// dots[t, k] = <x[t], rows[inv[t, k]]>.
struct GatherArgs {
  const void* rows;
  int64_t ld_rows;
  const void* x;
  int64_t ld_x;
  const float* w;
  void* out;
  float* dots;
  int H;
  SortPlan p;
};
cudaError_t launch_gather(int dtype, const GatherArgs& a, cudaStream_t st);

// The norm of v with optional weight, and what norm_after adds to it.
struct NormArgs {
  const void *x, *h, *weight, *next_weight, *gate;
  int64_t ld_x, ld_h, ld_gate;
  int T, H, norm, weight_f32, gate_kind, gate_act, next;
  float w_offset, alpha, beta, eps, next_eps;
  void *r, *y;  // norm_after: r always, y with next; norm_before: y only
};
cudaError_t launch_norm(int dtype, const NormArgs& a, int num_sms, cudaStream_t st);

struct NormBackwardArgs {
  NormArgs f;  // x unused; r is the forward's result
  const void *dr, *dy;
  int64_t ld_dr, ld_dy, ld_r;
  void *dx, *dh, *d_weight, *d_gate, *d_next_weight;
  float* partials;  // [2][kNormParts][H]
};
constexpr int kNormParts = 304;  // column sums are taken over at most this many row sets
cudaError_t launch_norm_backward(int dtype, const NormBackwardArgs& a, int num_sms, cudaStream_t st);

// 4-bit products.
struct MatvecShape {
  int fmt, N, K, group, swiglu;
};
size_t matvec_prepared_bytes(const MatvecShape& s);  // 0: unsupported
cudaError_t launch_matvec_prepare(const MatvecShape& s, const void* codes, const void* scale, int scale_dtype,
                                  const void* zero, void* prepared, cudaStream_t st);
cudaError_t launch_matvec(const MatvecShape& s, float limit, int scale_dtype, const void* prepared, int dtype,
                          const void* x, int64_t ld_x, int T, void* y, int num_sms, cudaStream_t st);

// Routing: the choice of experts and its gradient.
struct RouteArgs {
  const void* logits;
  int64_t ld;
  const float* bias;  // null: none
  int T, E, K, G, top_groups, group_max, sigmoid, renorm;
  float scale;
  int32_t* idx;
  float *w, *mean;  // mean null: not asked for
  float* partials;  // [kRouteParts][E] with mean
};
constexpr int kRouteParts = 608;  // the mean's column sums are taken over at most this many blocks
cudaError_t launch_route_softmax(int dtype, const RouteArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_route_sigmoid(int dtype, const RouteArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_route_tokens(int dtype, const RouteArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_route_tokens_backward(int dtype, const RouteArgs& a, const float* dw, const float* dmean, void* dx,
                                         int num_sms, cudaStream_t st);

// The FP4 format: rows of C elements, C a multiple of 32; codes 8-byte aligned when written.
cudaError_t launch_quantize_fp4(int dtype, const void* x, int64_t ld, int R, int C, uint8_t* codes, uint8_t* scale,
                                int num_sms, cudaStream_t st);
cudaError_t launch_dequantize_fp4(int dtype, const uint8_t* codes, const uint8_t* scale, int64_t blocks, void* out,
                                  int num_sms, cudaStream_t st);

// Tensor map of rows of `row_bytes` bytes (a multiple of 16), boxes of 128 bytes x
// box_rows rows in the 128-byte swizzle; false if it cannot be made (api.cu).
bool byte_tmap(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_rows);
// That of scale words [blocks][KB][128], boxes of 2 K blocks x box_blocks.
bool scale_tmap(CUtensorMap* m, const void* base, uint64_t KB, uint64_t blocks, uint32_t box_blocks);
// That of rows of 16-bit elements to be stored, contiguous and 16-byte aligned, boxes of box_cols x
// box_rows with rows of 128 bytes in the 128-byte swizzle.
bool store_tmap(CUtensorMap* m, void* base, uint64_t cols, uint64_t rows, uint32_t box_cols, uint32_t box_rows);

// FP4 x FP4 products.
struct MatmulShape {
  int N, K, swiglu;
};
struct MatmulLayout {  // prepared weights: codes, then scale words
  int KB, NT;          // 128-K blocks, 256-row tiles
  size_t codes_bytes, total;  // total 0: unsupported
};
MatmulLayout matmul_layout(const MatmulShape& s);
struct MatmulWorkspace {  // status word, then the quantized activations
  size_t sf, codes, total;
};
MatmulWorkspace matmul_workspace(int T, int K);
cudaError_t launch_matmul_prepare(const MatmulShape& s, const void* codes, const void* scale, void* prepared,
                                  cudaStream_t st);
// Activations [T][K] to codes [T][Kp / 2] and scale words; clears the status word.
cudaError_t launch_quantize_act(int dtype, const void* x, int64_t ld, int T, int K, uint8_t* codes, uint32_t* sf,
                                uint32_t* status, cudaStream_t st);
cudaError_t launch_matmul_fp4(const MatmulShape& s, float limit, const void* prepared, int dtype, const void* x,
                              int64_t ld, int T, void* y, uint8_t* workspace, int num_sms, cudaStream_t st);

}  // namespace bsmoe
