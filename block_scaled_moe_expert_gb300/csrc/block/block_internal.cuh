// Internal declarations of the operators around the experts forward
// (include/moe_block.h): what the C entry points share with the kernels.
#pragma once
#include "../device_check.h"
#include "../moe_internal.cuh"
#include "moe_block.h"
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

}  // namespace bsmoe
