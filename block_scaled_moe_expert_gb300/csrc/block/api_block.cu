// C entry points of the operators around the experts forward
// (include/moe_block.h): argument checks and launches on the caller's stream.
// No allocation, no host synchronization. Checks come in the order of the
// experts forward's: arguments and shapes, null pointers, alignment, sizes,
// device, memory of every pointer.
#include "block_internal.cuh"

using namespace bsmoe;

namespace {

struct Ptr {
  const void* p;
  size_t align;
};

moe_status check_ptrs(std::initializer_list<Ptr> ptrs, DevInfo* d) {
  for (const Ptr& p : ptrs)
    if (p.p != nullptr && reinterpret_cast<uintptr_t>(p.p) % p.align) return MOE_ERR_ALIGNMENT;
  moe_status s = current_device(d);
  if (s != MOE_OK) return s;
  for (const Ptr& p : ptrs)
    if (p.p != nullptr && (s = check_ptr(p.p, d->id)) != MOE_OK) return s;
  return MOE_OK;
}

bool dtype_ok(int dtype) { return dtype == MOE_BF16 || dtype == MOE_FP16 || dtype == MOE_FP32; }
size_t esize(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }
moe_status launched(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

SortPlan plan_view(const moe_sort_layout& L, const void* plan, int T, int E, int K, int align) {
  uint8_t* b = static_cast<uint8_t*>(const_cast<void*>(plan));
  SortPlan p;
  p.status = reinterpret_cast<uint32_t*>(b + L.status);
  p.counts = reinterpret_cast<int32_t*>(b + L.counts);
  p.offsets = reinterpret_cast<int32_t*>(b + L.offsets);
  p.inv = reinterpret_cast<int32_t*>(b + L.inv);
  p.row_slot = reinterpret_cast<int32_t*>(b + L.row_slot);
  p.T = T;
  p.E = E;
  p.K = K;
  p.S = T * K;
  p.M = L.row_capacity;
  p.align = align;
  return p;
}

// The checks that the four row movements share.
moe_status rows_call(int dtype, const void* in, int64_t ld_in, const void* other, int64_t ld_other,
                     const float* topk_w, float* dots, bool with_dots, const void* plan, size_t plan_bytes, int T,
                     int H, int E, int K, int row_align, const void* out, SortPlan* p) {
  moe_sort_layout L;
  if (!dtype_ok(dtype) || ld_in < 0 || ld_other < 0) return MOE_ERR_INVALID_ARG;
  if (!sort_layout(T, E, K, row_align, &L) || H < 1 || H > kMaxRowWidth) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (in == nullptr || plan == nullptr || out == nullptr) return MOE_ERR_INVALID_ARG;
  if (with_dots && topk_w != nullptr && (other == nullptr || dots == nullptr)) return MOE_ERR_INVALID_ARG;
  if (plan_bytes < L.total_bytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
  *p = plan_view(L, plan, T, E, K, row_align);
  DevInfo d;
  const size_t es = esize(dtype);
  return check_ptrs({{in, es}, {other, es}, {topk_w, 4}, {dots, 4}, {plan, 256}, {out, es}}, &d);
}

// A gate with one value for each token has none for no tokens.
bool gate_ok(int kind, int act, const void* gate, int T) {
  if (kind < MOE_GATE_NONE || kind > MOE_GATE_ELEMENT || act < MOE_GATE_LINEAR || act > MOE_GATE_TANH) return false;
  return (T == 0 && kind != MOE_GATE_CHANNEL) || (kind == MOE_GATE_NONE) == (gate == nullptr);
}

bool norm_shape_ok(int T, int H) { return T >= 0 && H >= 1 && H <= kMaxNormWidth; }

}  // namespace

extern "C" {

moe_status moe_query_sort_layout(int T, int E, int K, int row_align, moe_sort_layout* layout) {
  if (layout == nullptr) return MOE_ERR_INVALID_ARG;
  return sort_layout(T, E, K, row_align, layout) ? MOE_OK : MOE_ERR_UNSUPPORTED_SHAPE;
}

moe_status moe_sort_tokens(const int32_t* topk_idx, int T, int E, int K, int row_align, void* plan,
                           size_t plan_bytes, void* stream) {
  moe_sort_layout L;
  if (!sort_layout(T, E, K, row_align, &L)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (plan == nullptr || (topk_idx == nullptr && T > 0)) return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(plan) % 256 || reinterpret_cast<uintptr_t>(topk_idx) % 4) return MOE_ERR_ALIGNMENT;
  if (plan_bytes < L.total_bytes) return MOE_ERR_WORKSPACE_TOO_SMALL;
  DevInfo d;
  const moe_status s = check_ptrs({{plan, 256}, {T > 0 ? topk_idx : nullptr, 4}}, &d);
  if (s != MOE_OK) return s;
  return launched(launch_sort(topk_idx, plan_view(L, plan, T, E, K, row_align), static_cast<cudaStream_t>(stream)));
}

moe_status moe_permute_tokens(int dtype, const void* hidden, int64_t ld_hidden, const float* topk_w,
                              const void* plan, size_t plan_bytes, int T, int H, int E, int K, int row_align,
                              void* rows, void* stream) {
  PlaceArgs a = {hidden, ld_hidden, nullptr, 0, topk_w, rows, nullptr, H, {}};
  const moe_status s = rows_call(dtype, hidden, ld_hidden, nullptr, 0, topk_w, nullptr, false, plan, plan_bytes, T, H,
                                 E, K, row_align, rows, &a.p);
  if (s != MOE_OK || T == 0) return s;
  return launched(launch_place(dtype, a, static_cast<cudaStream_t>(stream)));
}

moe_status moe_unpermute_tokens_backward(int dtype, const void* d_out, int64_t ld_out, const void* rows,
                                         int64_t ld_rows, const float* topk_w, const void* plan, size_t plan_bytes,
                                         int T, int H, int E, int K, int row_align, void* d_rows, float* d_topk_w,
                                         void* stream) {
  const bool w = topk_w != nullptr;
  PlaceArgs a = {d_out, ld_out, w ? rows : nullptr, w ? ld_rows : 0, topk_w, d_rows, w ? d_topk_w : nullptr, H, {}};
  const moe_status s = rows_call(dtype, d_out, ld_out, a.other, a.ld_other, topk_w, a.dots, true, plan, plan_bytes, T,
                                 H, E, K, row_align, d_rows, &a.p);
  if (s != MOE_OK || T == 0) return s;
  return launched(launch_place(dtype, a, static_cast<cudaStream_t>(stream)));
}

moe_status moe_unpermute_tokens(int dtype, const void* rows, int64_t ld_rows, const float* topk_w,
                                const void* plan, size_t plan_bytes, int T, int H, int E, int K, int row_align,
                                void* out, void* stream) {
  GatherArgs a = {rows, ld_rows, nullptr, 0, topk_w, out, nullptr, H, {}};
  const moe_status s = rows_call(dtype, rows, ld_rows, nullptr, 0, topk_w, nullptr, false, plan, plan_bytes, T, H, E,
                                 K, row_align, out, &a.p);
  if (s != MOE_OK || T == 0) return s;
  return launched(launch_gather(dtype, a, static_cast<cudaStream_t>(stream)));
}

moe_status moe_permute_tokens_backward(int dtype, const void* d_rows, int64_t ld_rows, const void* hidden,
                                       int64_t ld_hidden, const float* topk_w, const void* plan, size_t plan_bytes,
                                       int T, int H, int E, int K, int row_align, void* d_hidden, float* d_topk_w,
                                       void* stream) {
  const bool w = topk_w != nullptr;
  GatherArgs a = {d_rows, ld_rows, w ? hidden : nullptr, w ? ld_hidden : 0, topk_w, d_hidden,
                  w ? d_topk_w : nullptr, H, {}};
  const moe_status s = rows_call(dtype, d_rows, ld_rows, a.x, a.ld_x, topk_w, a.dots, true, plan, plan_bytes, T, H, E,
                                 K, row_align, d_hidden, &a.p);
  if (s != MOE_OK || T == 0) return s;
  return launched(launch_gather(dtype, a, static_cast<cudaStream_t>(stream)));
}

moe_status moe_norm_before(int dtype, const void* x, int64_t ld_x, const void* weight, int weight_f32,
                           float w_offset, float eps, int T, int H, void* y, void* stream) {
  if (!dtype_ok(dtype) || ld_x < 0) return MOE_ERR_INVALID_ARG;
  if (!norm_shape_ok(T, H)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (x == nullptr || y == nullptr) return MOE_ERR_INVALID_ARG;
  DevInfo d;
  const size_t es = esize(dtype);
  const moe_status s = check_ptrs({{x, es}, {weight, weight_f32 ? 4 : es}, {y, es}}, &d);
  if (s != MOE_OK) return s;
  NormArgs a = {};
  a.x = x;
  a.ld_x = ld_x;
  a.next_weight = weight;
  a.weight_f32 = weight_f32;
  a.w_offset = w_offset;
  a.next_eps = eps;
  a.next = 1;
  a.T = T;
  a.H = H;
  a.y = y;
  return launched(launch_norm(dtype, a, d.sms, static_cast<cudaStream_t>(stream)));
}

size_t moe_norm_backward_workspace_bytes(int H) {
  return norm_shape_ok(0, H) ? sizeof(float) * 2 * kNormParts * H : 0;
}

moe_status moe_norm_before_backward(int dtype, const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                                    const void* dr, int64_t ld_dr, const void* weight, int weight_f32,
                                    float w_offset, float eps, int T, int H, void* dx, void* d_weight,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || ld_dy < 0 || ld_x < 0 || ld_dr < 0) return MOE_ERR_INVALID_ARG;
  if (!norm_shape_ok(T, H)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((weight == nullptr) != (d_weight == nullptr)) return MOE_ERR_INVALID_ARG;
  if (T == 0 && weight == nullptr) return MOE_OK;
  if (T > 0 && (dy == nullptr || x == nullptr || dx == nullptr)) return MOE_ERR_INVALID_ARG;
  if (workspace == nullptr) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_norm_backward_workspace_bytes(H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  DevInfo d;
  const size_t es = esize(dtype), ws = weight_f32 ? 4 : es;
  const bool any = T > 0;
  const moe_status s = check_ptrs({{any ? dy : nullptr, es}, {any ? x : nullptr, es}, {any ? dr : nullptr, es},
                                   {weight, ws}, {any ? dx : nullptr, es}, {d_weight, ws}, {workspace, 256}}, &d);
  if (s != MOE_OK) return s;
  NormBackwardArgs b = {};
  b.f.r = const_cast<void*>(x);
  b.ld_r = ld_x;
  b.f.next_weight = weight;
  b.f.weight_f32 = weight_f32;
  b.f.w_offset = w_offset;
  b.f.next_eps = eps;
  b.f.next = 1;
  b.f.beta = 1.f;
  b.f.T = T;
  b.f.H = H;
  b.dr = dr;
  b.ld_dr = ld_dr;
  b.dy = dy;
  b.ld_dy = ld_dy;
  b.dx = dx;
  b.d_next_weight = d_weight;
  b.partials = static_cast<float*>(workspace);
  return launched(launch_norm_backward(dtype, b, d.sms, static_cast<cudaStream_t>(stream)));
}

moe_status moe_norm_after(int dtype, const void* x, int64_t ld_x, const void* h, int64_t ld_h, int norm,
                          const void* weight, const void* next_weight, int weight_f32, float w_offset,
                          int gate_kind, int gate_act, const void* gate, int64_t ld_gate, float alpha, float beta,
                          float eps, float next_eps, int T, int H, void* r, void* y, void* stream) {
  if (!dtype_ok(dtype) || ld_x < 0 || ld_h < 0 || ld_gate < 0) return MOE_ERR_INVALID_ARG;
  if (!norm_shape_ok(T, H)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (!gate_ok(gate_kind, gate_act, gate, T)) return MOE_ERR_INVALID_ARG;
  if (x == nullptr || h == nullptr || r == nullptr) return MOE_ERR_INVALID_ARG;
  if ((!norm && weight != nullptr) || (y == nullptr && next_weight != nullptr)) return MOE_ERR_INVALID_ARG;
  DevInfo d;
  const size_t es = esize(dtype), ws = weight_f32 ? 4 : es;
  const moe_status s = check_ptrs(
      {{x, es}, {h, es}, {weight, ws}, {next_weight, ws}, {gate, es}, {r, es}, {y, es}}, &d);
  if (s != MOE_OK) return s;
  NormArgs a = {x, h, weight, next_weight, gate, ld_x, ld_h, ld_gate, T, H, norm ? 1 : 0, weight_f32, gate_kind,
                gate_act, y != nullptr, w_offset, alpha, beta, eps, next_eps, r, y};
  return launched(launch_norm(dtype, a, d.sms, static_cast<cudaStream_t>(stream)));
}

moe_status moe_norm_after_backward(int dtype, const void* dr, int64_t ld_dr, const void* dy, int64_t ld_dy,
                                   const void* h, int64_t ld_h, const void* r, int64_t ld_r, int norm,
                                   const void* weight, const void* next_weight, int weight_f32, float w_offset,
                                   int gate_kind, int gate_act, const void* gate, int64_t ld_gate, float alpha,
                                   float beta, float eps, float next_eps, int T, int H, void* dx, void* dh,
                                   void* d_weight, void* d_gate, void* d_next_weight, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || ld_dr < 0 || ld_dy < 0 || ld_h < 0 || ld_r < 0 || ld_gate < 0) return MOE_ERR_INVALID_ARG;
  if (!norm_shape_ok(T, H)) return MOE_ERR_UNSUPPORTED_SHAPE;
  const bool any = T > 0;
  if (!gate_ok(gate_kind, gate_act, gate, T)) return MOE_ERR_INVALID_ARG;
  if (gate_kind != MOE_GATE_NONE && d_gate == nullptr && (any || gate_kind == MOE_GATE_CHANNEL))
    return MOE_ERR_INVALID_ARG;
  if (any && (dr == nullptr || h == nullptr || dh == nullptr || (dy != nullptr && r == nullptr)))
    return MOE_ERR_INVALID_ARG;
  if ((weight == nullptr) != (d_weight == nullptr) || (next_weight == nullptr) != (d_next_weight == nullptr) ||
      (!norm && weight != nullptr) || (any && dy == nullptr && next_weight != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (workspace == nullptr) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe_norm_backward_workspace_bytes(H)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (!any && d_weight == nullptr && d_next_weight == nullptr && gate_kind != MOE_GATE_CHANNEL) return MOE_OK;
  DevInfo d;
  const size_t es = esize(dtype), ws = weight_f32 ? 4 : es;
  auto row = [&](const void* p) { return Ptr{any ? p : nullptr, es}; };
  const bool column = gate_kind == MOE_GATE_CHANNEL;
  const moe_status s =
      check_ptrs({row(dr), row(dy), row(h), row(dy != nullptr ? r : nullptr), {weight, ws}, {next_weight, ws},
                  {any || column ? gate : nullptr, es}, row(dx), row(dh), {d_weight, ws},
                  {any || column ? d_gate : nullptr, es},
                  {d_next_weight, ws}, {workspace, 256}}, &d);
  if (s != MOE_OK) return s;
  NormBackwardArgs b = {};
  b.f = {nullptr, h, weight, next_weight, gate, 0, ld_h, ld_gate, T, H, norm ? 1 : 0, weight_f32, gate_kind, gate_act,
         dy != nullptr, w_offset, alpha, beta, eps, next_eps, const_cast<void*>(r), nullptr};
  b.dr = dr;
  b.ld_dr = ld_dr;
  b.dy = dy;
  b.ld_dy = ld_dy;
  b.ld_r = ld_r;
  b.dx = dx;
  b.dh = dh;
  b.d_weight = d_weight;
  b.d_gate = d_gate;
  b.d_next_weight = d_next_weight;
  b.partials = static_cast<float*>(workspace);
  return launched(launch_norm_backward(dtype, b, d.sms, static_cast<cudaStream_t>(stream)));
}

size_t moe_matvec_prepared_bytes(int qfmt, int N, int K, int group, int swiglu) {
  return matvec_prepared_bytes({qfmt, N, K, group, swiglu ? 1 : 0});
}

moe_status moe_matvec_prepare(int qfmt, int N, int K, int group, int swiglu, const void* codes, const void* scale,
                              int scale_dtype, const void* zero, void* prepared, size_t prepared_bytes,
                              void* stream) {
  const MatvecShape shape = {qfmt, N, K, group, swiglu ? 1 : 0};
  const size_t need = matvec_prepared_bytes(shape);
  if (need == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (codes == nullptr || scale == nullptr || prepared == nullptr) return MOE_ERR_INVALID_ARG;
  if (qfmt == MOE_Q_INT4 && scale_dtype != MOE_BF16 && scale_dtype != MOE_FP16) return MOE_ERR_INVALID_ARG;
  if (qfmt == MOE_Q_FP4 && zero != nullptr) return MOE_ERR_INVALID_ARG;
  if (prepared_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  DevInfo d;
  const size_t ss = qfmt == MOE_Q_FP4 ? 1 : 2;
  const moe_status s = check_ptrs({{codes, 1}, {scale, ss}, {zero, 1}, {prepared, 256}}, &d);
  if (s != MOE_OK) return s;
  return launched(launch_matvec_prepare(shape, codes, scale, scale_dtype, zero, prepared,
                                        static_cast<cudaStream_t>(stream)));
}

moe_status moe_matvec(int qfmt, int N, int K, int group, int swiglu, float swiglu_limit, int scale_dtype,
                      const void* prepared, int dtype, const void* x, int64_t ld_x, int T, void* y, void* stream) {
  const MatvecShape shape = {qfmt, N, K, group, swiglu ? 1 : 0};
  if (T < 0 || ld_x < 0 || (dtype != MOE_BF16 && dtype != MOE_FP16)) return MOE_ERR_INVALID_ARG;
  if (matvec_prepared_bytes(shape) == 0) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (qfmt == MOE_Q_INT4 && scale_dtype != MOE_BF16 && scale_dtype != MOE_FP16) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (prepared == nullptr || x == nullptr || y == nullptr) return MOE_ERR_INVALID_ARG;
  DevInfo d;
  const moe_status s = check_ptrs({{prepared, 256}, {x, 2}, {y, 2}}, &d);
  if (s != MOE_OK) return s;
  return launched(launch_matvec(shape, swiglu_limit, scale_dtype, prepared, dtype, x, ld_x, T, y, d.sms,
                                static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
