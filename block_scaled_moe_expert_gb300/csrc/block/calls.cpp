// Python's way into the C entry points of include/moe_block.h and
// include/moe_route_fp4.h.
//
// The calls are short at decode (a kernel of a few microseconds), so their
// arguments are checked and their outputs allocated here rather than in
// Python: what Python spends on a dozen tensor attributes is more than the
// kernel. No arithmetic and no device code. The entry points come from the
// library that `binding` loads, by address.
#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <tuple>

#include "moe_route_fp4.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

namespace {

// ------------------------------------------------------------ entry points

#define MOE_BLOCK_CALLS(X)                                                                                       \
  X(moe_query_sort_layout)                                                                                      \
  X(moe_sort_tokens)                                                                                            \
  X(moe_permute_tokens)                                                                                         \
  X(moe_permute_tokens_backward)                                                                                \
  X(moe_unpermute_tokens)                                                                                       \
  X(moe_unpermute_tokens_backward)                                                                              \
  X(moe_norm_before)                                                                                            \
  X(moe_norm_backward_workspace_bytes)                                                                          \
  X(moe_norm_before_backward)                                                                                   \
  X(moe_norm_after)                                                                                             \
  X(moe_norm_after_backward)                                                                                    \
  X(moe_matvec_prepared_bytes)                                                                                  \
  X(moe_matvec_prepare)                                                                                         \
  X(moe_matvec)                                                                                                 \
  X(moe_route_workspace_bytes)                                                                                  \
  X(moe_route_tokens)                                                                                           \
  X(moe_route_tokens_backward)                                                                                  \
  X(moe_quantize_fp4)                                                                                           \
  X(moe_dequantize_fp4)                                                                                         \
  X(moe_matmul_fp4_prepared_bytes)                                                                              \
  X(moe_matmul_fp4_prepare)                                                                                     \
  X(moe_matmul_fp4_workspace_bytes)                                                                             \
  X(moe_matmul_fp4)

struct Api {
#define X(name) decltype(&::name) name = nullptr;
  MOE_BLOCK_CALLS(X)
#undef X
  PyObject* error = nullptr;  // MoeError(status, what)
} api;

// Names and addresses of the entry points, and the error type to raise.
void bind(const py::dict& address, const py::object& error) {
#define X(name) api.name = reinterpret_cast<decltype(&::name)>(address[#name].cast<uintptr_t>());
  MOE_BLOCK_CALLS(X)
#undef X
  api.error = error.inc_ref().ptr();
}

py::list entry_points() {
  py::list names;
#define X(name) names.append(#name);
  MOE_BLOCK_CALLS(X)
#undef X
  return names;
}

void check(int status, const char* what) {
  if (status == MOE_OK) return;
  const py::object e = py::reinterpret_borrow<py::object>(api.error)(status, what);
  PyErr_SetObject(api.error, e.ptr());
  throw py::error_already_set();
}

// ---------------------------------------------------------------- operands

// What every operand is asked. The kernels run past torch's dispatcher: neither a
// tangent nor a trace would learn of them.
void operand(const Tensor& t, int dev) {
  TORCH_CHECK(t.is_cuda() && t.get_device() == dev,
              "all tensors must live on the current CUDA device (one device per call)");
  TORCH_CHECK(!t._fw_grad(/*level=*/0).defined(), "forward-mode differentiation is not implemented for this operator");
  TORCH_CHECK(!torch::jit::tracer::isTracing(), "this operator cannot be traced: its kernels are not torch operators");
}

int dtype_code(at::ScalarType t) {
  return t == at::kBFloat16 ? MOE_BF16 : t == at::kHalf ? MOE_FP16 : t == at::kFloat ? MOE_FP32 : -1;
}

// Rows [n, H] with contiguous elements.
struct Rows {
  Tensor t;  // absent: null pointers
  int64_t ld = 0, n = 0, H = 0;
  const void* ptr() const { return t.defined() ? t.const_data_ptr() : nullptr; }
};

Rows strided(const Tensor& t) {
  Rows r{t, t.stride(0), t.size(0), t.size(1)};
  if (t.stride(1) != 1 && r.H != 1) {
    r.t = t.contiguous();
    r.ld = r.H;
  }
  return r;
}

// The operand that the others have to match.
struct First : Rows {
  at::ScalarType type;
  int code, dev;
};
First first(const Tensor& t, const char* what) {
  TORCH_CHECK_VALUE(t.dim() == 2, what, " must be [tokens, width], got ", t.sizes());
  const int code = dtype_code(t.scalar_type());
  TORCH_CHECK_VALUE(code >= 0, what, " must be bfloat16, float16 or float32, got ", t.scalar_type());
  const int dev = t.is_cuda() ? c10::cuda::current_device() : -1;
  operand(t, dev);
  First f;
  static_cast<Rows&>(f) = strided(t);
  TORCH_CHECK_VALUE(f.n <= INT32_MAX && f.H <= INT32_MAX, what, " is too large: ", t.sizes());
  f.type = t.scalar_type();
  f.code = code;
  f.dev = dev;
  return f;
}

Rows like(const Tensor& t, const First& f, int64_t n, const char* what) {
  TORCH_CHECK_VALUE(t.scalar_type() == f.type, what, " must be ", f.type, " like the rows it goes with, got ",
                    t.scalar_type());
  TORCH_CHECK_VALUE(t.dim() == 2 && t.size(0) == n && t.size(1) == f.H, what, " must have the shape [", n, ", ", f.H,
                    "], got ", t.sizes());
  operand(t, f.dev);
  return strided(t);
}
Rows like(const Maybe& t, const First& f, int64_t n, const char* what) { return t ? like(*t, f, n, what) : Rows(); }

Tensor output(const Maybe& out, const First& f, int64_t n, int64_t H) {
  if (!out) return at::empty({n, H}, f.t.options());
  TORCH_CHECK_VALUE(out->scalar_type() == f.type && out->dim() == 2 && out->size(0) == n && out->size(1) == H &&
                        out->is_contiguous(),
                    "out must be a contiguous ", f.type, " tensor of shape [", n, ", ", H, "]");
  operand(*out, f.dev);
  return *out;
}

void* stream(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
const void* ptr(const Tensor& t) { return t.defined() ? t.const_data_ptr() : nullptr; }
void* out_ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
py::object or_none(const Tensor& t) { return t.defined() ? py::cast(t) : py::none(); }

// -------------------------------------------------------- tokens by expert

struct Plan {
  Tensor buffer;
  moe_sort_layout layout;
  int T, E, K, align;
  Tensor counts, offsets, inv, row_slot;  // made when asked for

  // A contiguous part of the buffer, without the dispatcher's way to a view
  // (whole numbers have no gradient).
  Tensor part(Tensor& view, size_t at, std::initializer_list<int64_t> sizes) {
    if (!view.defined()) {
      view = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(), buffer.dtype());
      c10::TensorImpl* t = view.unsafeGetTensorImpl();
      t->set_storage_offset(static_cast<int64_t>(at / 4));
      t->set_sizes_contiguous(sizes);
    }
    return view;
  }
};

Plan sort_tokens(const Tensor& topk_idx, int E, int align) {
  TORCH_CHECK_VALUE(topk_idx.scalar_type() == at::kInt && topk_idx.dim() == 2,
                    "topk_idx must be an int32 tensor [T, K]");
  const int dev = topk_idx.is_cuda() ? c10::cuda::current_device() : -1;
  operand(topk_idx, dev);
  const Tensor idx = topk_idx.contiguous();
  TORCH_CHECK_VALUE(idx.size(0) <= INT32_MAX && idx.size(1) <= INT32_MAX, "topk_idx is too large: ", idx.sizes());
  Plan p;
  p.T = static_cast<int>(idx.size(0));
  p.K = static_cast<int>(idx.size(1));
  p.E = E;
  p.align = align;
  check(api.moe_query_sort_layout(p.T, E, p.K, align, &p.layout), "moe_query_sort_layout");
  p.buffer = at::empty({static_cast<int64_t>(p.layout.total_bytes / 4)}, idx.options());
  check(api.moe_sort_tokens(static_cast<const int32_t*>(ptr(idx)), p.T, E, p.K, align, p.buffer.data_ptr(),
                            p.layout.total_bytes, stream(dev)),
        "moe_sort_tokens");
  return p;
}

First plan_rows(const Tensor& t, const Plan& p, int n, const char* what) {
  First f = first(t, what);
  TORCH_CHECK_VALUE(f.n == n, what, " has ", f.n, " rows, the plan ", n);
  operand(p.buffer, f.dev);
  return f;
}

Tensor plan_weights(const Maybe& w, const Plan& p, int dev) {
  if (!w) return Tensor();
  TORCH_CHECK_VALUE(w->scalar_type() == at::kFloat && w->dim() == 2 && w->size(0) == p.T && w->size(1) == p.K,
                    "topk_w must be a float32 tensor [", p.T, ", ", p.K, "]");
  operand(*w, dev);
  return w->contiguous();
}

// permute_tokens and unpermute_tokens
Tensor move_rows(bool there, const Tensor& in, const Plan& p, const Maybe& topk_w, const Maybe& out) {
  const int M = p.layout.row_capacity;
  const First f = plan_rows(in, p, there ? p.T : M, there ? "hidden" : "rows");
  const Tensor w = plan_weights(topk_w, p, f.dev);
  const Tensor o = output(out, f, there ? M : p.T, f.H);
  check((there ? api.moe_permute_tokens : api.moe_unpermute_tokens)(
            f.code, f.ptr(), f.ld, static_cast<const float*>(ptr(w)), p.buffer.const_data_ptr(), p.layout.total_bytes,
            p.T, static_cast<int>(f.H), p.E, p.K, p.align, o.data_ptr(), stream(f.dev)),
        there ? "moe_permute_tokens" : "moe_unpermute_tokens");
  return o;
}

// and their gradients: `there` names the direction whose gradient it is
std::tuple<Tensor, py::object> move_rows_backward(bool there, const Tensor& grad, const Plan& p, const Maybe& other,
                                                  const Maybe& topk_w) {
  const int M = p.layout.row_capacity;
  const First f = plan_rows(grad, p, there ? M : p.T, there ? "d_rows" : "d_out");
  const Tensor w = plan_weights(topk_w, p, f.dev);
  const int n = there ? p.T : M;
  Rows o;
  Tensor dw;
  if (w.defined()) {
    const char* what = there ? "hidden" : "rows";
    TORCH_CHECK_VALUE(other.has_value(), "the gradient of topk_w needs ", what);
    o = like(*other, f, n, what);
    dw = at::empty(w.sizes(), w.options());
  }
  const Tensor d = at::empty({n, f.H}, f.t.options());
  check((there ? api.moe_permute_tokens_backward : api.moe_unpermute_tokens_backward)(
            f.code, f.ptr(), f.ld, o.ptr(), o.ld, static_cast<const float*>(ptr(w)), p.buffer.const_data_ptr(),
            p.layout.total_bytes, p.T, static_cast<int>(f.H), p.E, p.K, p.align, d.data_ptr(),
            static_cast<float*>(out_ptr(dw)), stream(f.dev)),
        there ? "moe_permute_tokens_backward" : "moe_unpermute_tokens_backward");
  return {d, or_none(dw)};
}

// ----------------------------------------------------- norms around a block

struct NormWeights {
  Tensor w, next;
  int f32 = 0;
};

Tensor norm_weight(const Maybe& w, const First& f, const char* what) {
  if (!w) return Tensor();
  TORCH_CHECK_VALUE(w->dim() == 1 && w->size(0) == f.H, what, " must have the shape (", f.H, ",), got ", w->sizes());
  TORCH_CHECK_VALUE(w->scalar_type() == f.type || w->scalar_type() == at::kFloat, what, " must be ", f.type,
                    " or float32, got ", w->scalar_type());
  operand(*w, f.dev);
  return w->contiguous();
}

NormWeights norm_weights(const Maybe& w, const Maybe& next, const First& f) {
  NormWeights n{norm_weight(w, f, "weight"), norm_weight(next, f, "next_weight")};
  const Tensor& any = n.w.defined() ? n.w : n.next;
  TORCH_CHECK_VALUE(!n.w.defined() || !n.next.defined() || n.w.scalar_type() == n.next.scalar_type(),
                    "weight and next_weight must have one type");
  n.f32 = any.defined() && any.scalar_type() == at::kFloat;
  return n;
}

struct Gate {
  Tensor t;
  int kind = MOE_GATE_NONE, act;
  int64_t ld = 0;
};

Gate gate_arg(const Maybe& gate, const std::string& act, const First& f) {
  Gate g;
  g.act = act == "none" ? MOE_GATE_LINEAR : act == "sigmoid" ? MOE_GATE_SIGMOID : act == "tanh" ? MOE_GATE_TANH : -1;
  TORCH_CHECK_VALUE(g.act >= 0, "gate_act must be 'none', 'sigmoid' or 'tanh', got '", act, "'");
  if (!gate) return g;
  TORCH_CHECK_VALUE(gate->scalar_type() == f.type, "gate must be ", f.type, " like x, got ", gate->scalar_type());
  operand(*gate, f.dev);
  if (gate->dim() == 1 && gate->size(0) == f.H) {
    g.kind = MOE_GATE_CHANNEL;
    g.t = gate->contiguous();
  } else if (gate->dim() == 2 && gate->size(0) == f.n && gate->size(1) == f.H && f.H > 1) {
    g.kind = MOE_GATE_ELEMENT;
    const Rows r = strided(*gate);
    g.t = r.t;
    g.ld = r.ld;
  } else if (gate->dim() == 2 && gate->size(0) == f.n && gate->size(1) == 1) {
    g.kind = MOE_GATE_TOKEN;
    g.t = *gate;
    g.ld = gate->stride(0);
  } else {
    TORCH_CHECK_VALUE(false, "gate must be [H], [T, 1] or [T, H] for x of [", f.n, ", ", f.H, "], got ", gate->sizes());
  }
  return g;
}

Tensor norm_workspace(const First& f, size_t* bytes) {
  *bytes = f.H > INT32_MAX ? 0 : api.moe_norm_backward_workspace_bytes(static_cast<int>(f.H));
  if (*bytes == 0) check(MOE_ERR_UNSUPPORTED_SHAPE, "moe_norm_backward_workspace_bytes");
  return at::empty({static_cast<int64_t>(*bytes)}, f.t.options().dtype(at::kByte));
}

Tensor empty_like(const Tensor& t) { return t.defined() ? at::empty(t.sizes(), t.options()) : Tensor(); }

Tensor norm_before(const Tensor& x, const Maybe& weight, double eps, double w_offset, const Maybe& out) {
  const First f = first(x, "x");
  const NormWeights w = norm_weights(weight, std::nullopt, f);
  const Tensor y = output(out, f, f.n, f.H);
  check(api.moe_norm_before(f.code, f.ptr(), f.ld, ptr(w.w), w.f32, static_cast<float>(w_offset),
                            static_cast<float>(eps), static_cast<int>(f.n), static_cast<int>(f.H), y.data_ptr(),
                            stream(f.dev)),
        "moe_norm_before");
  return y;
}

std::tuple<Tensor, py::object> norm_before_backward(const Tensor& dy, const Tensor& x, const Maybe& weight, double eps,
                                                    double w_offset, const Maybe& dr) {
  const First f = first(x, "x");
  const Rows d = like(dy, f, f.n, "dy"), res = like(dr, f, f.n, "dr");
  const NormWeights w = norm_weights(weight, std::nullopt, f);
  const Tensor dx = at::empty({f.n, f.H}, f.t.options()), dw = empty_like(w.w);
  size_t bytes;
  const Tensor ws = norm_workspace(f, &bytes);
  check(api.moe_norm_before_backward(f.code, d.ptr(), d.ld, f.ptr(), f.ld, res.ptr(), res.ld, ptr(w.w), w.f32,
                                     static_cast<float>(w_offset), static_cast<float>(eps), static_cast<int>(f.n),
                                     static_cast<int>(f.H), dx.data_ptr(), out_ptr(dw), ws.data_ptr(), bytes,
                                     stream(f.dev)),
        "moe_norm_before_backward");
  return {dx, or_none(dw)};
}

// (r, y); y is None without the next norm
std::tuple<Tensor, py::object> norm_after(const Tensor& x, const Tensor& h, const Maybe& weight, const Maybe& gate,
                                          const std::string& gate_act, double alpha, double beta, double eps,
                                          double w_offset, bool norm, const Maybe& next_weight, bool next_norm,
                                          double next_eps) {
  const First f = first(x, "x");
  const Rows rh = like(h, f, f.n, "h");
  TORCH_CHECK_VALUE(norm || !weight, "weight belongs to the norm of h: norm must be true");
  TORCH_CHECK_VALUE(next_norm || !next_weight,
                    "next_weight belongs to the next block's norm: next_norm must not be False");
  const NormWeights w = norm_weights(weight, next_weight, f);
  const Gate g = gate_arg(gate, gate_act, f);
  const Tensor r = at::empty({f.n, f.H}, f.t.options());
  const Tensor y = next_norm ? at::empty({f.n, f.H}, f.t.options()) : Tensor();
  check(api.moe_norm_after(f.code, f.ptr(), f.ld, rh.ptr(), rh.ld, norm, ptr(w.w), ptr(w.next), w.f32,
                           static_cast<float>(w_offset), g.kind, g.act, ptr(g.t), g.ld, static_cast<float>(alpha),
                           static_cast<float>(beta), static_cast<float>(eps), static_cast<float>(next_eps),
                           static_cast<int>(f.n), static_cast<int>(f.H), r.data_ptr(), out_ptr(y), stream(f.dev)),
        "moe_norm_after");
  return {r, or_none(y)};
}

py::tuple norm_after_backward(const Tensor& dr, const Tensor& h, const Maybe& weight, const Maybe& gate,
                              const std::string& gate_act, double alpha, double beta, double eps, double w_offset,
                              bool norm, const Maybe& dy, const Maybe& r, const Maybe& next_weight, double next_eps) {
  const First f = first(h, "h");
  const Rows d = like(dr, f, f.n, "dr");
  TORCH_CHECK_VALUE(dy.has_value() == r.has_value(), "dy and r come together");
  TORCH_CHECK_VALUE(norm || !weight, "weight belongs to the norm of h: norm must be true");
  TORCH_CHECK_VALUE(dy || !next_weight, "next_weight belongs to the next block's norm: dy is missing");
  const Rows rdy = like(dy, f, f.n, "dy"), rr = like(r, f, f.n, "r");
  const NormWeights w = norm_weights(weight, next_weight, f);
  const Gate g = gate_arg(gate, gate_act, f);
  const bool same = !dy && beta == 1.0;  // dx is dr
  const Tensor dx = same ? Tensor() : at::empty({f.n, f.H}, f.t.options());
  const Tensor dh = at::empty({f.n, f.H}, f.t.options());
  const Tensor dw = empty_like(w.w), dnext = empty_like(w.next), dgate = empty_like(g.t);
  size_t bytes;
  const Tensor ws = norm_workspace(f, &bytes);
  check(api.moe_norm_after_backward(
            f.code, d.ptr(), d.ld, rdy.ptr(), rdy.ld, f.ptr(), f.ld, rr.ptr(), rr.ld, norm, ptr(w.w), ptr(w.next),
            w.f32, static_cast<float>(w_offset), g.kind, g.act, ptr(g.t), g.ld, static_cast<float>(alpha),
            static_cast<float>(beta), static_cast<float>(eps), static_cast<float>(next_eps), static_cast<int>(f.n),
            static_cast<int>(f.H), out_ptr(dx), dh.data_ptr(), out_ptr(dw), out_ptr(dgate), out_ptr(dnext),
            ws.data_ptr(), bytes, stream(f.dev)),
        "moe_norm_after_backward");
  return py::make_tuple(same ? dr : dx, dh, or_none(dw), or_none(dgate), or_none(dnext));
}

// --------------------------------------------- products with 4-bit weights

struct MatvecWeights {
  int qfmt, N, K, group, scale_dtype;
  bool swiglu;
  Tensor prepared;
};

MatvecWeights prepare_matvec(int qfmt, int N, int K, int group, bool swiglu, const Tensor& w, const Tensor& scale,
                             const Maybe& zero) {
  const size_t bytes = api.moe_matvec_prepared_bytes(qfmt, N, K, group, swiglu);
  if (bytes == 0) check(MOE_ERR_UNSUPPORTED_SHAPE, "moe_matvec_prepared_bytes");
  const int64_t groups = (K + group - 1) / group;
  auto shaped = [&](const Tensor& t, int64_t cols) { return t.dim() == 2 && t.size(0) == N && t.size(1) == cols; };
  TORCH_CHECK_VALUE(w.scalar_type() == at::kByte && shaped(w, K / 2), "w must be uint8 [", N, ", ", K / 2, "]");
  const at::ScalarType st = scale.scalar_type();
  TORCH_CHECK_VALUE((qfmt == MOE_Q_FP4 ? st == at::kByte : st == at::kBFloat16 || st == at::kHalf) &&
                        shaped(scale, groups),
                    "w_scale must be ", qfmt == MOE_Q_FP4 ? "uint8" : "bfloat16 or float16", " [", N, ", ", groups, "]");
  TORCH_CHECK_VALUE(!zero || (qfmt == MOE_Q_INT4 && zero->scalar_type() == at::kByte && shaped(*zero, groups)),
                    "w_zero must be uint8 [", N, ", ", groups, "], for int4 weights");
  const int dev = w.is_cuda() ? c10::cuda::current_device() : -1;
  operand(w, dev);
  operand(scale, dev);
  if (zero) operand(*zero, dev);
  const Tensor wc = w.contiguous(), sc = scale.contiguous(), zc = zero ? zero->contiguous() : Tensor();
  MatvecWeights m{qfmt, N, K, group, qfmt == MOE_Q_FP4 ? 0 : dtype_code(st), swiglu,
                  at::empty({static_cast<int64_t>(bytes)}, w.options())};
  check(api.moe_matvec_prepare(qfmt, N, K, group, swiglu, ptr(wc), ptr(sc), m.scale_dtype, ptr(zc),
                               m.prepared.data_ptr(), bytes, stream(dev)),
        "moe_matvec_prepare");
  return m;
}

Tensor matvec(const Tensor& x, const MatvecWeights& m, std::optional<double> limit, const Maybe& out) {
  const First f = first(x, "x");
  TORCH_CHECK_VALUE(f.code != MOE_FP32, "matvec takes bfloat16 or float16 x, got ", f.type);
  TORCH_CHECK_VALUE(f.H == m.K, "x has ", f.H, " columns, the prepared weights ", m.K);
  TORCH_CHECK_VALUE(!x.requires_grad() || !c10::GradMode::is_enabled(),
                    "matvec has no gradient: call it without gradients (torch.no_grad) or on x.detach()");
  TORCH_CHECK_VALUE(!limit || m.swiglu, "swiglu_limit is for weights prepared with swiglu=True");
  operand(m.prepared, f.dev);
  const Tensor y = output(out, f, f.n, m.swiglu ? m.N / 2 : m.N);
  check(api.moe_matvec(m.qfmt, m.N, m.K, m.group, m.swiglu, limit ? static_cast<float>(*limit) : -1.f, m.scale_dtype,
                       m.prepared.const_data_ptr(), f.code, f.ptr(), f.ld, static_cast<int>(f.n), y.data_ptr(),
                       stream(f.dev)),
        "moe_matvec");
  return y;
}

// ------------------------------------------------------------------ outputs

// An uninitialised tensor on the current device, without the dispatcher's way to it: that
// takes longer than the small calls' kernels.
Tensor make_empty(at::IntArrayRef sizes, at::ScalarType type) {
  return Tensor(at::detail::empty_generic(sizes, c10::cuda::CUDACachingAllocator::get(),
                                          c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt));
}
// A contiguous part of such a tensor as one of its own (element offset `at` in units of type).
Tensor part_of(const Tensor& whole, int64_t at, at::IntArrayRef sizes, at::ScalarType type) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(),
                                                      c10::scalarTypeToTypeMeta(type));
  c10::TensorImpl* impl = t.unsafeGetTensorImpl();
  impl->set_storage_offset(at);
  impl->set_sizes_contiguous(sizes);
  return t;
}
int64_t round_up(int64_t n, int64_t unit) { return (n + unit - 1) / unit * unit; }

// ----------------------------------------------------------------- routing

int score_code(const std::string& score) {
  const int c = score == "softmax" ? MOE_SCORE_SOFTMAX : score == "sigmoid" ? MOE_SCORE_SIGMOID : -1;
  TORCH_CHECK_VALUE(c >= 0, "score must be 'softmax' or 'sigmoid', got '", score, "'");
  return c;
}

Tensor f32_vector(const Maybe& t, const First& f, const char* what) {
  if (!t) return Tensor();
  TORCH_CHECK_VALUE(t->scalar_type() == at::kFloat && t->dim() == 1 && t->size(0) == f.H, what,
                    " must be a float32 tensor of shape (", f.H, ",)");
  operand(*t, f.dev);
  return t->contiguous();
}

// (topk_idx, topk_w) or (topk_idx, topk_w, mean_scores), parts of one allocation
py::tuple route_tokens(const Tensor& logits, int k, const std::string& score, const Maybe& bias, int num_groups,
                       int top_groups, const std::string& group_score, bool renormalize, double scale, bool mean) {
  const First f = first(logits, "logits");
  const int by = score_code(score);
  TORCH_CHECK_VALUE(group_score == "top2" || group_score == "max", "group_score must be 'top2' or 'max', got '",
                    group_score, "'");
  const Tensor b = f32_vector(bias, f, "bias");
  // sizes are checked by the call below, before any use of these
  const int64_t cols = k > 0 && k <= 32 ? k : 1, slots = round_up(f.n * cols, 64), experts = mean ? round_up(f.H, 64) : 0;
  const Tensor all = make_empty({2 * slots + experts}, at::kInt);
  const Tensor idx = part_of(all, 0, {f.n, cols}, at::kInt), w = part_of(all, slots, {f.n, cols}, at::kFloat);
  Tensor m, ws;
  size_t bytes = 0;
  if (mean) {
    m = part_of(all, 2 * slots, {f.H}, at::kFloat);
    bytes = api.moe_route_workspace_bytes(static_cast<int>(f.H));
    ws = make_empty({static_cast<int64_t>(bytes)}, at::kByte);
  }
  check(api.moe_route_tokens(f.code, f.ptr(), f.ld, static_cast<const float*>(ptr(b)), static_cast<int>(f.n),
                             static_cast<int>(f.H), k, by, num_groups, top_groups,
                             group_score == "top2" ? MOE_GROUP_TOP2 : MOE_GROUP_MAX, renormalize,
                             static_cast<float>(scale), static_cast<int32_t*>(idx.data_ptr()),
                             static_cast<float*>(w.data_ptr()), static_cast<float*>(out_ptr(m)), out_ptr(ws), bytes,
                             stream(f.dev)),
        "moe_route_tokens");
  return mean ? py::make_tuple(idx, w, m) : py::make_tuple(idx, w);
}

Tensor route_tokens_backward(const Tensor& d_w, const Tensor& logits, const Tensor& topk_idx, const std::string& score,
                             bool renormalize, double scale, const Maybe& d_mean) {
  const First f = first(logits, "logits");
  const int by = score_code(score);
  TORCH_CHECK_VALUE(topk_idx.scalar_type() == at::kInt && topk_idx.dim() == 2 && topk_idx.size(0) == f.n,
                    "topk_idx must be an int32 tensor [", f.n, ", K]");
  TORCH_CHECK_VALUE(d_w.scalar_type() == at::kFloat && d_w.sizes() == topk_idx.sizes(),
                    "d_topk_w must be a float32 tensor of topk_idx's shape");
  TORCH_CHECK_VALUE(topk_idx.size(1) <= INT32_MAX, "topk_idx is too large: ", topk_idx.sizes());
  operand(topk_idx, f.dev);
  operand(d_w, f.dev);
  const Tensor idx = topk_idx.contiguous(), dw = d_w.contiguous(), dm = f32_vector(d_mean, f, "d_mean_scores");
  const Tensor dx = make_empty({f.n, f.H}, f.type);
  check(api.moe_route_tokens_backward(f.code, static_cast<const float*>(ptr(dw)), static_cast<const float*>(ptr(dm)),
                                      f.ptr(), f.ld, static_cast<const int32_t*>(ptr(idx)), static_cast<int>(f.n),
                                      static_cast<int>(f.H), static_cast<int>(idx.size(1)), by, renormalize,
                                      static_cast<float>(scale), dx.data_ptr(), stream(f.dev)),
        "moe_route_tokens_backward");
  return dx;
}

// ----------------------------------------------------------- the FP4 format

void no_gradient(const Tensor& x, const char* what) {
  TORCH_CHECK_VALUE(!x.requires_grad() || !c10::GradMode::is_enabled(), what,
                    " has no gradient: call it without gradients (torch.no_grad) or on x.detach()");
}

// (codes, scale) of x [..., C]
std::tuple<Tensor, Tensor> quantize_fp4(const Tensor& x) {
  const at::IntArrayRef sizes = x.sizes();
  TORCH_CHECK_VALUE(x.dim() >= 1, "x must have at least one dimension");
  no_gradient(x, "quantize_fp4");
  const int64_t C = sizes.back();
  // rows: every dimension but the last
  const First f = first(x.dim() == 2 ? x : x.contiguous().view({C == 0 ? 0 : x.numel() / C, C}), "x");
  TORCH_CHECK_VALUE(C > 0 && C % 32 == 0, "the last dimension must be a multiple of 32, got ", C);
  c10::SmallVector<int64_t, 6> cs(sizes.begin(), sizes.end()), ss(cs);
  cs.back() = C / 2;
  ss.back() = C / 32;
  const Tensor codes = make_empty(cs, at::kByte), scale = make_empty(ss, at::kByte);
  check(api.moe_quantize_fp4(f.code, f.ptr(), f.ld, static_cast<int>(f.n), static_cast<int>(C), codes.data_ptr(),
                             scale.data_ptr(), stream(f.dev)),
        "moe_quantize_fp4");
  return {codes, scale};
}

Tensor dequantize_fp4(const Tensor& codes, const Tensor& scale, at::ScalarType dtype) {
  const int code = dtype_code(dtype);
  TORCH_CHECK_VALUE(code >= 0, "dtype must be bfloat16, float16 or float32, got ", dtype);
  TORCH_CHECK_VALUE(codes.scalar_type() == at::kByte && codes.dim() >= 1 && codes.size(-1) % 16 == 0 && codes.size(-1) > 0,
                    "codes must be uint8 [..., C / 2], C a multiple of 32");
  c10::SmallVector<int64_t, 6> sizes(codes.sizes().begin(), codes.sizes().end());
  const int64_t C = 2 * sizes.back();
  sizes.back() = C / 32;
  TORCH_CHECK_VALUE(scale.scalar_type() == at::kByte && scale.sizes() == at::IntArrayRef(sizes),
                    "scale must be uint8 of shape ", at::IntArrayRef(sizes), ", got ", scale.sizes());
  const int dev = codes.is_cuda() ? c10::cuda::current_device() : -1;
  operand(codes, dev);
  operand(scale, dev);
  const Tensor c = codes.contiguous(), s = scale.contiguous();
  sizes.back() = C;
  const Tensor out = make_empty(sizes, dtype);
  const int64_t rows = c.numel() / (C / 2);
  TORCH_CHECK_VALUE(rows <= INT32_MAX && C <= INT32_MAX, "codes is too large: ", codes.sizes());
  check(api.moe_dequantize_fp4(code, ptr(c), ptr(s), static_cast<int>(rows), static_cast<int>(C), out.data_ptr(),
                               stream(dev)),
        "moe_dequantize_fp4");
  return out;
}

struct MatmulWeights {
  int N, K;
  bool swiglu;
  Tensor prepared;
};

MatmulWeights prepare_matmul_fp4(int N, int K, bool swiglu, const Tensor& w, const Tensor& scale) {
  const size_t bytes = api.moe_matmul_fp4_prepared_bytes(N, K, swiglu);
  if (bytes == 0) check(MOE_ERR_UNSUPPORTED_SHAPE, "moe_matmul_fp4_prepared_bytes");
  auto shaped = [&](const Tensor& t, int64_t cols) {
    return t.scalar_type() == at::kByte && t.dim() == 2 && t.size(0) == N && t.size(1) == cols;
  };
  TORCH_CHECK_VALUE(shaped(w, K / 2), "w must be uint8 [", N, ", ", K / 2, "]");
  TORCH_CHECK_VALUE(shaped(scale, K / 32), "w_scale must be uint8 [", N, ", ", K / 32, "]");
  const int dev = w.is_cuda() ? c10::cuda::current_device() : -1;
  operand(w, dev);
  operand(scale, dev);
  const Tensor wc = w.contiguous(), sc = scale.contiguous();
  MatmulWeights m{N, K, swiglu, at::empty({static_cast<int64_t>(bytes)}, w.options())};
  check(api.moe_matmul_fp4_prepare(N, K, swiglu, ptr(wc), ptr(sc), m.prepared.data_ptr(), bytes, stream(dev)),
        "moe_matmul_fp4_prepare");
  return m;
}

int64_t matmul_fp4_workspace_bytes(const MatmulWeights& m, int64_t T) {
  const size_t bytes = T < 0 || T > INT32_MAX ? 0 : api.moe_matmul_fp4_workspace_bytes(static_cast<int>(T), m.K);
  if (bytes == 0) check(MOE_ERR_UNSUPPORTED_SHAPE, "moe_matmul_fp4_workspace_bytes");
  return static_cast<int64_t>(bytes);
}

Tensor matmul_fp4(const Tensor& x, const MatmulWeights& m, std::optional<double> limit, const Maybe& workspace,
                  const Maybe& out) {
  const First f = first(x, "x");
  TORCH_CHECK_VALUE(f.code != MOE_FP32, "matmul_fp4 takes bfloat16 or float16 x, got ", f.type);
  TORCH_CHECK_VALUE(f.H == m.K, "x has ", f.H, " columns, the prepared weights ", m.K);
  no_gradient(x, "matmul_fp4");
  TORCH_CHECK_VALUE(!limit || m.swiglu, "swiglu_limit is for weights prepared with swiglu=True");
  operand(m.prepared, f.dev);
  const int64_t need = matmul_fp4_workspace_bytes(m, f.n), cols = m.swiglu ? m.N / 2 : m.N;
  Tensor ws, y;
  if (out) y = output(out, f, f.n, cols);
  if (workspace) {
    TORCH_CHECK_VALUE(workspace->scalar_type() == at::kByte && workspace->is_contiguous(),
                      "workspace must be a contiguous uint8 tensor");
    operand(*workspace, f.dev);
    ws = *workspace;
  }
  if (!out && !workspace && need <= 256) {  // a few tokens: y and the status word are one allocation
    const int64_t status_at = round_up(2 * f.n * cols, 256);
    ws = make_empty({status_at + need}, at::kByte);
    y = part_of(ws, 0, {f.n, cols}, f.type);
    ws = part_of(ws, status_at, {need}, at::kByte);
  }
  if (!ws.defined()) ws = make_empty({need}, at::kByte);
  if (!y.defined()) y = make_empty({f.n, cols}, f.type);
  check(api.moe_matmul_fp4(m.N, m.K, m.swiglu, limit ? static_cast<float>(*limit) : -1.f, m.prepared.const_data_ptr(),
                           f.code, f.ptr(), f.ld, static_cast<int>(f.n), ws.data_ptr(),
                           static_cast<size_t>(ws.numel()), y.data_ptr(), stream(f.dev)),
        "moe_matmul_fp4");
  return y;
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  using torch::wrap_pybind_function;
  m.def("bind", &bind);
  m.def("entry_points", &entry_points);
  py::class_<Plan>(m, "Plan")
      .def_readonly("buffer", &Plan::buffer)
      .def_readonly("T", &Plan::T)
      .def_readonly("E", &Plan::E)
      .def_readonly("K", &Plan::K)
      .def_readonly("align", &Plan::align)
      .def_property_readonly("row_capacity", [](const Plan& p) { return p.layout.row_capacity; })
      .def_property_readonly("counts", [](Plan& p) { return p.part(p.counts, p.layout.counts, {p.E}); })
      .def_property_readonly("offsets", [](Plan& p) { return p.part(p.offsets, p.layout.offsets, {p.E + 1}); })
      .def_property_readonly("inv", [](Plan& p) { return p.part(p.inv, p.layout.inv, {p.T, p.K}); })
      .def_property_readonly("row_slot", [](Plan& p) {
        return p.part(p.row_slot, p.layout.row_slot, {p.layout.row_capacity});
      });
  m.def("sort_tokens", wrap_pybind_function(sort_tokens));
  m.def("move_rows", wrap_pybind_function(move_rows));
  m.def("move_rows_backward", wrap_pybind_function(move_rows_backward));
  m.def("norm_before", wrap_pybind_function(norm_before));
  m.def("norm_before_backward", wrap_pybind_function(norm_before_backward));
  m.def("norm_after", wrap_pybind_function(norm_after));
  m.def("norm_after_backward", wrap_pybind_function(norm_after_backward));
  py::class_<MatvecWeights>(m, "MatvecWeights").def_readonly("prepared", &MatvecWeights::prepared);
  m.def("prepare_matvec", wrap_pybind_function(prepare_matvec));
  m.def("matvec", wrap_pybind_function(matvec));
  m.def("route_tokens", wrap_pybind_function(route_tokens));
  m.def("route_tokens_backward", wrap_pybind_function(route_tokens_backward));
  m.def("quantize_fp4", wrap_pybind_function(quantize_fp4));
  m.def("dequantize_fp4", wrap_pybind_function(dequantize_fp4));
  py::class_<MatmulWeights>(m, "MatmulWeights").def_readonly("prepared", &MatmulWeights::prepared);
  m.def("prepare_matmul_fp4", wrap_pybind_function(prepare_matmul_fp4));
  m.def("matmul_fp4_workspace_bytes", wrap_pybind_function(matmul_fp4_workspace_bytes));
  m.def("matmul_fp4", wrap_pybind_function(matmul_fp4));
}
