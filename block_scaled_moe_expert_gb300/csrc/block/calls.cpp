// Python's way into the C entry points of include/moe_block.h.
//
// The calls are short at decode (a kernel of a few microseconds), so their
// arguments are checked and their outputs allocated here rather than in
// Python: what Python spends on a dozen tensor attributes is more than the
// kernel. No arithmetic and no device code. The entry points come from the
// library that `binding` loads, by address.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/jit/frontend/tracer.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <tuple>

#include "moe_block.h"

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
  X(moe_matvec)

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
}
