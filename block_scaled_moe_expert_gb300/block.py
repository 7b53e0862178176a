"""Operators around the experts forward (ctypes binding of include/moe_block.h).

* sort_tokens / permute_tokens / unpermute_tokens: tokens sorted by expert and
  back with the routing weights applied, and their gradients;
* norm_before / norm_after: the norms around a block fused with its gate, the
  residual scale and the next block's norm, and their gradients;
* prepare_matvec / matvec: products of a few tokens with 4-bit weights.

As in `binding`, every step runs in the CUDA library on torch's current
stream, and a missing library raises. permute_tokens, unpermute_tokens,
norm_before and norm_after take part in autograd; the *_backward functions are
their gradients as plain calls. Rows may be strided (the elements of a row
contiguous); anything else is made contiguous first.
"""
import ctypes
import math

import torch
from torch.autograd.function import once_differentiable

from . import binding as _b

_c = ctypes
_vp, _sz, _int, _f32, _i64 = _c.c_void_p, _c.c_size_t, _c.c_int, _c.c_float, _c.c_int64

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
MOE_Q_FP4, MOE_Q_INT4 = 0, 1
QFMT = {"fp4": MOE_Q_FP4, "int4": MOE_Q_INT4}
GATE_ACT = {"none": 0, "sigmoid": 1, "tanh": 2}
_NO_LIMIT = float("nan")


class MoeSortLayout(_c.Structure):
    _fields_ = [("total_bytes", _sz), ("status", _sz), ("counts", _sz), ("offsets", _sz), ("inv", _sz),
                ("row_slot", _sz), ("row_capacity", _c.c_int32)]


_ROWS_TAIL = [_vp, _sz, _int, _int, _int, _int, _int]  # plan, plan_bytes, T, H, E, K, row_align
_SIGS = {
    "moe_query_sort_layout": (_int, [_int, _int, _int, _int, _c.POINTER(MoeSortLayout)]),
    "moe_sort_tokens": (_int, [_vp, _int, _int, _int, _int, _vp, _sz, _vp]),
    "moe_permute_tokens": (_int, [_int, _vp, _i64, _vp, *_ROWS_TAIL, _vp, _vp]),
    "moe_permute_tokens_backward": (_int, [_int, _vp, _i64, _vp, _i64, _vp, *_ROWS_TAIL, _vp, _vp, _vp]),
    "moe_unpermute_tokens": (_int, [_int, _vp, _i64, _vp, *_ROWS_TAIL, _vp, _vp]),
    "moe_unpermute_tokens_backward": (_int, [_int, _vp, _i64, _vp, _i64, _vp, *_ROWS_TAIL, _vp, _vp, _vp]),
    "moe_norm_before": (_int, [_int, _vp, _i64, _vp, _int, _f32, _f32, _int, _int, _vp, _vp]),
    "moe_norm_backward_workspace_bytes": (_sz, [_int]),
    "moe_norm_before_backward": (_int, [_int, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _int, _f32, _f32, _int, _int,
                                        _vp, _vp, _vp, _sz, _vp]),
    "moe_norm_after": (_int, [_int, _vp, _i64, _vp, _i64, _int, _vp, _vp, _int, _f32, _int, _int, _vp, _i64, _f32,
                              _f32, _f32, _f32, _int, _int, _vp, _vp, _vp]),
    "moe_norm_after_backward": (_int, [_int, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp, _vp, _int, _f32,
                                       _int, _int, _vp, _i64, _f32, _f32, _f32, _f32, _int, _int, _vp, _vp, _vp,
                                       _vp, _vp, _vp, _sz, _vp]),
    "moe_matvec_prepared_bytes": (_sz, [_int, _int, _int, _int, _int]),
    "moe_matvec_prepare": (_int, [_int, _int, _int, _int, _int, _vp, _vp, _int, _vp, _vp, _sz, _vp]),
    "moe_matvec": (_int, [_int, _int, _int, _int, _int, _f32, _int, _vp, _int, _vp, _i64, _int, _vp, _vp]),
}

_lib_seen = None


def lib():
    """The library of `binding`, with the signatures of include/moe_block.h."""
    global _lib_seen
    L = _b.lib()
    if L is not _lib_seen:
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib_seen = L
    return L


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _check(status, what):
    if status != 0:
        raise _b.MoeError(status, what)


def _dtype(t, what):
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _rows(t, like, shape, what):
    """A [n, H] operand of `like`'s type with contiguous rows."""
    if t.dtype != like.dtype:
        raise ValueError(f"{what} must be {like.dtype} like the rows it goes with, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    return _row_strided(t)


def _row_strided(t):
    return t if (t.stride(1) == 1 or t.shape[1] == 1) and t.stride(0) >= 0 else t.contiguous()


def _2d(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what} must be [tokens, width], got {tuple(t.shape)}")


def _out(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.dtype != dtype or tuple(out.shape) != tuple(shape) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    return out


def _p(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------ tokens by expert

class SortPlan:
    """Where the T * K slots of a batch go (moe_sort_tokens): group e holds the
    rows offsets[e] .. offsets[e] + counts[e] - 1; inv [T, K] is each slot's
    row (-1 if skipped), row_slot [row_capacity] each row's slot (-1 if none).
    `buffer` starts with the status word that `device_status` reads."""

    def __init__(self, buffer, layout, T, E, K, row_align):
        self.buffer, self.nbytes = buffer, layout.total_bytes
        self.T, self.num_experts, self.K, self.row_align = T, E, K, row_align
        self.row_capacity = layout.row_capacity
        i, M = buffer, layout.row_capacity
        self.counts = i.as_strided((E,), (1,), layout.counts // 4)
        self.offsets = i.as_strided((E + 1,), (1,), layout.offsets // 4)
        self.inv = i.as_strided((T, K), (K, 1), layout.inv // 4)
        self.row_slot = i.as_strided((M,), (1,), layout.row_slot // 4)


def sort_layout(T, num_experts, K, row_align=1):
    out = MoeSortLayout()
    _check(lib().moe_query_sort_layout(T, num_experts, K, row_align, _c.byref(out)), "moe_query_sort_layout")
    return out


def sort_tokens(topk_idx, num_experts, row_align=1):
    """Sort the slots of topk_idx (int32 [T, K], -1 = skipped) by expert, each
    group starting at a multiple of row_align. Returns a SortPlan. An id outside
    [-1, num_experts) counts as skipped and sets MOE_DEV_BAD_EXPERT_ID, which
    device_status(plan.buffer) reads."""
    if topk_idx.dtype != torch.int32 or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be an int32 tensor [T, K]")
    topk_idx = topk_idx.contiguous()
    _b._same_device(topk_idx)
    T, K = topk_idx.shape
    layout = sort_layout(T, num_experts, K, row_align)
    buffer = torch.empty(layout.total_bytes // 4, dtype=torch.int32, device=topk_idx.device)
    _check(lib().moe_sort_tokens(topk_idx.data_ptr(), T, num_experts, K, row_align, buffer.data_ptr(),
                                 layout.total_bytes, _stream()), "moe_sort_tokens")
    return SortPlan(buffer, layout, T, num_experts, K, row_align)


def _plan_args(plan, H):
    return plan.buffer.data_ptr(), plan.nbytes, plan.T, H, plan.num_experts, plan.K, plan.row_align


def _weights_arg(topk_w, plan):
    if topk_w is None:
        return None
    if topk_w.dtype != torch.float32 or tuple(topk_w.shape) != (plan.T, plan.K):
        raise ValueError(f"topk_w must be a float32 tensor [{plan.T}, {plan.K}]")
    return topk_w.contiguous()


def _tokens(t, plan, what):
    _2d(t, what)
    if t.shape[0] != plan.T:
        raise ValueError(f"{what} has {t.shape[0]} tokens, the plan {plan.T}")
    return _row_strided(t)


def _plan_rows(t, plan, what):
    _2d(t, what)
    if t.shape[0] != plan.row_capacity:
        raise ValueError(f"{what} has {t.shape[0]} rows, the plan {plan.row_capacity}")
    return _row_strided(t)


def _permute(hidden, plan, topk_w, out=None):
    hidden, topk_w = _tokens(hidden, plan, "hidden"), _weights_arg(topk_w, plan)
    code, H = _dtype(hidden, "hidden"), hidden.shape[1]
    out = _out(out, (plan.row_capacity, H), hidden.dtype, hidden.device)
    _b._same_device(hidden, plan.buffer, out, *([] if topk_w is None else [topk_w]))
    _check(lib().moe_permute_tokens(code, hidden.data_ptr(), hidden.stride(0), _p(topk_w), *_plan_args(plan, H),
                                    out.data_ptr(), _stream()), "moe_permute_tokens")
    return out


def _unpermute(rows, plan, topk_w, out=None):
    rows, topk_w = _plan_rows(rows, plan, "rows"), _weights_arg(topk_w, plan)
    code, H = _dtype(rows, "rows"), rows.shape[1]
    out = _out(out, (plan.T, H), rows.dtype, rows.device)
    _b._same_device(rows, plan.buffer, out, *([] if topk_w is None else [topk_w]))
    _check(lib().moe_unpermute_tokens(code, rows.data_ptr(), rows.stride(0), _p(topk_w), *_plan_args(plan, H),
                                      out.data_ptr(), _stream()), "moe_unpermute_tokens")
    return out


def permute_tokens_backward(d_rows, plan, hidden=None, topk_w=None):
    """Gradient of permute_tokens: (d_hidden, d_topk_w). hidden is needed with
    topk_w only; without it d_topk_w is None."""
    d_rows, topk_w = _plan_rows(d_rows, plan, "d_rows"), _weights_arg(topk_w, plan)
    code, H = _dtype(d_rows, "d_rows"), d_rows.shape[1]
    d_hidden = torch.empty(plan.T, H, dtype=d_rows.dtype, device=d_rows.device)
    d_w, ld = None, 0
    tensors = [d_rows, plan.buffer]
    if topk_w is not None:
        if hidden is None:
            raise ValueError("the gradient of topk_w needs hidden")
        hidden = _rows(hidden, d_rows, (plan.T, H), "hidden")
        d_w, ld = torch.empty_like(topk_w), hidden.stride(0)
        tensors += [hidden, topk_w]
    else:
        hidden = None
    _b._same_device(*tensors)
    _check(lib().moe_permute_tokens_backward(code, d_rows.data_ptr(), d_rows.stride(0), _p(hidden), ld, _p(topk_w),
                                             *_plan_args(plan, H), d_hidden.data_ptr(), _p(d_w), _stream()),
           "moe_permute_tokens_backward")
    return d_hidden, d_w


def unpermute_tokens_backward(d_out, plan, rows=None, topk_w=None):
    """Gradient of unpermute_tokens: (d_rows, d_topk_w). rows is needed with
    topk_w only; without it d_topk_w is None. Rows of no slot get zeros."""
    d_out, topk_w = _tokens(d_out, plan, "d_out"), _weights_arg(topk_w, plan)
    code, H = _dtype(d_out, "d_out"), d_out.shape[1]
    d_rows = torch.empty(plan.row_capacity, H, dtype=d_out.dtype, device=d_out.device)
    d_w, ld = None, 0
    tensors = [d_out, plan.buffer]
    if topk_w is not None:
        if rows is None:
            raise ValueError("the gradient of topk_w needs rows")
        rows = _rows(rows, d_out, (plan.row_capacity, H), "rows")
        d_w, ld = torch.empty_like(topk_w), rows.stride(0)
        tensors += [rows, topk_w]
    else:
        rows = None
    _b._same_device(*tensors)
    _check(lib().moe_unpermute_tokens_backward(code, d_out.data_ptr(), d_out.stride(0), _p(rows), ld, _p(topk_w),
                                               *_plan_args(plan, H), d_rows.data_ptr(), _p(d_w), _stream()),
           "moe_unpermute_tokens_backward")
    return d_rows, d_w


class _Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, topk_w, plan):
        ctx.plan = plan
        ctx.save_for_backward(*([] if topk_w is None else [hidden, topk_w]))
        return _permute(hidden, plan, topk_w)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_rows):
        return (*permute_tokens_backward(d_rows, ctx.plan, *ctx.saved_tensors), None)


class _Unpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, topk_w, plan):
        ctx.plan = plan
        ctx.save_for_backward(*([] if topk_w is None else [rows, topk_w]))
        return _unpermute(rows, plan, topk_w)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        return (*unpermute_tokens_backward(d_out, ctx.plan, *ctx.saved_tensors), None)


def _tracked(*ts):
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in ts)


def _no_out(out):
    if out is not None:
        raise ValueError("out cannot be given for inputs that require gradients")


def permute_tokens(hidden, plan, topk_w=None, out=None):
    """Rows of the tokens in the plan's order, [plan.row_capacity, H]:
    rows[inv[t, k]] = topk_w[t, k] * hidden[t] (copies without topk_w), zeros in
    rows of no slot."""
    if _tracked(hidden, topk_w):
        _no_out(out)
        return _Permute.apply(hidden, topk_w, plan)
    return _permute(hidden, plan, topk_w, out)


def unpermute_tokens(rows, plan, topk_w=None, out=None):
    """The way back, [T, H]: out[t] = sum over k, ascending and in fp32, of
    topk_w[t, k] * rows[inv[t, k]]. Rows of no slot are not read."""
    if _tracked(rows, topk_w):
        _no_out(out)
        return _Unpermute.apply(rows, topk_w, plan)
    return _unpermute(rows, plan, topk_w, out)


# --------------------------------------------------------- norms around a block

def _norm_weight(w, x, what):
    if w is None:
        return None
    if w.dim() != 1 or w.shape[0] != x.shape[1]:
        raise ValueError(f"{what} must have the shape ({x.shape[1]},), got {tuple(w.shape)}")
    if w.dtype != x.dtype and w.dtype != torch.float32:
        raise ValueError(f"{what} must be {x.dtype} or float32, got {w.dtype}")
    return w.contiguous()


def _norm_weights(x, weight, next_weight):
    """(weight, next_weight, are they fp32)."""
    weight, next_weight = _norm_weight(weight, x, "weight"), _norm_weight(next_weight, x, "next_weight")
    if weight is not None and next_weight is not None and weight.dtype != next_weight.dtype:
        raise ValueError("weight and next_weight must have one type")
    w = weight if weight is not None else next_weight
    return weight, next_weight, int(w is not None and w.dtype == torch.float32)


def _gate(gate, gate_act, x):
    """(gate, kind, act, row stride)."""
    act = GATE_ACT.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACT)}, got {gate_act!r}")
    if gate is None:
        return None, 0, act, 0
    T, H = x.shape
    if gate.dtype != x.dtype:
        raise ValueError(f"gate must be {x.dtype} like x, got {gate.dtype}")
    if gate.dim() == 1 and gate.shape[0] == H:
        return gate.contiguous(), 1, act, 0
    if gate.dim() == 2 and tuple(gate.shape) == (T, H) and H > 1:
        gate = _row_strided(gate)
        return gate, 3, act, gate.stride(0)
    if gate.dim() == 2 and tuple(gate.shape) == (T, 1):
        gate = gate if gate.stride(0) >= 0 else gate.contiguous()
        return gate, 2, act, gate.stride(0)
    raise ValueError(f"gate must be [H], [T, 1] or [T, H] for x of {tuple(x.shape)}, got {tuple(gate.shape)}")


def _present(*ts):
    return [t for t in ts if t is not None]


def _norm_before(x, weight, eps, w_offset, out=None):
    _2d(x, "x")
    code = _dtype(x, "x")
    x = _row_strided(x)
    weight, _, f32 = _norm_weights(x, weight, None)
    out = _out(out, x.shape, x.dtype, x.device)
    _b._same_device(*_present(x, weight, out))
    T, H = x.shape
    _check(lib().moe_norm_before(code, x.data_ptr(), x.stride(0), _p(weight), f32, w_offset, eps, T, H,
                                 out.data_ptr(), _stream()), "moe_norm_before")
    return out


def _norm_workspace(H, device):
    n = lib().moe_norm_backward_workspace_bytes(H)
    if n == 0:
        raise _b.MoeError(2, "moe_norm_backward_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device), n


def norm_before_backward(dy, x, weight=None, eps=1e-6, weight_offset=0.0, dr=None):
    """Gradient of norm_before: (dx, d_weight); d_weight is None without weight.
    dr, if given, is added to dx: the gradient that reaches x by the residual."""
    _2d(x, "x")
    code = _dtype(x, "x")
    x = _row_strided(x)
    T, H = x.shape
    dy = _rows(dy, x, x.shape, "dy")
    dr = None if dr is None else _rows(dr, x, x.shape, "dr")
    weight, _, f32 = _norm_weights(x, weight, None)
    dx = torch.empty_like(x, memory_format=torch.contiguous_format)
    d_weight = None if weight is None else torch.empty_like(weight)
    _b._same_device(*_present(x, dy, dr, weight))
    ws, n = _norm_workspace(H, x.device)
    _check(lib().moe_norm_before_backward(code, dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0), _p(dr),
                                          0 if dr is None else dr.stride(0), _p(weight), f32, weight_offset, eps, T,
                                          H, dx.data_ptr(), _p(d_weight), ws.data_ptr(), n, _stream()),
           "moe_norm_before_backward")
    return dx, d_weight


def _after_args(x, weight, gate, gate_act, norm, next_weight, next_norm):
    if weight is not None and not norm:
        raise ValueError("weight belongs to the norm of h: norm must be true")
    if next_weight is not None and next_norm is False:
        raise ValueError("next_weight belongs to the next block's norm: next_norm must not be False")
    return (*_norm_weights(x, weight, next_weight), *_gate(gate, gate_act, x))


def _norm_after(x, h, weight, gate, gate_act, alpha, beta, eps, w_offset, norm, next_weight, next_norm, next_eps):
    _2d(x, "x")
    code = _dtype(x, "x")
    x = _row_strided(x)
    h = _rows(h, x, x.shape, "h")
    weight, next_weight, f32, gate, kind, act, ld_gate = _after_args(x, weight, gate, gate_act, norm, next_weight,
                                                                     next_norm)
    T, H = x.shape
    r = torch.empty(T, H, dtype=x.dtype, device=x.device)
    y = torch.empty_like(r) if next_norm else None
    _b._same_device(*_present(x, h, weight, next_weight, gate))
    _check(lib().moe_norm_after(code, x.data_ptr(), x.stride(0), h.data_ptr(), h.stride(0), int(norm), _p(weight),
                                _p(next_weight), f32, w_offset, kind, act, _p(gate), ld_gate, alpha, beta, eps,
                                next_eps, T, H, r.data_ptr(), _p(y), _stream()), "moe_norm_after")
    return (r, y) if next_norm else r


def norm_after_backward(dr, h, weight=None, *, gate=None, gate_act="none", alpha=1.0, beta=1.0, eps=1e-6,
                        weight_offset=0.0, norm=True, dy=None, r=None, next_weight=None, next_eps=None):
    """Gradient of norm_after: (dx, dh, d_weight, d_gate, d_next_weight), None
    for what the forward did not have. dr is the gradient of r; with the next
    norm, dy that of y, and r the forward's result. Without the next norm and
    with beta = 1, dx is dr itself."""
    _2d(h, "h")
    code = _dtype(h, "h")
    h = _row_strided(h)
    T, H = h.shape
    dr = _rows(dr, h, h.shape, "dr")
    if (dy is None) != (r is None):
        raise ValueError("dy and r come together")
    if dy is None and next_weight is not None:
        raise ValueError("next_weight belongs to the next block's norm: dy is missing")
    if dy is not None:
        dy, r = _rows(dy, h, h.shape, "dy"), _rows(r, h, h.shape, "r")
    weight, next_weight, f32, gate, kind, act, ld_gate = _after_args(h, weight, gate, gate_act, norm, next_weight,
                                                                     dy is not None)
    dx = None if dy is None and beta == 1.0 else torch.empty(T, H, dtype=h.dtype, device=h.device)
    dh = torch.empty(T, H, dtype=h.dtype, device=h.device)
    d_weight = None if weight is None else torch.empty_like(weight)
    d_next = None if next_weight is None else torch.empty_like(next_weight)
    d_gate = None if gate is None else torch.empty(gate.shape, dtype=gate.dtype, device=gate.device)
    _b._same_device(*_present(dr, dy, h, r, weight, next_weight, gate))
    ws, n = _norm_workspace(H, h.device)
    _check(lib().moe_norm_after_backward(
        code, dr.data_ptr(), dr.stride(0), _p(dy), 0 if dy is None else dy.stride(0), h.data_ptr(), h.stride(0),
        _p(r), 0 if r is None else r.stride(0), int(norm), _p(weight), _p(next_weight), f32, weight_offset, kind,
        act, _p(gate), ld_gate, alpha, beta, eps, eps if next_eps is None else next_eps, T, H, _p(dx), dh.data_ptr(),
        _p(d_weight), _p(d_gate), _p(d_next), ws.data_ptr(), n, _stream()), "moe_norm_after_backward")
    return dr if dx is None else dx, dh, d_weight, d_gate, d_next


class _NormBefore(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps, w_offset):
        ctx.args = eps, w_offset
        ctx.save_for_backward(x, weight)
        return _norm_before(x, weight, eps, w_offset)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return (*norm_before_backward(dy, *ctx.saved_tensors, *ctx.args), None, None)


class _NormAfter(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, h, weight, gate, next_weight, gate_act, alpha, beta, eps, w_offset, norm, next_norm,
                next_eps):
        ctx.args = dict(gate_act=gate_act, alpha=alpha, beta=beta, eps=eps, weight_offset=w_offset, norm=norm,
                        next_eps=next_eps)
        out = _norm_after(x, h, weight, gate, gate_act, alpha, beta, eps, w_offset, norm, next_weight, next_norm,
                          next_eps)
        ctx.save_for_backward(h, weight, gate, next_weight, out[0] if next_norm else None)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dr, dy=None):
        h, weight, gate, next_weight, r = ctx.saved_tensors
        dx, dh, d_weight, d_gate, d_next = norm_after_backward(dr, h, weight, gate=gate, next_weight=next_weight,
                                                               dy=dy, r=r, **ctx.args)
        return (dx, dh, d_weight, d_gate, d_next) + (None,) * 8


def norm_before(x, weight=None, eps=1e-6, weight_offset=0.0, out=None):
    """y = x * rsqrt(mean(x^2) + eps) * (weight + weight_offset), x [T, H];
    the factor is 1 without weight."""
    if _tracked(x, weight):
        _no_out(out)
        return _NormBefore.apply(x, weight, float(eps), float(weight_offset))
    return _norm_before(x, weight, eps, weight_offset, out)


def norm_after(x, h, weight=None, *, gate=None, gate_act="none", alpha=1.0, beta=1.0, eps=1e-6, weight_offset=0.0,
               norm=True, next_weight=None, next_norm=None, next_eps=None):
    """r = beta * x + alpha * act(gate) * N(h; weight) around a block with the
    residual x and the output h (h itself where norm is false), and with
    next_weight (or next_norm=True) also y = N(r; next_weight), the next block's
    input, from the unrounded r. gate: None, [H], [T, 1] or [T, H]; gate_act:
    "none", "sigmoid" or "tanh". Returns r, or (r, y)."""
    next_norm = next_weight is not None if next_norm is None else bool(next_norm)
    next_eps = eps if next_eps is None else next_eps
    if _tracked(x, h, weight, gate, next_weight):
        return _NormAfter.apply(x, h, weight, gate, next_weight, gate_act, float(alpha), float(beta), float(eps),
                                float(weight_offset), bool(norm), next_norm, float(next_eps))
    return _norm_after(x, h, weight, gate, gate_act, alpha, beta, eps, weight_offset, norm, next_weight, next_norm,
                       next_eps)


# ------------------------------------------------- products with 4-bit weights

class PreparedMatvec:
    """Kernel-layout 4-bit weights made once by moe_matvec_prepare."""

    def __init__(self, fmt, N, K, group, swiglu, scale_dtype, prepared):
        self.fmt, self.N, self.K, self.group, self.swiglu = fmt, N, K, group, swiglu
        self.scale_dtype, self.prepared = scale_dtype, prepared

    @property
    def out_features(self):
        return self.N // 2 if self.swiglu else self.N


def prepare_matvec(weights, swiglu=False):
    """Lay out one matrix [N, K] of 4-bit weights for matvec. weights:
    dict(fmt="fp4", N, K, w, w_scale): codes u8 [N, K/2], UE8M0 u8 [N, K/32],
    one matrix in the format of the experts' FP4 weights; or
    dict(fmt="int4", N, K, group, w, w_scale[, w_zero]): codes u8 [N, K/2],
    scales bf16 or fp16 and zeros u8 [N, ceil(K/group)], weight =
    (code - zero) * scale, zero 8 where w_zero is missing or None. swiglu: rows
    [0, N/2) are gate, [N/2, N) up, and matvec returns silu(gate) * up."""
    fmt, N, K = weights["fmt"], weights["N"], weights["K"]
    if fmt not in QFMT:
        raise ValueError(f"fmt must be 'fp4' or 'int4', got {fmt!r}")
    group = 32 if fmt == "fp4" else weights["group"]
    n = lib().moe_matvec_prepared_bytes(QFMT[fmt], N, K, group, int(swiglu))
    if n == 0:
        raise _b.MoeError(2, "moe_matvec_prepared_bytes")
    w, scale, zero = weights["w"], weights["w_scale"], weights.get("w_zero")
    if w.dtype != torch.uint8 or tuple(w.shape) != (N, K // 2):
        raise ValueError(f"w must be uint8 [{N}, {K // 2}]")
    scale_types = (torch.uint8,) if fmt == "fp4" else (torch.bfloat16, torch.float16)
    groups = math.ceil(K / group)
    if scale.dtype not in scale_types or tuple(scale.shape) != (N, groups):
        raise ValueError(f"w_scale must be {' or '.join(map(str, scale_types))} [{N}, {groups}]")
    if zero is not None and (fmt == "fp4" or zero.dtype != torch.uint8 or tuple(zero.shape) != (N, groups)):
        raise ValueError(f"w_zero must be uint8 [{N}, {groups}], for int4 weights")
    w, scale, zero = w.contiguous(), scale.contiguous(), None if zero is None else zero.contiguous()
    _b._same_device(*_present(w, scale, zero))
    prepared = torch.empty(n, dtype=torch.uint8, device=w.device)
    scale_dtype = 0 if fmt == "fp4" else DTYPES[scale.dtype]
    _check(lib().moe_matvec_prepare(QFMT[fmt], N, K, group, int(swiglu), w.data_ptr(), scale.data_ptr(), scale_dtype,
                                    _p(zero), prepared.data_ptr(), n, _stream()), "moe_matvec_prepare")
    return PreparedMatvec(fmt, N, K, group, bool(swiglu), scale_dtype, prepared)


def matvec(x, prepared, swiglu_limit=None, out=None):
    """x [T, K] bf16 or fp16 times the prepared weights, [T, N] ([T, N/2] with
    SwiGLU) of x's type, for few tokens. Not differentiable."""
    _2d(x, "x")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"matvec takes bfloat16 or float16 x, got {x.dtype}")
    p = prepared
    if x.shape[1] != p.K:
        raise ValueError(f"x has {x.shape[1]} columns, the prepared weights {p.K}")
    if swiglu_limit is not None and not p.swiglu:
        raise ValueError("swiglu_limit is for weights prepared with swiglu=True")
    x = _row_strided(x)
    out = _out(out, (x.shape[0], p.out_features), x.dtype, x.device)
    _b._same_device(x, p.prepared, out)
    _check(lib().moe_matvec(QFMT[p.fmt], p.N, p.K, p.group, int(p.swiglu),
                            _NO_LIMIT if swiglu_limit is None else swiglu_limit, p.scale_dtype,
                            p.prepared.data_ptr(), DTYPES[x.dtype], x.data_ptr(), x.stride(0), x.shape[0],
                            out.data_ptr(), _stream()), "moe_matvec")
    return out


__all__ = ["SortPlan", "sort_layout", "sort_tokens", "permute_tokens", "permute_tokens_backward", "unpermute_tokens",
           "unpermute_tokens_backward", "norm_before", "norm_before_backward", "norm_after", "norm_after_backward",
           "PreparedMatvec", "prepare_matvec", "matvec"]
