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
import functools
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


# The calls below are short at decode, so the checks are written to cost little
# where they pass: one comparison for each property, the message built only on
# a refusal.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _check(status, what):
    if status != 0:
        raise _b.MoeError(status, what)


def _device(t):
    """The current device's index, which t must live on."""
    dev = torch.cuda.current_device() if t.is_cuda else -1
    if t.get_device() != dev:
        _b._same_device(t)
    return dev


def _dtype(t, what):
    code = DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _2d(t, what):
    if t.dim() != 2:
        raise ValueError(f"{what} must be [tokens, width], got {tuple(t.shape)}")


def _rows(t, dtype, shape, dev, what):
    """(tensor, row stride) of an operand [n, H] of the given type with
    contiguous rows."""
    if t.dtype is not dtype:
        raise ValueError(f"{what} must be {dtype} like the rows it goes with, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        _b._same_device(t)
    ld, step = t.stride()
    if step != 1 and shape[1] != 1:
        t = t.contiguous()
        ld = t.stride(0)
    return t, ld


def _first(t, what):
    """(tensor, row stride, dtype code, device, shape): the operand that the
    others have to match."""
    if t.dim() != 2:
        _2d(t, what)
    code = DTYPES.get(t.dtype)
    if code is None:
        _dtype(t, what)
    dev = _device(t)
    shape = t.shape
    ld, step = t.stride()
    if step != 1 and shape[1] != 1:
        t = t.contiguous()
        ld = t.stride(0)
    return t, ld, code, dev, shape


def _out(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.dtype is not dtype or out.shape != shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    _b._same_device(out)
    return out


def _p(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------ tokens by expert

class SortPlan:
    """Where the T * K slots of a batch go (moe_sort_tokens): group e holds the
    rows offsets[e] .. offsets[e] + counts[e] - 1; inv [T, K] is each slot's
    row (-1 if skipped), row_slot [row_capacity] each row's slot (-1 if none).
    `buffer` starts with the status word that `device_status` reads."""

    __slots__ = ("buffer", "T", "num_experts", "K", "row_align", "row_capacity", "_layout", "_args", "_parts")

    def __init__(self, buffer, layout, T, E, K, row_align):
        self.buffer, self._layout, self._parts = buffer, layout, None
        self.T, self.num_experts, self.K, self.row_align = T, E, K, row_align
        self.row_capacity = layout.row_capacity
        self._args = buffer.data_ptr(), layout.total_bytes, T

    def _views(self):
        if self._parts is None:
            self._parts = self.buffer.split_with_sizes(self._layout.split)
        return self._parts

    @property
    def counts(self):
        return self._views()[1][:self.num_experts]

    @property
    def offsets(self):
        return self._views()[2][:self.num_experts + 1]

    @property
    def inv(self):
        return self.buffer.as_strided((self.T, self.K), (self.K, 1), self._layout.inv // 4)

    @property
    def row_slot(self):
        return self._views()[4][:self.row_capacity]


@functools.lru_cache(maxsize=256)
def sort_layout(T, num_experts, K, row_align=1):
    """The plan's layout for these sizes (moe_query_sort_layout)."""
    out = MoeSortLayout()
    _check(lib().moe_query_sort_layout(T, num_experts, K, row_align, _c.byref(out)), "moe_query_sort_layout")
    ends = [out.counts, out.offsets, out.inv, out.row_slot, out.total_bytes]
    out.split = [(e - b) // 4 for b, e in zip([0] + ends, ends)]
    return out


def sort_tokens(topk_idx, num_experts, row_align=1):
    """Sort the slots of topk_idx (int32 [T, K], -1 = skipped) by expert, each
    group starting at a multiple of row_align. Returns a SortPlan. An id outside
    [-1, num_experts) counts as skipped and sets MOE_DEV_BAD_EXPERT_ID, which
    device_status(plan.buffer) reads."""
    if topk_idx.dtype is not torch.int32 or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be an int32 tensor [T, K]")
    dev = _device(topk_idx)
    if not topk_idx.is_contiguous():
        topk_idx = topk_idx.contiguous()
    T, K = topk_idx.shape
    layout = sort_layout(T, num_experts, K, row_align)
    nbytes = layout.total_bytes
    buffer = torch.empty(nbytes // 4, dtype=torch.int32, device=topk_idx.device)
    plan = SortPlan(buffer, layout, T, num_experts, K, row_align)
    _check(lib().moe_sort_tokens(topk_idx.data_ptr(), T, num_experts, K, row_align, plan._args[0], nbytes,
                                 _raw_stream(dev)), "moe_sort_tokens")
    return plan


def _weights_arg(topk_w, plan, dev):
    if topk_w is None:
        return None
    if topk_w.dtype is not torch.float32 or topk_w.shape != (plan.T, plan.K):
        raise ValueError(f"topk_w must be a float32 tensor [{plan.T}, {plan.K}]")
    if topk_w.get_device() != dev:
        _b._same_device(topk_w)
    return topk_w if topk_w.is_contiguous() else topk_w.contiguous()


def _plan_operand(t, plan, n, what):
    """_first of [n, H] rows that go with the plan."""
    first = _first(t, what)
    if first[4][0] != n:
        raise ValueError(f"{what} has {first[4][0]} rows, the plan {n}")
    if plan.buffer.get_device() != first[3]:
        _b._same_device(plan.buffer)
    return first


def _permute(hidden, plan, topk_w, out=None):
    hidden, ld, code, dev, (_, H) = _plan_operand(hidden, plan, plan.T, "hidden")
    topk_w = _weights_arg(topk_w, plan, dev)
    out = _out(out, (plan.row_capacity, H), hidden.dtype, hidden.device)
    _check(lib().moe_permute_tokens(code, hidden.data_ptr(), ld, _p(topk_w), *plan._args, H, plan.num_experts, plan.K,
                                    plan.row_align, out.data_ptr(), _raw_stream(dev)), "moe_permute_tokens")
    return out


def _unpermute(rows, plan, topk_w, out=None):
    rows, ld, code, dev, (_, H) = _plan_operand(rows, plan, plan.row_capacity, "rows")
    topk_w = _weights_arg(topk_w, plan, dev)
    out = _out(out, (plan.T, H), rows.dtype, rows.device)
    _check(lib().moe_unpermute_tokens(code, rows.data_ptr(), ld, _p(topk_w), *plan._args, H, plan.num_experts, plan.K,
                                      plan.row_align, out.data_ptr(), _raw_stream(dev)), "moe_unpermute_tokens")
    return out


def _rows_backward(fn, grad, n_grad, other, n_other, plan, topk_w, out_rows, names):
    """The two gradients differ in which side is rows and which tokens."""
    grad, ld, code, dev, (_, H) = _plan_operand(grad, plan, n_grad, names[0])
    topk_w = _weights_arg(topk_w, plan, dev)
    d_in = torch.empty((out_rows, H), dtype=grad.dtype, device=grad.device)
    d_w, ld_other = None, 0
    if topk_w is None:
        other = None
    elif other is None:
        raise ValueError(f"the gradient of topk_w needs {names[1]}")
    else:
        other, ld_other = _rows(other, grad.dtype, (n_other, H), dev, names[1])
        d_w = torch.empty_like(topk_w)
    _check(getattr(lib(), fn)(code, grad.data_ptr(), ld, _p(other), ld_other, _p(topk_w), *plan._args, H,
                              plan.num_experts, plan.K, plan.row_align, d_in.data_ptr(), _p(d_w), _raw_stream(dev)),
           fn)
    return d_in, d_w


def permute_tokens_backward(d_rows, plan, hidden=None, topk_w=None):
    """Gradient of permute_tokens: (d_hidden, d_topk_w). hidden is needed with
    topk_w only; without it d_topk_w is None."""
    return _rows_backward("moe_permute_tokens_backward", d_rows, plan.row_capacity, hidden, plan.T, plan, topk_w,
                          plan.T, ("d_rows", "hidden"))


def unpermute_tokens_backward(d_out, plan, rows=None, topk_w=None):
    """Gradient of unpermute_tokens: (d_rows, d_topk_w). rows is needed with
    topk_w only; without it d_topk_w is None. Rows of no slot get zeros."""
    return _rows_backward("moe_unpermute_tokens_backward", d_out, plan.T, rows, plan.row_capacity, plan, topk_w,
                          plan.row_capacity, ("d_out", "rows"))


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
    for t in ts:
        if t is not None and t.requires_grad:
            return torch.is_grad_enabled()
    return False


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

def _norm_weight(w, H, dtype, dev, what):
    if w.dim() != 1 or w.shape[0] != H:
        raise ValueError(f"{what} must have the shape ({H},), got {tuple(w.shape)}")
    if w.dtype is not dtype and w.dtype is not torch.float32:
        raise ValueError(f"{what} must be {dtype} or float32, got {w.dtype}")
    if w.get_device() != dev:
        _b._same_device(w)
    return w if w.is_contiguous() else w.contiguous()


def _norm_weights(weight, next_weight, H, dtype, dev):
    """(weight, next_weight, are they fp32)."""
    f32 = 0
    if weight is not None:
        weight = _norm_weight(weight, H, dtype, dev, "weight")
        f32 = int(weight.dtype is torch.float32)
    if next_weight is not None:
        next_weight = _norm_weight(next_weight, H, dtype, dev, "next_weight")
        if weight is not None and next_weight.dtype is not weight.dtype:
            raise ValueError("weight and next_weight must have one type")
        f32 = int(next_weight.dtype is torch.float32)
    return weight, next_weight, f32


def _gate(gate, gate_act, shape, dtype, dev):
    """(gate, kind, act, row stride)."""
    act = GATE_ACT.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACT)}, got {gate_act!r}")
    if gate is None:
        return None, 0, act, 0
    T, H = shape
    if gate.dtype is not dtype:
        raise ValueError(f"gate must be {dtype} like x, got {gate.dtype}")
    if gate.get_device() != dev:
        _b._same_device(gate)
    if gate.dim() == 1 and gate.shape[0] == H:
        return gate.contiguous(), 1, act, 0
    if gate.dim() == 2 and gate.shape == shape and H > 1:
        gate, ld = _rows(gate, dtype, shape, dev, "gate")
        return gate, 3, act, ld
    if gate.dim() == 2 and gate.shape == (T, 1):
        return gate, 2, act, gate.stride(0)
    raise ValueError(f"gate must be [H], [T, 1] or [T, H] for x of {tuple(shape)}, got {tuple(gate.shape)}")


def _norm_before(x, weight, eps, w_offset, out=None):
    x, ld, code, dev, shape = _first(x, "x")
    T, H = shape
    weight, _, f32 = _norm_weights(weight, None, H, x.dtype, dev)
    out = _out(out, shape, x.dtype, x.device)
    _check(lib().moe_norm_before(code, x.data_ptr(), ld, _p(weight), f32, w_offset, eps, T, H, out.data_ptr(),
                                 _raw_stream(dev)), "moe_norm_before")
    return out


def _norm_workspace(H, device):
    n = lib().moe_norm_backward_workspace_bytes(H)
    if n == 0:
        raise _b.MoeError(2, "moe_norm_backward_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device), n


def norm_before_backward(dy, x, weight=None, eps=1e-6, weight_offset=0.0, dr=None):
    """Gradient of norm_before: (dx, d_weight); d_weight is None without weight.
    dr, if given, is added to dx: the gradient that reaches x by the residual."""
    x, ld, code, dev, shape = _first(x, "x")
    T, H = shape
    dy, ld_dy = _rows(dy, x.dtype, shape, dev, "dy")
    ld_dr = 0
    if dr is not None:
        dr, ld_dr = _rows(dr, x.dtype, shape, dev, "dr")
    weight, _, f32 = _norm_weights(weight, None, H, x.dtype, dev)
    dx = torch.empty(shape, dtype=x.dtype, device=x.device)
    d_weight = None if weight is None else torch.empty_like(weight)
    ws, n = _norm_workspace(H, x.device)
    _check(lib().moe_norm_before_backward(code, dy.data_ptr(), ld_dy, x.data_ptr(), ld, _p(dr), ld_dr, _p(weight), f32,
                                          weight_offset, eps, T, H, dx.data_ptr(), _p(d_weight), ws.data_ptr(), n,
                                          _raw_stream(dev)), "moe_norm_before_backward")
    return dx, d_weight


def _norm_after(x, h, weight, gate, gate_act, alpha, beta, eps, w_offset, norm, next_weight, next_norm, next_eps):
    x, ld, code, dev, shape = _first(x, "x")
    T, H = shape
    dtype = x.dtype
    h, ld_h = _rows(h, dtype, shape, dev, "h")
    if weight is not None and not norm:
        raise ValueError("weight belongs to the norm of h: norm must be true")
    if next_weight is not None and not next_norm:
        raise ValueError("next_weight belongs to the next block's norm: next_norm must not be False")
    weight, next_weight, f32 = _norm_weights(weight, next_weight, H, dtype, dev)
    gate, kind, act, ld_gate = _gate(gate, gate_act, shape, dtype, dev)
    r = torch.empty(shape, dtype=dtype, device=x.device)
    y = torch.empty_like(r) if next_norm else None
    _check(lib().moe_norm_after(code, x.data_ptr(), ld, h.data_ptr(), ld_h, int(norm), _p(weight), _p(next_weight),
                                f32, w_offset, kind, act, _p(gate), ld_gate, alpha, beta, eps, next_eps, T, H,
                                r.data_ptr(), _p(y), _raw_stream(dev)), "moe_norm_after")
    return (r, y) if next_norm else r


def norm_after_backward(dr, h, weight=None, *, gate=None, gate_act="none", alpha=1.0, beta=1.0, eps=1e-6,
                        weight_offset=0.0, norm=True, dy=None, r=None, next_weight=None, next_eps=None):
    """Gradient of norm_after: (dx, dh, d_weight, d_gate, d_next_weight), None
    for what the forward did not have. dr is the gradient of r; with the next
    norm, dy that of y, and r the forward's result. Without the next norm and
    with beta = 1, dx is dr itself."""
    h, ld_h, code, dev, shape = _first(h, "h")
    T, H = shape
    dtype, device = h.dtype, h.device
    dr, ld_dr = _rows(dr, dtype, shape, dev, "dr")
    if (dy is None) != (r is None):
        raise ValueError("dy and r come together")
    if weight is not None and not norm:
        raise ValueError("weight belongs to the norm of h: norm must be true")
    ld_dy = ld_r = 0
    if dy is not None:
        dy, ld_dy = _rows(dy, dtype, shape, dev, "dy")
        r, ld_r = _rows(r, dtype, shape, dev, "r")
    elif next_weight is not None:
        raise ValueError("next_weight belongs to the next block's norm: dy is missing")
    weight, next_weight, f32 = _norm_weights(weight, next_weight, H, dtype, dev)
    gate, kind, act, ld_gate = _gate(gate, gate_act, shape, dtype, dev)
    dx = None if dy is None and beta == 1.0 else torch.empty(shape, dtype=dtype, device=device)
    dh = torch.empty(shape, dtype=dtype, device=device)
    d_weight = None if weight is None else torch.empty_like(weight)
    d_next = None if next_weight is None else torch.empty_like(next_weight)
    d_gate = None if gate is None else torch.empty(gate.shape, dtype=dtype, device=device)
    ws, n = _norm_workspace(H, device)
    _check(lib().moe_norm_after_backward(
        code, dr.data_ptr(), ld_dr, _p(dy), ld_dy, h.data_ptr(), ld_h, _p(r), ld_r, int(norm), _p(weight),
        _p(next_weight), f32, weight_offset, kind, act, _p(gate), ld_gate, alpha, beta, eps,
        eps if next_eps is None else next_eps, T, H, _p(dx), dh.data_ptr(), _p(d_weight), _p(d_gate), _p(d_next),
        ws.data_ptr(), n, _raw_stream(dev)), "moe_norm_after_backward")
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
        self.out_features = N // 2 if swiglu else N
        self._args = QFMT[fmt], N, K, group, int(swiglu)


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
    dev = _device(w)
    _b._same_device(scale, *([] if zero is None else [zero]))
    prepared = torch.empty(n, dtype=torch.uint8, device=w.device)
    scale_dtype = 0 if fmt == "fp4" else DTYPES[scale.dtype]
    _check(lib().moe_matvec_prepare(QFMT[fmt], N, K, group, int(swiglu), w.data_ptr(), scale.data_ptr(), scale_dtype,
                                    _p(zero), prepared.data_ptr(), n, _raw_stream(dev)), "moe_matvec_prepare")
    return PreparedMatvec(fmt, N, K, group, bool(swiglu), scale_dtype, prepared)


def matvec(x, prepared, swiglu_limit=None, out=None):
    """x [T, K] bf16 or fp16 times the prepared weights, [T, N] ([T, N/2] with
    SwiGLU) of x's type, for few tokens. Not differentiable."""
    x, ld, code, dev, (T, K) = _first(x, "x")
    if code == 2:
        raise ValueError("matvec takes bfloat16 or float16 x, got torch.float32")
    p = prepared
    if K != p.K:
        raise ValueError(f"x has {K} columns, the prepared weights {p.K}")
    if swiglu_limit is not None and not p.swiglu:
        raise ValueError("swiglu_limit is for weights prepared with swiglu=True")
    if p.prepared.get_device() != dev:
        _b._same_device(p.prepared)
    out = _out(out, (T, p.out_features), x.dtype, x.device)
    _check(lib().moe_matvec(*p._args, _NO_LIMIT if swiglu_limit is None else swiglu_limit, p.scale_dtype,
                            p.prepared.data_ptr(), code, x.data_ptr(), ld, T, out.data_ptr(), _raw_stream(dev)),
           "moe_matvec")
    return out


__all__ = ["SortPlan", "sort_layout", "sort_tokens", "permute_tokens", "permute_tokens_backward", "unpermute_tokens",
           "unpermute_tokens_backward", "norm_before", "norm_before_backward", "norm_after", "norm_after_backward",
           "PreparedMatvec", "prepare_matvec", "matvec"]
