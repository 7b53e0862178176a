"""Operators around the experts forward (include/moe_block.h, include/moe_route_fp4.h).

* sort_tokens / permute_tokens / unpermute_tokens: tokens sorted by expert and
  back with the routing weights applied, and their gradients;
* norm_before / norm_after: the norms around a block fused with its gate, the
  residual scale and the next block's norm, and their gradients;
* prepare_matvec / matvec: products of a few tokens with 4-bit weights;
* route_tokens: the router's choice of experts with its weights, and its gradient;
* quantize_fp4 / dequantize_fp4: the FP4 format of the weights and back;
  prepare_matmul_fp4 / matmul_fp4: products of many tokens with FP4 weights and
  activations quantized to FP4 on the way.

As in `binding`, every step runs in the CUDA library on torch's current
stream, and a missing library raises. Arguments are checked and outputs
allocated in csrc/block/calls.cpp: these calls are short at decode, and the
checks in Python would take longer than the kernels. permute_tokens,
unpermute_tokens, norm_before, norm_after and route_tokens take part in autograd (backward
only: forward-mode tangents and tracing are refused); the *_backward functions
are their gradients as plain calls. Rows may be strided
(the elements of a row contiguous); anything else is made contiguous first.
"""
import ctypes
import importlib.machinery
import importlib.util
import os

import torch
from torch.autograd.function import once_differentiable

from . import binding as _b

CALLS_PATH = os.path.join(_b.HERE, "_calls.so")
QFMT = {"fp4": 0, "int4": 1}


class _Calls:
    """The compiled calls, loaded at the first use."""

    def __getattr__(self, name):
        lib = _b.lib()
        if not os.path.exists(CALLS_PATH):
            raise RuntimeError(f"{CALLS_PATH} is missing: build it with block_scaled_moe_expert_gb300.build.build()")
        loader = importlib.machinery.ExtensionFileLoader("_calls", CALLS_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_calls", loader))
        loader.exec_module(module)
        module.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in module.entry_points()}, _b.MoeError)
        global _calls
        _calls = module
        return getattr(module, name)


_calls = _Calls()


def _tracked(*ts):
    for t in ts:
        if t is not None and t.requires_grad:
            return torch.is_grad_enabled()
    return False


def _no_out(out):
    if out is not None:
        raise ValueError("out cannot be given for inputs that require gradients")


# ------------------------------------------------------------ tokens by expert

class SortPlan:
    """Where the T * K slots of a batch go (moe_sort_tokens): group e holds the
    rows offsets[e] .. offsets[e] + counts[e] - 1; inv [T, K] is each slot's
    row (-1 if skipped), row_slot [row_capacity] each row's slot (-1 if none).
    `buffer` starts with the status word that `device_status` reads."""

    __slots__ = ("_plan",)

    def __init__(self, plan):
        self._plan = plan

    buffer = property(lambda self: self._plan.buffer)
    T = property(lambda self: self._plan.T)
    K = property(lambda self: self._plan.K)
    num_experts = property(lambda self: self._plan.E)
    row_align = property(lambda self: self._plan.align)
    row_capacity = property(lambda self: self._plan.row_capacity)
    counts = property(lambda self: self._plan.counts)
    offsets = property(lambda self: self._plan.offsets)
    inv = property(lambda self: self._plan.inv)
    row_slot = property(lambda self: self._plan.row_slot)


def sort_tokens(topk_idx, num_experts, row_align=1):
    """Sort the slots of topk_idx (int32 [T, K], -1 = skipped) by expert, each
    group starting at a multiple of row_align. Returns a SortPlan. An id outside
    [-1, num_experts) counts as skipped and sets MOE_DEV_BAD_EXPERT_ID, which
    device_status(plan.buffer) reads."""
    return SortPlan(_calls.sort_tokens(topk_idx, num_experts, row_align))


def permute_tokens_backward(d_rows, plan, hidden=None, topk_w=None):
    """Gradient of permute_tokens: (d_hidden, d_topk_w). hidden is needed with
    topk_w only; without it d_topk_w is None."""
    return _calls.move_rows_backward(True, d_rows, plan._plan, hidden, topk_w)


def unpermute_tokens_backward(d_out, plan, rows=None, topk_w=None):
    """Gradient of unpermute_tokens: (d_rows, d_topk_w). rows is needed with
    topk_w only; without it d_topk_w is None. Rows of no slot get zeros."""
    return _calls.move_rows_backward(False, d_out, plan._plan, rows, topk_w)


class _Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, topk_w, plan):
        ctx.plan = plan
        ctx.save_for_backward(*([] if topk_w is None else [hidden, topk_w]))
        return _calls.move_rows(True, hidden, plan._plan, topk_w, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_rows):
        return (*permute_tokens_backward(d_rows, ctx.plan, *ctx.saved_tensors), None)


class _Unpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, topk_w, plan):
        ctx.plan = plan
        ctx.save_for_backward(*([] if topk_w is None else [rows, topk_w]))
        return _calls.move_rows(False, rows, plan._plan, topk_w, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        return (*unpermute_tokens_backward(d_out, ctx.plan, *ctx.saved_tensors), None)


def permute_tokens(hidden, plan, topk_w=None, out=None):
    """Rows of the tokens in the plan's order, [plan.row_capacity, H]:
    rows[inv[t, k]] = topk_w[t, k] * hidden[t] (copies without topk_w), zeros in
    rows of no slot."""
    if _tracked(hidden, topk_w):
        _no_out(out)
        return _Permute.apply(hidden, topk_w, plan)
    return _calls.move_rows(True, hidden, plan._plan, topk_w, out)


def unpermute_tokens(rows, plan, topk_w=None, out=None):
    """The way back, [T, H]: out[t] = sum over k, ascending and in fp32, of
    topk_w[t, k] * rows[inv[t, k]]. Rows of no slot are not read."""
    if _tracked(rows, topk_w):
        _no_out(out)
        return _Unpermute.apply(rows, topk_w, plan)
    return _calls.move_rows(False, rows, plan._plan, topk_w, out)


# --------------------------------------------------------- norms around a block

def norm_before_backward(dy, x, weight=None, eps=1e-6, weight_offset=0.0, dr=None):
    """Gradient of norm_before: (dx, d_weight); d_weight is None without weight.
    dr, if given, is added to dx: the gradient that reaches x by the residual."""
    return _calls.norm_before_backward(dy, x, weight, eps, weight_offset, dr)


def norm_after_backward(dr, h, weight=None, *, gate=None, gate_act="none", alpha=1.0, beta=1.0, eps=1e-6,
                        weight_offset=0.0, norm=True, dy=None, r=None, next_weight=None, next_eps=None):
    """Gradient of norm_after: (dx, dh, d_weight, d_gate, d_next_weight), None
    for what the forward did not have. dr is the gradient of r; with the next
    norm, dy that of y, and r the forward's result. Without the next norm and
    with beta = 1, dx is dr itself."""
    return _calls.norm_after_backward(dr, h, weight, gate, gate_act, alpha, beta, eps, weight_offset, norm, dy, r,
                                      next_weight, eps if next_eps is None else next_eps)


class _NormBefore(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, eps, w_offset):
        ctx.args = eps, w_offset
        ctx.save_for_backward(x, weight)
        return _calls.norm_before(x, weight, eps, w_offset, None)

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
        r, y = _calls.norm_after(x, h, weight, gate, gate_act, alpha, beta, eps, w_offset, norm, next_weight,
                                 next_norm, next_eps)
        ctx.save_for_backward(h, weight, gate, next_weight, r if next_norm else None)
        return (r, y) if next_norm else r

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
    return _calls.norm_before(x, weight, eps, weight_offset, out)


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
    r, y = _calls.norm_after(x, h, weight, gate, gate_act, alpha, beta, eps, weight_offset, norm, next_weight,
                             next_norm, next_eps)
    return (r, y) if next_norm else r


# ------------------------------------------------- products with 4-bit weights

class PreparedMatvec:
    """Kernel-layout 4-bit weights made once by moe_matvec_prepare."""

    def __init__(self, fmt, N, K, group, swiglu, weights):
        self.fmt, self.N, self.K, self.group, self.swiglu = fmt, N, K, group, swiglu
        self.out_features = N // 2 if swiglu else N
        self._weights = weights

    prepared = property(lambda self: self._weights.prepared)


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
    made = _calls.prepare_matvec(QFMT[fmt], N, K, group, bool(swiglu), weights["w"], weights["w_scale"],
                                 weights.get("w_zero"))
    return PreparedMatvec(fmt, N, K, group, bool(swiglu), made)


def matvec(x, prepared, swiglu_limit=None, out=None):
    """x [T, K] bf16 or fp16 times the prepared weights, [T, N] ([T, N/2] with
    SwiGLU) of x's type, for few tokens. It has no gradient: an x that requires
    one is refused while gradients are recorded."""
    return _calls.matvec(x, prepared._weights, swiglu_limit, out)


# -------------------------------------------------------------------- routing

def route_tokens_backward(d_topk_w, logits, topk_idx, *, score="softmax", renormalize=True, scale=1.0,
                          d_mean_scores=None):
    """Gradient of route_tokens: d_logits [T, E] of the logits' type, for the
    choice topk_idx. Slots with an id outside [0, E) count for nothing."""
    return _calls.route_tokens_backward(d_topk_w, logits, topk_idx, score, renormalize, scale, d_mean_scores)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, score, bias, num_groups, top_groups, group_score, renormalize, scale, mean_scores):
        ctx.args = dict(score=score, renormalize=renormalize, scale=scale)
        out = _calls.route_tokens(logits, k, score, bias, num_groups, top_groups, group_score, renormalize, scale,
                                  mean_scores)
        ctx.save_for_backward(logits, out[0])
        ctx.mark_non_differentiable(out[0])
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, _, d_w, d_mean=None):
        logits, idx = ctx.saved_tensors
        if d_w is None and d_mean is None:
            return (None,) * 10
        if d_w is None:
            d_w = torch.zeros(idx.shape, dtype=torch.float32, device=idx.device)
        return (route_tokens_backward(d_w, logits, idx, d_mean_scores=d_mean, **ctx.args),) + (None,) * 9


def route_tokens(logits, k, *, score="softmax", bias=None, num_groups=1, top_groups=1, group_score="top2",
                 renormalize=True, scale=1.0, mean_scores=False):
    """The k experts of each token and their weights: (topk_idx int32 [T, k],
    topk_w float32 [T, k]), best first, what experts_forward and sort_tokens take.
    logits [T, E]; score: "softmax" over a token's experts, or "sigmoid" of each.
    bias, float32 [E], is added to the scores for the choice only (a balance bias;
    it has no gradient). With num_groups > 1 the choice is among the experts of the
    top_groups groups of E / num_groups neighbours whose two best ("top2") or best
    ("max") biased scores are largest. topk_w: the scores of the chosen, divided by
    their sum with renormalize, times scale. Ties go to the lowest index; an expert
    with a logit of -inf is never chosen, and slots left over get -1 and weight 0.
    A NaN logit, and +inf under softmax, make the token's weights NaN (and the mean
    scores); scores do not choose its expert.
    mean_scores=True returns also the mean over the tokens of the scores divided by
    their sum, float32 [E]: with the plan's counts, the terms of a balance loss.
    topk_w and the mean scores are differentiable with respect to the logits.
    The results are parts of one storage: keeping or saving one keeps the others' bytes."""
    if _tracked(logits):
        return _Route.apply(logits, k, score, bias, num_groups, top_groups, group_score, renormalize, float(scale),
                            mean_scores)
    return _calls.route_tokens(logits, k, score, bias, num_groups, top_groups, group_score, renormalize, scale,
                               mean_scores)


# --------------------------------------------------------------- the FP4 format

def quantize_fp4(x):
    """(codes uint8 [..., C/2], scale uint8 [..., C/32]) of x [..., C], C a multiple
    of 32: the FP4 format that prepare_weights, prepare_matvec and
    prepare_matmul_fp4 take. A block of 32 gets the scale 2^n, n the smallest with
    amax <= 6 * 2^n, and its elements round to the nearest e2m1 value, ties to even.
    A block with a NaN or an infinity reads as NaN. It has no gradient: an x that
    requires one is refused while gradients are recorded."""
    return _calls.quantize_fp4(x)


def dequantize_fp4(codes, scale, dtype=torch.bfloat16):
    """The values [..., C] that codes and scale of quantize_fp4 stand for, in dtype."""
    return _calls.dequantize_fp4(codes, scale, dtype)


class PreparedMatmulFp4:
    """Kernel-layout FP4 weights made once by moe_matmul_fp4_prepare."""

    def __init__(self, N, K, swiglu, weights):
        self.N, self.K, self.swiglu = N, K, swiglu
        self.out_features = N // 2 if swiglu else N
        self._weights = weights

    prepared = property(lambda self: self._weights.prepared)

    def workspace_bytes(self, T):
        """Bytes of workspace for calls of up to T tokens."""
        return _calls.matmul_fp4_workspace_bytes(self._weights, T)


def prepare_matmul_fp4(weights, swiglu=False):
    """Lay out one matrix [N, K] of FP4 weights for matmul_fp4. weights:
    dict(fmt="fp4", N, K, w, w_scale) as prepare_matvec takes them (codes u8
    [N, K/2], UE8M0 u8 [N, K/32]: what quantize_fp4 returns for the matrix).
    swiglu: rows [0, N/2) are gate, [N/2, N) up, and matmul_fp4 returns
    silu(gate) * up."""
    fmt, N, K = weights["fmt"], weights["N"], weights["K"]
    if fmt != "fp4":
        raise ValueError(f"fmt must be 'fp4', got {fmt!r}")
    made = _calls.prepare_matmul_fp4(N, K, bool(swiglu), weights["w"], weights["w_scale"])
    return PreparedMatmulFp4(N, K, bool(swiglu), made)


def matmul_fp4(x, prepared, swiglu_limit=None, workspace=None, out=None):
    """x [T, K] bf16 or fp16, quantized as quantize_fp4 does, times the prepared
    weights: [T, N] ([T, N/2] with SwiGLU) of x's type, on the FP4 tensor cores.
    matvec takes the same weights with the activations as they are, for few tokens.
    workspace: uint8, at least prepared.workspace_bytes(T), 256-byte aligned
    (allocated if None). device_status(workspace) reads its flags, which say whether
    a wait in the kernel gave up and y is invalid; a call that allocates its own
    leaves no way to read them, and its y may share its storage. It has no gradient:
    an x that requires one is refused while gradients are recorded."""
    return _calls.matmul_fp4(x, prepared._weights, swiglu_limit, workspace, out)


__all__ = ["SortPlan", "sort_tokens", "permute_tokens", "permute_tokens_backward", "unpermute_tokens",
           "unpermute_tokens_backward", "norm_before", "norm_before_backward", "norm_after", "norm_after_backward",
           "PreparedMatvec", "prepare_matvec", "matvec", "route_tokens", "route_tokens_backward", "quantize_fp4",
           "dequantize_fp4", "PreparedMatmulFp4", "prepare_matmul_fp4", "matmul_fp4"]
