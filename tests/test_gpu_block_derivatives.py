"""GPU: derivatives that the operators do not have are refused, not dropped."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import block_scaled_moe_expert_gb300 as M
from tests import block_cases as C

pytestmark = pytest.mark.gpu


def operands():
    g = C.gen(1)
    x, h = (C.randn(g, 6, 64, dtype=torch.bfloat16) for _ in range(2))
    w = C.randn(g, 64)
    idx = torch.randint(0, 4, (6, 2), generator=g, device="cuda", dtype=torch.int32)
    plan = M.sort_tokens(idx, 4)
    weights = dict(fmt="fp4", N=16, K=64, w=torch.randint(0, 256, (16, 32), generator=g, device="cuda", dtype=torch.uint8),
                   w_scale=torch.full((16, 2), 127, device="cuda", dtype=torch.uint8))
    return x, h, w, plan, torch.rand(6, 2, generator=g, device="cuda"), M.prepare_matvec(weights)


def test_forward_mode_is_refused():
    x, h, w, plan, tw, prepared = operands()
    rows = M.permute_tokens(x, plan)
    with fwd.dual_level():
        def dual(t):
            return fwd.make_dual(t, torch.ones_like(t))
        for call in (lambda: M.norm_before(dual(x), w), lambda: M.norm_before(x, dual(w)),
                     lambda: M.norm_after(dual(x), h), lambda: M.norm_after(x, dual(h)),
                     lambda: M.norm_after(x, h, next_weight=dual(w)), lambda: M.norm_after(x, h, gate=dual(h)),
                     lambda: M.permute_tokens(dual(x), plan), lambda: M.permute_tokens(x, plan, dual(tw)),
                     lambda: M.unpermute_tokens(dual(rows), plan), lambda: M.unpermute_tokens(rows, plan, dual(tw)),
                     lambda: M.norm_before_backward(dual(x), x), lambda: M.norm_after_backward(x, dual(h)),
                     lambda: M.permute_tokens_backward(dual(rows), plan),
                     lambda: M.unpermute_tokens_backward(dual(x), plan), lambda: M.matvec(dual(x), prepared)):
            with pytest.raises(RuntimeError):
                call()
        # what is not a dual tensor is computed as ever
        assert torch.equal(M.permute_tokens(x, plan), rows)
    assert torch.equal(M.permute_tokens(x, plan), rows)


def test_tracing_is_refused():
    """A trace would hold the outputs as memory that nothing fills."""
    x, h, w, plan, tw, prepared = operands()
    rows = M.permute_tokens(x, plan)
    for call, arg in ((lambda t: M.norm_before(t, w) + t, x), (lambda t: M.norm_after(t, h) + t, x),
                      (lambda t: M.permute_tokens(t, plan) + t[:1], x), (lambda t: M.unpermute_tokens(t, plan) + t[:1], rows),
                      (lambda t: M.matvec(t, prepared) + t[:, :16], x),
                      (lambda t: M.sort_tokens(t, 4).inv + t, plan.inv * 0)):
        call(arg)
        with pytest.raises(RuntimeError):
            torch.jit.trace(call, (arg,), check_trace=False)


def test_matvec_of_tracked_activations_is_refused():
    x, _, _, _, _, prepared = operands()
    want = M.matvec(x, prepared)
    x.requires_grad_()
    with pytest.raises(ValueError):
        M.matvec(x, prepared)
    with torch.no_grad():
        assert torch.equal(M.matvec(x, prepared), want)
    assert torch.equal(M.matvec(x.detach(), prepared), want)
