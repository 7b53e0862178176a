"""Shared by the tests of the operators around the experts forward: error
bounds and input makers.

A result held in a type with unit roundoff u, computed in fp32 from terms whose
absolute values add up to `mag` in at most `steps` roundings on any path, is off
by at most u |exact| + steps 2^-24 mag to first order (Higham's bound for sums
in any order), plus half the type's smallest subnormal.
"""
import torch

ROUNDOFF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def bound(exact, mag, steps, dtype):
    # 1.01: terms of second order
    return 1.01 * (ROUNDOFF[dtype] * exact.abs() + steps * 2.0 ** -24 * mag) + TINY[dtype]


def check(out, exact, mag, steps, what=""):
    assert out.shape == exact.shape, (what, out.shape, exact.shape)
    err = (out.double() - exact).abs()
    tol = bound(exact, mag, steps, out.dtype)
    bad = ~(err <= tol)  # a NaN fails
    assert not bad.any(), (what, "worst error / bound", float((err / tol).nan_to_num(nan=1e30).max()),
                           int(bad.sum()), "of", err.numel())


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def strided(t, pad, lead=0):
    """The same values as rows inside a wider buffer, `lead` elements in."""
    T, H = t.shape
    wide = torch.full((T, H + pad + lead), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, lead:lead + H] = t
    return wide[:, lead:lead + H]
