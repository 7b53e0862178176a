"""CPU: the 64-bit oracle of the operators around the experts forward, against
closed forms, autograd and differences."""
import math

import pytest
import torch

from oracle import block as O

G = torch.Generator().manual_seed(0)


def randn(*s):
    return torch.randn(*s, generator=G, dtype=torch.float64)


def test_sort_by_hand():
    idx = torch.tensor([[2, 0], [-1, 2], [0, 3], [5, 0]])
    counts, offsets, inv, row_slot = O.sort_tokens(idx, 4, 4)
    assert counts == [3, 0, 2, 1] and offsets == [0, 4, 4, 8, 12]
    assert inv == [4, 0, -1, 5, 1, 8, -1, 2]
    assert row_slot[:12] == [1, 4, 7, -1, 0, 3, -1, -1, 5, -1, -1, -1] and set(row_slot[12:]) <= {-1}
    assert len(row_slot) == O.row_capacity(8, 4, 4) == 20


def test_place_and_gather_are_adjoint():
    """<place(x), y> = <x, gather(y)>, and the dots are the weights' gradient."""
    idx = torch.randint(-1, 5, (30, 3), generator=G)
    inv = torch.tensor(O.sort_tokens(idx, 5, 4)[2]).reshape(30, 3)
    M = O.row_capacity(90, 5, 4)
    x, y, w = randn(30, 7), randn(M, 7), torch.rand(30, 3, generator=G, dtype=torch.float64).requires_grad_()
    left = (O.place(x, w.detach(), inv, M) * y).sum()
    assert torch.allclose(left, (x * O.gather(y, w.detach(), inv)).sum())
    out = torch.zeros(())
    for t in range(30):
        for k in range(3):
            if inv[t, k] >= 0:
                out = out + w[t, k] * (x[t] * y[inv[t, k]]).sum()
    out.backward()
    assert torch.allclose(w.grad, O.dots(x, y, inv)) and torch.allclose(left, out.detach())


@pytest.mark.parametrize("kind,act", [("none", "none"), ("channel", "sigmoid"), ("token", "tanh"),
                                      ("element", "sigmoid"), ("element", "none")])
@pytest.mark.parametrize("has_norm", [True, False])
def test_gradients_of_the_norms(kind, act, has_norm):
    """The written-out gradients against autograd of the forward, and a
    directional difference."""
    T, H = 5, 12
    shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[kind]
    x, h, pr, py = (randn(T, H) for _ in range(4))
    w, nw = randn(H), randn(H)
    gate = None if shape is None else randn(*shape)
    leaves = [t.requires_grad_() for t in (x, h, w, nw) + (() if gate is None else (gate,))]

    def loss():
        r = O.norm_after(x, h, w if has_norm else None, gate, act, 0.7, 1.2, 1e-3, 0.5, has_norm)
        return (r * pr).sum() + (O.norm(r, nw, 2e-3, 0.5) * py).sum(), r

    value, r = loss()
    value.backward()
    with torch.no_grad():
        dx, dh, dw, dg, dn = O.norm_after_backward(pr, h, w if has_norm else None, gate, act, 0.7, 1.2, 1e-3, 0.5,
                                                   has_norm, py, r, nw, 2e-3)
        assert torch.allclose(dx, x.grad) and torch.allclose(dh, h.grad) and torch.allclose(dn, nw.grad)
        assert (dw is None) == (not has_norm) and (dw is None or torch.allclose(dw, w.grad))
        assert (dg is None) == (gate is None) and (dg is None or torch.allclose(dg, gate.grad))
        grads = [x.grad, h.grad, nw.grad] + ([] if gate is None else [gate.grad])
        for t, g in zip([x, h, nw] + ([] if gate is None else [gate]), grads):
            d, step = randn(*t.shape), 1e-5
            t += step * d
            up = loss()[0]
            t -= 2 * step * d
            down = loss()[0]
            t += step * d
            assert abs((up - down) / (2 * step) - (g * d).sum()) < 1e-6 * (1 + (g * d).abs().sum())


@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
def test_slopes_of_saturated_gates(act):
    """Even in the gate, log-linear in its distance from 0 far out, and their own magnitude."""
    v = torch.linspace(0, 60, 241, dtype=torch.float64)
    s = O.gate_slope(v, act)
    assert torch.allclose(s, O.gate_slope(-v, act), rtol=1e-14, atol=0) and (s > 0).all()
    rate = 1 if act == "sigmoid" else 2
    far = v > 20
    assert torch.allclose(s[far].log() + rate * v[far], torch.full_like(v[far], 0.0 if rate == 1 else math.log(4)),
                          atol=1e-8)
    near = v < 3
    g = O.gate_value(v[near], act)
    assert torch.allclose(s[near], g * (1 - g) if act == "sigmoid" else 1 - g * g, rtol=1e-12, atol=0)


def test_norm_of_a_constant_row_and_magnitudes():
    y = O.norm(torch.full((1, 8), -3.0), None, 0.0)
    assert torch.allclose(y, torch.full((1, 8), -1.0, dtype=torch.float64))
    d, v, w = randn(3, 9), randn(3, 9), randn(9)
    exact, mag = O.norm_backward(d, v, w, 1e-6), O.norm_backward(d, v, w, 1e-6, mag=True)
    assert all((e.abs() <= m + 1e-12).all() for e, m in zip(exact, mag))


def test_4bit_weights_by_hand():
    codes = torch.tensor([[0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2], dtype=torch.uint8)
    w = O.weights_4bit(dict(fmt="fp4", N=1, K=32, w=codes, w_scale=torch.tensor([[130]], dtype=torch.uint8)))
    assert w[0, :16].tolist() == [8 * v for v in O.E2M1] and torch.equal(w[0, :16], w[0, 16:])
    nan = O.weights_4bit(dict(fmt="fp4", N=1, K=32, w=codes, w_scale=torch.tensor([[255]], dtype=torch.uint8)))
    assert nan.isnan().all()
    scale = torch.tensor([[0.5]], dtype=torch.bfloat16)
    w = O.weights_4bit(dict(fmt="int4", N=1, K=32, group=64, w=codes, w_scale=scale))
    assert w[0, :16].tolist() == [0.5 * (v - 8) for v in range(16)]
    w = O.weights_4bit(dict(fmt="int4", N=1, K=32, group=64, w=codes, w_scale=scale,
                            w_zero=torch.tensor([[3]], dtype=torch.uint8)))
    assert w[0, :16].tolist() == [0.5 * (v - 3) for v in range(16)]


def test_swiglu_and_its_limit():
    y = torch.tensor([[2.0, -1.0, 3.0, -5.0]], dtype=torch.float64)
    silu = lambda v: v * torch.sigmoid(torch.tensor(v, dtype=torch.float64))  # noqa: E731
    assert torch.allclose(O.swiglu(y), torch.stack([silu(2.0) * 3, silu(-1.0) * -5])[None])
    assert torch.allclose(O.swiglu(y, 1.5), torch.stack([silu(1.5) * 1.5, silu(-1.0) * -1.5])[None])
