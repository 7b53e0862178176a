"""GPU: gradients of gates whose activation has saturated."""
import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from oracle import block as O
from tests import block_cases as C
from tests.test_gpu_norms import steps

pytestmark = pytest.mark.gpu

EPS = 1e-6
LOGITS = [0.0, 1.0, -1.0, 4.0, -4.0, 8.0, -8.0, 12.0, -12.0, 16.0, -16.0, 20.0, -20.0, 40.0, -40.0]


def slope_of(logit, act):
    """d act / d logit, without the difference that cancels."""
    v = logit.double().abs()
    e = torch.exp(-v) if act == "sigmoid" else torch.exp(-2 * v)
    return e / (1 + e) ** 2 * (1 if act == "sigmoid" else 4)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["sigmoid", "tanh"])
@pytest.mark.parametrize("kind", ["channel", "token", "element"])
# widths: packs of a warp, of a block, shifted packs, loose rows, rows without a ring, rows read again
@pytest.mark.parametrize("H", [256, 2048, 1001, 5001, 8200])
def test_gradient_of_a_saturated_gate(H, kind, act, dtype):
    T = 30
    g = C.gen(H)
    h, dr = (C.randn(g, T, H, dtype=dtype) for _ in range(2))
    w = C.randn(g, H, dtype=dtype)
    n = {"channel": H, "token": T, "element": T * H}[kind]
    gate = torch.tensor(LOGITS, device="cuda").repeat(-(-n // len(LOGITS)))[:n].to(dtype)
    gate = gate if kind == "channel" else gate.reshape(T, 1 if kind == "token" else H)
    for hh in (h, C.strided(h, 3, 1)):  # the second starts its rows elsewhere
        dgate = M.norm_after_backward(dr, hh, w, gate=gate, gate_act=act, alpha=0.7, eps=EPS)[3]
        full = 0.7 * dr.double() * O.norm(h, w, EPS) * slope_of(gate, act)
        exact, mag = (full, full.abs()) if kind == "element" else \
            (full.sum(0), full.abs().sum(0)) if kind == "channel" else \
            (full.sum(1, keepdim=True), full.abs().sum(1, keepdim=True))
        C.check(dgate, exact, mag, 3 * steps(H, T if kind == "channel" else 1), (kind, act))
