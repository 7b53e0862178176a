"""GPU: products with 4-bit weights over the whole range of their operands: what
overflows, underflows or disappears beside a larger value only on the way does
not change the result."""
import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from oracle import block as O
from tests import block_cases as C
from tests.test_gpu_matvec import steps

pytestmark = pytest.mark.gpu


def weights_of(g, fmt, N, K, group, scale):
    """Random codes, one scale for all (a power of two)."""
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if fmt == "fp4":
        s = torch.full((N, K // 32), 127 + scale, dtype=torch.uint8, device="cuda")
        return dict(fmt=fmt, N=N, K=K, w=w, w_scale=s)
    s = torch.full((N, -(-K // group)), 2.0 ** scale, dtype=torch.bfloat16, device="cuda")
    return dict(fmt=fmt, N=N, K=K, group=group, w=w, w_scale=s)


def check(x, weights, out):
    """The bound of sums in fp32 over the terms themselves."""
    W = O.weights_4bit(weights)
    C.check(out, O.matvec(x, W), O.matvec(x, W, mag=True), steps(weights["K"]))


# x = normal numbers times 2^at, weights of scale 2^scale: the product is an
# ordinary number, x times the codes alone or the scale's share alone may not be
RANGES = [(121, -20), (125, -125), (118, -60), (-120, 120), (-125, 60), (60, -127), (0, 100), (0, -110)]


@pytest.mark.parametrize("at,scale", RANGES)
@pytest.mark.parametrize("fmt,group", [("fp4", 32), ("int4", 32), ("int4", 128)])
def test_large_activations_meet_small_scales_and_the_other_way(fmt, group, at, scale):
    scale = max(scale, -126) if fmt == "int4" else scale
    for T, N, K in ((1, 40, 512), (5, 33, 288), (11, 48, 1024)):
        g = C.gen(T + at + 1000)
        weights = weights_of(g, fmt, N, K, group, scale)
        x = (torch.randn(T, K, generator=g, device="cuda", dtype=torch.float64).clamp(-3.9, 3.9) * 2.0 ** at).to(torch.bfloat16)
        check(x, weights, M.matvec(x, M.prepare_matvec(weights)))


def test_every_term_is_the_largest():
    """All codes 6, all activations alike: the sum of a group's products is far
    above fp32's range where the scaled sum is not."""
    K = 512
    for at, scale in ((121, -20), (127, -30), (127, -127), (126, -12)):
        weights = dict(fmt="fp4", N=24, K=K, w=torch.full((24, K // 2), 0x77, dtype=torch.uint8, device="cuda"),
                       w_scale=torch.full((24, K // 32), 127 + scale, dtype=torch.uint8, device="cuda"))
        x = torch.full((3, K), 2.0 ** at, dtype=torch.bfloat16, device="cuda")
        check(x, weights, M.matvec(x, M.prepare_matvec(weights)))
    for at, scale in ((118, -30), (127, -126)):
        weights = dict(fmt="int4", N=24, K=K, group=128, w=torch.full((24, K // 2), 0xFF, dtype=torch.uint8, device="cuda"),
                       w_scale=torch.full((24, K // 128), 2.0 ** scale, dtype=torch.bfloat16, device="cuda"),
                       w_zero=torch.zeros(24, K // 128, dtype=torch.uint8, device="cuda"))
        x = torch.full((3, K), 2.0 ** at, dtype=torch.bfloat16, device="cuda")
        check(x, weights, M.matvec(x, M.prepare_matvec(weights)))
