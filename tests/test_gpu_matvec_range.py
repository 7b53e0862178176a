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


# the largest of a row's elements is 2^gap times the others and meets zero weights
@pytest.mark.parametrize("gap", [24, 29, 32, 36, 48, 80, 120])
@pytest.mark.parametrize("fmt,group", [("fp4", 32), ("int4", 32), ("int4", 64), ("int4", 128)])
def test_small_activations_beside_a_large_one_that_meets_zeros(fmt, group, gap):
    for T, N, K in ((1, 40, 128), (1, 16, 8192), (5, 33, 544), (12, 300, 1024)):
        g = C.gen(T + N + gap)
        weights = weights_of(g, fmt, N, K, group, -4)
        x = C.randn(g, T, K, dtype=torch.bfloat16)
        zero = 0x00 if fmt == "fp4" else 0x88  # code 8 is zero without zero points
        for k in range(0, K, 256):
            weights["w"][:, k // 2] = zero
            x[::2, k] = 2.0 ** gap
        check(x, weights, M.matvec(x, M.prepare_matvec(weights)))


def test_large_activations_in_a_part_of_one_row():
    """CTAs that share a tile's K range, and passes of tokens, need not agree."""
    for T, N, K, where in ((3, 16, 8192, 0), (3, 16, 8192, 8191), (1, 40, 16384, 5000), (20, 33, 4096, 700)):
        g = C.gen(T + K + where)
        weights = weights_of(g, "fp4", N, K, 32, -4)
        x = C.randn(g, T, K, dtype=torch.bfloat16)
        x[T // 2, where] = 2.0 ** 60
        weights["w"][:, where // 2] = 0
        check(x, weights, M.matvec(x, M.prepare_matvec(weights)))


def test_the_whole_range_of_bf16_in_one_row():
    """Zero weights for all but one magnitude at a time, from the smallest
    subnormal to the largest exponent: that magnitude alone is the result."""
    K, N = 512, 261
    at = torch.arange(N, device="cuda") - 133.0
    x = torch.zeros(2, K, dtype=torch.bfloat16, device="cuda")
    x[:, :N] = (2.0 ** at.double()).to(torch.bfloat16)
    x[1] = -x[1]
    w = torch.zeros(N, K, dtype=torch.uint8, device="cuda")
    w[torch.arange(N), torch.arange(N)] = 2  # e2m1 1.0
    weights = dict(fmt="fp4", N=N, K=K, w=(w[:, 0::2] | (w[:, 1::2] << 4)).contiguous(),
                   w_scale=torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda"))
    out = M.matvec(x, M.prepare_matvec(weights))
    assert torch.equal(out.view(torch.int16), x[:, :N].contiguous().view(torch.int16))


def test_special_values_beside_small_ones():
    """An infinity or a NaN marks its own row only, and small elements beside a
    large one still count where the infinity's weight is zero's sign apart."""
    g = C.gen(5)
    weights = weights_of(g, "fp4", 40, 256, 32, 0)
    weights["w"][:] = 0x22
    x = C.randn(g, 5, 256, dtype=torch.bfloat16).abs()
    x[:, 7] = 2.0 ** 60
    x[0, 3], x[1, 5], x[2, 9] = float("inf"), float("-inf"), float("nan")
    out = M.matvec(x, M.prepare_matvec(weights))
    assert (out[0] == float("inf")).all() and (out[1] == float("-inf")).all() and out[2].isnan().all()
    check(x[3:], weights, out[3:])


@pytest.mark.parametrize("T", [1, 3, 16, 20])
def test_swiglu_keeps_small_activations(T):
    g = C.gen(T)
    weights = weights_of(g, "fp4", 64, 384, 32, -4)
    weights["w"][:, 16] = 0
    x = C.randn(g, T, 384, dtype=torch.bfloat16)
    x[:, 32] = 2.0 ** 50
    W = O.weights_4bit(weights)
    y, mag = O.matvec(x, W), O.matvec(x, W, mag=True)
    gate, up = y.chunk(2, dim=1)
    mg, mu = mag.chunk(2, dim=1)
    s = gate * torch.sigmoid(gate)
    # the slope of silu is below 1.1
    C.check(M.matvec(x, M.prepare_matvec(weights, swiglu=True)), O.swiglu(y),
            1.1 * mg * up.abs() + s.abs() * mu + (s * up).abs(), steps(384))
