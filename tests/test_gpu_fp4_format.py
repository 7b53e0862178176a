"""GPU: the FP4 format (quantize_fp4, dequantize_fp4), bit for bit against the 64-bit oracle."""
import math

import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from block_scaled_moe_expert_gb300 import workloads as W
from oracle import block as O
from tests import block_cases as C

pytestmark = pytest.mark.gpu


def check(x):
    codes, scale = M.quantize_fp4(x)
    rows = x.reshape(-1, x.shape[-1])
    code, n = O.quantize_fp4(rows)
    got = codes.reshape(rows.shape[0], -1)
    assert codes.dtype == scale.dtype == torch.uint8
    assert codes.shape == (*x.shape[:-1], x.shape[-1] // 2) and scale.shape == (*x.shape[:-1], x.shape[-1] // 32)
    assert torch.equal(got & 15, code[:, 0::2].to(torch.uint8)) and torch.equal(got >> 4, code[:, 1::2].to(torch.uint8))
    assert torch.equal(scale.reshape(n.shape).long(), n + 127)
    for dtype in C.DTYPES:
        back = M.dequantize_fp4(codes, scale, dtype)
        assert back.dtype == dtype and back.shape == x.shape
        assert torch.equal(back.reshape(rows.shape).double(), O.fp4_values(code, n).to(dtype).double())
    return codes, scale


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("R,Cn", [(1, 32), (3, 32), (5, 96), (37, 2880), (128, 4096), (1001, 160), (2, 16384), (70000, 32)])
def test_rows(R, Cn, dtype):
    g = C.gen(R + Cn)
    x = C.randn(g, R, Cn) * torch.exp2(torch.randint(-6, 7, (R, Cn), generator=g, device="cuda").float())
    x[R // 2, : 32] = 0
    check(x.to(dtype))


def test_every_bf16_value_of_a_block():
    """Each finite bf16 beside the blocks' largest: every rounding border, subnormals, both zeros."""
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    check(v[: v.numel() // 32 * 32].view(-1, 32))
    for top in (1.0, 6.0, 6.03125, 7.0, 448.0, 2.0 ** 100, 2.0 ** -120):
        small = v[v.abs() <= top]
        n = small.numel() // 31
        check(torch.cat([torch.full((n, 1), top, device="cuda", dtype=torch.bfloat16), small[: n * 31].view(n, 31)], 1))


def test_borders_in_fp32():
    """Values on the borders between codes and one step beside them, for scales over the whole range."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    one = torch.cat([mid, torch.nextafter(mid, mid * 0), torch.nextafter(mid, mid * 9)])
    row = torch.cat([one, -one[:10], torch.tensor([6.0], device="cuda")])
    rows = torch.stack([row * 2.0 ** n for n in range(-140, 125, 3)])
    check(rows)
    check(torch.full((4, 64), torch.finfo(torch.float32).max, device="cuda"))
    check(torch.full((4, 64), 2.0 ** -149, device="cuda"))


def test_blocks_with_nan_and_infinity_read_as_nan():
    for dtype in C.DTYPES:
        x = C.randn(C.gen(1), 6, 128, dtype=dtype)
        x[0, 5] = math.nan
        x[1, 40] = math.inf
        x[2, 127] = -math.inf
        x[3] = math.nan
        codes, scale = M.quantize_fp4(x)
        bad = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
        bad[0, 0] = bad[1, 1] = bad[2, 3] = True
        bad[3] = True
        assert torch.equal(scale == 255, bad)
        back = M.dequantize_fp4(codes, scale, dtype)
        assert torch.equal(back.isnan(), bad.repeat_interleave(32, 1)) and not bool(back.isinf().any())


def test_shapes_strides_and_alignment():
    x = C.randn(C.gen(2), 4, 33, 64, dtype=torch.bfloat16)
    codes, scale = check(x)
    wide = C.randn(C.gen(3), 50, 96)
    for dtype in C.DTYPES:
        want = M.quantize_fp4(wide.to(dtype))
        for pad, lead in ((32, 0), (8, 8), (1, 0), (5, 3), (16, 4)):
            got = M.quantize_fp4(C.strided(wide.to(dtype), pad, lead))
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        got = M.quantize_fp4(wide.to(dtype).t().contiguous().t())
        assert torch.equal(got[0], want[0])
        same = M.quantize_fp4(wide.to(dtype)[:1].expand(7, 96))
        assert torch.equal(same[0], want[0][:1].expand(7, 48))
    # codes at odd addresses, strided codes, a vector, nothing
    flat = torch.zeros(codes.numel() + 3, dtype=torch.uint8, device="cuda")
    flat[3:] = codes.reshape(-1)
    odd = M.dequantize_fp4(flat[3:].view(codes.shape), scale)
    assert torch.equal(odd, M.dequantize_fp4(codes, scale))
    assert torch.equal(M.dequantize_fp4(codes.transpose(0, 1), scale.transpose(0, 1)), odd.transpose(0, 1))
    check(x[0, 0])
    empty = M.quantize_fp4(x[:, :0])
    assert empty[0].shape == (4, 0, 32) and M.dequantize_fp4(*empty).shape == (4, 0, 64)


def test_it_is_the_format_of_the_weights():
    """The codes of the synthetic checkpoints, and products with what quantize_fp4 makes."""
    wl = W.Workload("fmt", 4, 256, 128, 2, 1, "fp4", "softmax", seed=3)
    weights = W.make_weights(wl, "cuda")
    w13 = M.dequantize_fp4(weights["w13"], weights["w13_scale"], torch.float32)
    codes, scale = M.quantize_fp4(w13)
    assert torch.equal(M.dequantize_fp4(codes, scale, torch.float32), w13)
    x = C.randn(C.gen(4), 3, 256, dtype=torch.bfloat16)
    one = M.prepare_matvec(dict(fmt="fp4", N=256, K=256, w=weights["w13"][1], w_scale=weights["w13_scale"][1]))
    two = M.prepare_matvec(dict(fmt="fp4", N=256, K=256, w=codes[1], w_scale=scale[1]))
    assert torch.equal(M.matvec(x, one), M.matvec(x, two))


def test_large_offsets():
    """More than 2^32 elements: the last rows are those of a small call."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    R = (1 << 32) // 8192 + 3
    x = torch.empty(R, 8192, dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.randn(1, 8192, device="cuda"))
    x[-4:] = torch.randn(4, 8192, device="cuda").bfloat16()
    codes, scale = M.quantize_fp4(x)
    tail = M.quantize_fp4(x[-4:])
    assert torch.equal(codes[-4:], tail[0]) and torch.equal(scale[-4:], tail[1])
    assert torch.equal(codes[1 << 18], codes[0])
    back = M.dequantize_fp4(codes, scale)
    assert torch.equal(back[-4:], M.dequantize_fp4(*tail))
