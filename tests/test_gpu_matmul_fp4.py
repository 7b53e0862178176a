"""GPU: products of many tokens with FP4 weights (matmul_fp4) against the 64-bit oracle.

Bounds. Products of e2m1 values are exact. The tensor cores add 64 of them with
their scales at a time into fp32 accumulators, cutting bits off: a step loses at
most 2^-22 of what it adds up, so K / 64 steps and the sums inside them (counted
with 8 more) at most (K / 64 + 8) 2^-22 of the sum of magnitudes, and a split of
K over several CTAs adds fewer than 8 fp32 roundings.
"""
import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from oracle import block as O
from tests import block_cases as C

pytestmark = pytest.mark.gpu


def weights_of(g, N, K, lo=120, hi=124):
    return dict(fmt="fp4", N=N, K=K, w=torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                w_scale=torch.randint(lo, hi, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8))


def steps(K):
    return 4 * (K // 64 + 8) + 8


def dq(x):
    return O.fp4_values(*O.quantize_fp4(x))


def check(x, weights, y):
    Wd = O.weights_4bit(weights)
    q = dq(x)
    C.check(y, O.matvec(q, Wd), O.matvec(q, Wd, mag=True), steps(weights["K"]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (1, 4096, 7168), (3, 17, 160), (4, 255, 256), (16, 256, 2880), (17, 257, 512),
                                   (32, 1000, 4096), (33, 640, 96), (64, 7168, 2048), (65, 129, 1056), (100, 2871, 4096),
                                   (127, 128, 64), (128, 256, 128), (129, 300, 288), (200, 5000, 320), (256, 512, 16384),
                                   (257, 1024, 2880), (700, 2880, 2880), (1001, 333, 608), (2048, 1536, 1024)])
def test_products(T, N, K, dtype):
    g = C.gen(T + N + K)
    weights = weights_of(g, N, K)
    x = C.randn(g, T, K, dtype=dtype)
    check(x, weights, M.matmul_fp4(x, M.prepare_matmul_fp4(weights)))


def test_largest_width():
    g = C.gen(1)
    weights = weights_of(g, 300, 32768)
    for T in (2, 200):
        x = C.randn(g, T, 32768, dtype=torch.bfloat16)
        check(x, weights, M.matmul_fp4(x, M.prepare_matmul_fp4(weights)))


@pytest.mark.parametrize("limit", [None, 0.7])
@pytest.mark.parametrize("T,N,K", [(1, 2, 32), (4, 4096, 7168), (7, 130, 160), (30, 1022, 512), (100, 5760, 2880), (130, 256, 128),
                                   (300, 2050, 1024)])
def test_swiglu(T, N, K, limit):
    """silu(g) u changes with g by at most 1.1 |u| and with u by |silu(g)| <= |g|: the products' errors times these,
    and a dozen roundings of its own."""
    g = C.gen(T + N)
    weights = weights_of(g, N, K)
    x = C.randn(g, T, K, dtype=torch.float16, scale=K ** -0.5)
    y = M.matmul_fp4(x, M.prepare_matmul_fp4(weights, swiglu=True), swiglu_limit=limit)
    Wd, q = O.weights_4bit(weights), dq(x)
    full, mag = O.matvec(q, Wd), O.matvec(q, Wd, mag=True)
    exact = O.swiglu(full, limit)
    e = steps(K) * 2.0 ** -24 * mag
    eg, eu = e.chunk(2, dim=1)
    gate, up = (v.abs() for v in full.chunk(2, dim=1))
    tol = 1.01 * (C.ROUNDOFF[y.dtype] * exact.abs() + 1.1 * eg * (up + eu) + eu * (gate + eg) +
                  16 * 2.0 ** -23 * exact.abs()) + C.TINY[y.dtype]
    assert y.shape == (T, N // 2)
    assert bool(((y.double() - exact).abs() <= tol).all())


def test_quantised_like_quantize_fp4():
    """The same bits as a product of what dequantize_fp4 gives back: quantising that again changes nothing."""
    g = C.gen(3)
    prepared = M.prepare_matmul_fp4(weights_of(g, 384, 1024))
    for T in (5, 300):
        x = C.randn(g, T, 1024, dtype=torch.bfloat16) * torch.exp2(torch.randint(-9, 9, (T, 1024), generator=g, device="cuda").float())
        x = x.bfloat16()
        again = M.dequantize_fp4(*M.quantize_fp4(x))
        assert torch.equal(M.matmul_fp4(x, prepared), M.matmul_fp4(again, prepared))


def test_rows_do_not_depend_on_their_neighbours():
    """Every row of a batch has the bits of the row in other places; those behind the last are left as they were."""
    g = C.gen(4)
    prepared = M.prepare_matmul_fp4(weights_of(g, 500, 672))
    x = C.randn(g, 300, 672, dtype=torch.bfloat16)
    x[7] = float("nan")
    x[290] = float("inf")
    buffer = torch.full((400, 500), 5.0, dtype=torch.bfloat16, device="cuda")
    y = M.matmul_fp4(x, prepared, out=buffer[:300])
    assert y.data_ptr() == buffer.data_ptr() and bool((buffer[300:] == 5.0).all())
    assert torch.equal(y.isnan().all(1), y.isnan().any(1))
    assert y.isnan().any(1).nonzero().flatten().tolist() == [7, 290]
    flipped = M.matmul_fp4(x.flip(0), prepared).flip(0)
    assert torch.equal(y.nan_to_num(9), flipped.nan_to_num(9))


def test_scales_over_the_whole_range():
    g = C.gen(5)
    weights = weights_of(g, 64, 256, 100, 150)
    weights["w_scale"][3, 2] = 255
    x = C.randn(g, 9, 256, dtype=torch.bfloat16)
    x[4] *= 2.0 ** -60
    x[5] *= 2.0 ** 60
    x[6] = 0
    y = M.matmul_fp4(x, M.prepare_matmul_fp4(weights))
    assert bool(y[:, 3].isnan().all())
    weights["w_scale"][3, 2] = 127
    keep = [i for i in range(64) if i != 3]
    Wd, q = O.weights_4bit(weights), dq(x)
    C.check(y[:, keep], O.matvec(q, Wd)[:, keep], O.matvec(q, Wd, mag=True)[:, keep], steps(256))


def test_strides_alignment_and_outputs():
    g = C.gen(6)
    for N in (512, 500, 501):
        prepared = M.prepare_matmul_fp4(weights_of(g, N, 320))
        for T in (6, 150):
            x = C.randn(g, T, 320, dtype=torch.float16)
            want = M.matmul_fp4(x, prepared)
            for pad, lead in ((8, 0), (1, 1), (16, 4)):
                assert torch.equal(M.matmul_fp4(C.strided(x, pad, lead), prepared), want)
            flat = torch.zeros(T * N + 1, dtype=torch.float16, device="cuda")
            M.matmul_fp4(x, prepared, out=flat[1:].view(T, N))  # rows that take no 16-byte stores
            assert torch.equal(flat[1:].view(T, N), want) and float(flat[0]) == 0
            assert torch.equal(M.matmul_fp4(x[:1].expand(T, 320), prepared), want[:1].expand(T, N))
    assert M.matmul_fp4(x[:0], prepared).shape == (0, 501)


def test_workspace_and_status():
    g = C.gen(7)
    prepared = M.prepare_matmul_fp4(weights_of(g, 700, 1000 // 32 * 32))
    x = C.randn(g, 140, 992, dtype=torch.bfloat16)
    ws = torch.full((prepared.workspace_bytes(200),), 255, dtype=torch.uint8, device="cuda")
    want = M.matmul_fp4(x, prepared)
    for T in (140, 3, 64):
        assert torch.equal(M.matmul_fp4(x[:T], prepared, workspace=ws), M.matmul_fp4(x[:T], prepared))
        assert M.device_status(ws) == 0
    with pytest.raises(M.MoeError):
        M.matmul_fp4(x, prepared, workspace=ws[: prepared.workspace_bytes(140) - 1])
    assert torch.equal(M.matmul_fp4(x, prepared, workspace=ws), want)


def test_captured_calls_on_other_streams():
    g = C.gen(8)
    for swiglu, T in ((False, 4), (True, 70), (False, 260)):
        prepared = M.prepare_matmul_fp4(weights_of(g, 1024, 2880), swiglu=swiglu)
        x = C.randn(g, T, 2880, dtype=torch.bfloat16)
        want = M.matmul_fp4(x, prepared)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            assert torch.equal(M.matmul_fp4(x, prepared), want)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = M.matmul_fp4(x, prepared)
        for _ in range(3):
            got.zero_()
            graph.replay()
            assert torch.equal(got, want)
        x.copy_(torch.randn_like(x))
        graph.replay()
        assert torch.equal(got, M.matmul_fp4(x, prepared))


def test_same_bits_every_time():
    g = C.gen(9)
    prepared = M.prepare_matmul_fp4(weights_of(g, 7168, 2048))
    for T in (1, 16, 100, 1000):
        x = C.randn(g, T, 2048, dtype=torch.bfloat16)
        want = M.matmul_fp4(x, prepared)
        for _ in range(20):
            assert torch.equal(M.matmul_fp4(x, prepared), want)


def test_offsets_that_pass_32_bits():
    """y of more than 2^31 elements; the last rows are those of a small call."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g = C.gen(10)
    prepared = M.prepare_matmul_fp4(weights_of(g, 131072, 64))
    x = C.randn(g, 17000, 64, dtype=torch.bfloat16)
    y = M.matmul_fp4(x, prepared)
    assert torch.equal(y[-200:], M.matmul_fp4(x[-200:], prepared))


def test_weights_at_any_address():
    """Checkpoint bytes that start at no 16-byte boundary prepare to the same bytes."""
    g = C.gen(11)
    for swiglu in (False, True):
        weights = weights_of(g, 130, 352)
        want = M.prepare_matmul_fp4(weights, swiglu=swiglu)
        for lead in (1, 8):
            moved = dict(weights)
            for name in ("w", "w_scale"):
                flat = torch.zeros(weights[name].numel() + lead, dtype=torch.uint8, device="cuda")
                flat[lead:] = weights[name].reshape(-1)
                moved[name] = flat[lead:].view(weights[name].shape)
            got = M.prepare_matmul_fp4(moved, swiglu=swiglu)
            assert torch.equal(got.prepared, want.prepared)


def test_bits_of_a_row_in_batches_of_other_sizes():
    """The sums' order goes by the way a batch takes (up to 8, up to 128, more tokens), not by its size."""
    g = C.gen(12)
    for N, K in ((4096, 2048), (300, 4128), (20000, 512)):
        prepared = M.prepare_matmul_fp4(weights_of(g, N, K))
        x = C.randn(g, 520, K, dtype=torch.bfloat16)
        for sizes in ((1, 2, 8), (9, 16, 17, 40, 65, 128), (129, 256, 257, 520)):
            rows = [M.matmul_fp4(x[:T], prepared)[0] for T in sizes]
            assert all(torch.equal(r, rows[0]) for r in rows)


def test_a_clamp_leaves_nan():
    g = C.gen(13)
    weights = weights_of(g, 64, 128)
    weights["w_scale"][5, 1] = weights["w_scale"][32 + 9, 0] = 255  # a gate's row, an up's row
    prepared = M.prepare_matmul_fp4(weights, swiglu=True)
    for T in (3, 30, 150):
        x = C.randn(g, T, 128, dtype=torch.bfloat16)
        x[1] = float("nan")
        y = M.matmul_fp4(x, prepared, swiglu_limit=2.0)
        bad = torch.zeros(T, 32, dtype=torch.bool, device="cuda")
        bad[1] = bad[:, 5] = bad[:, 9] = True
        assert torch.equal(y.isnan(), bad)
