"""GPU: products of a few tokens with 4-bit weights against the 64-bit oracle."""
import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from block_scaled_moe_expert_gb300 import binding as B
from oracle import block as O
from tests import block_cases as C

pytestmark = pytest.mark.gpu


def make_weights(g, fmt, N, K, group=32, zero=False, scale_dtype=torch.bfloat16):
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    G = -(-K // group)
    if fmt == "fp4":
        s = torch.randint(110, 130, (N, G), generator=g, device="cuda", dtype=torch.uint8)
        return dict(fmt=fmt, N=N, K=K, w=w, w_scale=s)
    s = (torch.rand(N, G, generator=g, device="cuda") * 0.02 + 0.001).to(scale_dtype)
    z = torch.randint(0, 16, (N, G), generator=g, device="cuda", dtype=torch.uint8) if zero else None
    return dict(fmt=fmt, N=N, K=K, group=group, w=w, w_scale=s, w_zero=z)


def steps(K):
    # 16 products an instruction, whose adder may cut instead of rounding; the
    # groups' sums one after another; 16 warps and 8 blocks join
    return K // 8 + 64


def check(x, weights, out, swiglu=False, limit=None):
    W = O.weights_4bit(weights)
    y, mag = O.matvec(x, W), O.matvec(x, W, mag=True)
    # x in fp16 after scaling: elements far below the row's largest
    mag = mag + 2.0 ** -14 * x.double().abs().amax(1, keepdim=True) * W.abs().sum(1) / steps(weights["K"])
    if not swiglu:
        C.check(out, y, mag, steps(weights["K"]))
        return
    gate, up = y.chunk(2, dim=1)
    mg, mu = mag.chunk(2, dim=1)
    if limit is not None:
        gate, up = gate.clamp(max=limit), up.clamp(-limit, limit)
    s = gate * torch.sigmoid(gate)
    C.check(out, O.swiglu(y, limit), 1.1 * mg * up.abs() + s.abs() * mu + (s * up).abs(), steps(weights["K"]))


SHAPES = [  # T, N, K
    (1, 1, 32), (1, 16, 128), (2, 17, 160), (1, 64, 7168), (3, 1000, 2880), (1, 4096, 1024), (8, 333, 544),
    (9, 129, 4096), (16, 2050, 256), (17, 40, 96), (40, 77, 1152), (5, 30, 32768), (16, 48, 16416), (1, 60000, 64),
    (2, 36866, 512),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_fp4(T, N, K, dtype):
    g = C.gen(T + N + K)
    weights = make_weights(g, "fp4", N, K)
    x = C.randn(g, T, K, dtype=dtype)
    weights["w_scale"].clamp_(max=119)  # fp16 results stay in range
    check(x, weights, M.matvec(x, M.prepare_matvec(weights)))


@pytest.mark.parametrize("scale_dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zero", [False, True])
def test_int4(group, zero, scale_dtype):
    for T, N, K, dtype in ((1, 50, 96, torch.bfloat16), (7, 2000, 2912, torch.float16), (16, 130, 5152, torch.bfloat16),
                           (1, 9, 32, torch.float16)):
        g = C.gen(T + N + group)
        weights = make_weights(g, "int4", N, K, group, zero, scale_dtype)
        x = C.randn(g, T, K, dtype=dtype)
        check(x, weights, M.matvec(x, M.prepare_matvec(weights)))


@pytest.mark.parametrize("fmt", ["fp4", "int4"])
@pytest.mark.parametrize("T,N,K", [(1, 4096, 7168), (3, 2, 32), (11, 34, 288), (16, 1022, 1024), (20, 258, 640)])
def test_swiglu(T, N, K, fmt):
    g = C.gen(N + K)
    weights = make_weights(g, fmt, N, K, 32, fmt == "int4")
    if fmt == "fp4":
        weights["w_scale"].clamp_(max=120)
    prepared = M.prepare_matvec(weights, swiglu=True)
    x = C.randn(g, T, K, dtype=torch.bfloat16)
    for limit in (None, 0.75):
        check(x, weights, M.matvec(x, prepared, swiglu_limit=limit), True, limit)


def test_every_code_and_scale():
    """One column at a time: each of the 16 codes with each UE8M0 byte, exactly
    (bf16 holds code * 2^n; the smallest scales give bf16 subnormals)."""
    N, K = 256, 512
    codes = torch.arange(K, device="cuda") % 16
    w = (codes[0::2] | (codes[1::2] << 4)).to(torch.uint8).repeat(N, 1)
    scale = torch.arange(256, device="cuda", dtype=torch.uint8)[:, None].repeat(1, K // 32)
    weights = dict(fmt="fp4", N=N, K=K, w=w.contiguous(), w_scale=scale.contiguous())
    x = torch.zeros(16, K, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(16), torch.arange(16) * 33 % K] = 1.0
    out = M.matvec(x, M.prepare_matvec(weights))
    want = O.matvec(x, O.weights_4bit(weights)[:255])
    assert torch.equal(out[:, :255].double(), want.to(torch.float32).to(torch.bfloat16).double())
    assert out[:, 255].isnan().all()  # UE8M0 255


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_special_values_in_x(dtype):
    g = C.gen(8)
    weights = make_weights(g, "fp4", 40, 256)
    weights["w"][:] = 0x22  # every weight is positive
    prepared = M.prepare_matvec(weights)
    x = C.randn(g, 6, 256, dtype=dtype)
    x[0] = 0.0
    x[1, 3], x[2, 7], x[3, 9] = float("inf"), float("-inf"), float("nan")
    out = M.matvec(x, prepared)
    assert (out[0] == 0).all() and (out[1] == float("inf")).all() and (out[2] == float("-inf")).all()
    assert out[3].isnan().all() and out[4:].isfinite().all()
    check(x[4:], weights, out[4:])


def test_bf16_rows_of_any_magnitude():
    """Rows far above and below fp16's range, and elements 2^24 below the
    row's largest, keep their part in the sum."""
    g = C.gen(10)
    weights = make_weights(g, "fp4", 64, 512)
    weights["w_scale"][:] = 127
    x = C.randn(g, 5, 512, dtype=torch.bfloat16)
    x[0] *= 2.0 ** 100
    x[1] *= 2.0 ** -100
    x[2, 1:] *= 2.0 ** -24
    x[3] *= 2.0 ** -130  # bf16 subnormals
    check(x, weights, M.matvec(x, M.prepare_matvec(weights)))
    # the largest element meets a zero weight: the small ones alone remain
    weights["w"][:, 0] = 0
    check(x, weights, M.matvec(x, M.prepare_matvec(weights)))


def test_strides_streams_and_graphs():
    g = C.gen(12)
    weights = make_weights(g, "int4", 1000, 1024, 128, True)
    prepared = M.prepare_matvec(weights)
    x = C.randn(g, 4, 1024, dtype=torch.bfloat16)
    want = M.matvec(x, prepared)
    assert torch.equal(M.matvec(C.strided(x, 7, 3), prepared), want)
    assert torch.equal(M.matvec(x.t().contiguous().t(), prepared), want)
    out = torch.empty_like(want)
    assert M.matvec(x, prepared, out=out) is out and torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = M.matvec(x, prepared)
    side.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = M.matvec(x, prepared)
    got.zero_()
    graph.replay()
    assert torch.equal(got, want)
    assert M.matvec(x[:0], prepared).shape == (0, 1000)


def test_weights_beyond_4_gb():
    """The last rows of a matrix whose byte offsets pass 2^32."""
    N, K, n = 270001, 32768, 37
    g = C.gen(14)
    last = make_weights(g, "fp4", n, K)
    last["w_scale"].clamp_(max=119)
    w = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    scale = torch.full((N, K // 32), 119, dtype=torch.uint8, device="cuda")
    w[-n:], scale[-n:] = last["w"], last["w_scale"]
    assert w.numel() > 2 ** 32
    x = C.randn(g, 2, K, dtype=torch.bfloat16)
    out = M.matvec(x, M.prepare_matvec(dict(fmt="fp4", N=N, K=K, w=w, w_scale=scale)))
    check(x, last, out[:, -n:].contiguous())
    assert int(torch.count_nonzero(out[:, :-n])) == 0


def test_one_matrix_of_the_experts_fp4_weights():
    """The checkpoint layout is that of the experts' FP4 weights."""
    from block_scaled_moe_expert_gb300 import workloads as W
    wl = W.Workload("matvec_fp4", 4, 256, 128, 2, 1, "fp4", "softmax", seed=77)
    ws = W.make_weights(wl, "cuda")
    weights = dict(fmt="fp4", N=256, K=256, w=ws["w13"][1], w_scale=ws["w13_scale"][1])
    x = W.make_hidden(wl, "cuda")
    check(x, weights, M.matvec(x, M.prepare_matvec(weights, swiglu=True)), True)


def test_refusals():
    g = C.gen(1)
    fp4, int4 = make_weights(g, "fp4", 32, 64), make_weights(g, "int4", 32, 64, 64, True)
    x = C.randn(g, 2, 64, dtype=torch.bfloat16)
    for bad in (dict(fp4, fmt="fp8"), dict(fp4, w=fp4["w"][:, 1:]), dict(fp4, w_scale=fp4["w_scale"].float()),
                dict(int4, w_scale=int4["w_scale"].float()), dict(int4, w_zero=int4["w_zero"][:3]),
                dict(fp4, w_zero=fp4["w_scale"])):
        with pytest.raises(ValueError):
            M.prepare_matvec(bad)
    for bad in (dict(fp4, K=48), dict(fp4, N=0), dict(int4, group=16), dict(int4, group=96)):
        with pytest.raises(B.MoeError):
            M.prepare_matvec(bad)
    with pytest.raises(B.MoeError):
        M.prepare_matvec(make_weights(g, "fp4", 33, 64), swiglu=True)
    p = M.prepare_matvec(fp4)
    for bad in (x.float(), x[0], x[:, :32]):
        with pytest.raises(ValueError):
            M.matvec(bad, p)
    with pytest.raises(ValueError):
        M.matvec(x, p, swiglu_limit=1.0)
    with pytest.raises(ValueError):
        M.matvec(x, p, out=torch.empty(2, 31, dtype=x.dtype, device="cuda"))
    with pytest.raises(RuntimeError):
        M.matvec(x.cpu(), p)
