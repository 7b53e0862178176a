"""CPU: refusals of the C ABI and of the Python calls of routing, the FP4 format and
the FP4 products, and the oracle's gradient and rounding against other forms."""
import ctypes

import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from block_scaled_moe_expert_gb300 import binding as B
from block_scaled_moe_expert_gb300 import workloads as W
from oracle import block as O

vp, c_int, i64, size_t, c_float = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
INVALID, SHAPE, ALIGNMENT, WORKSPACE = 1, 2, 5, 6
a, odd, f = vp(0x100000), vp(0x100001), c_float(1.0)


@pytest.fixture(scope="module")
def L():
    lib = ctypes.CDLL(B.LIB_PATH)
    for name in ("moe_route_workspace_bytes", "moe_matmul_fp4_prepared_bytes", "moe_matmul_fp4_workspace_bytes"):
        getattr(lib, name).restype = size_t
    return lib


def test_route_refusals(L):
    ws = L.moe_route_workspace_bytes(64)
    assert ws > 0 and L.moe_route_workspace_bytes(0) == 0 and L.moe_route_workspace_bytes(513) == 0

    def route(dtype=0, x=a, ld=64, bias=None, T=4, E=64, K=4, score=0, G=1, top=1, gs=0, idx=a, w=a, mean=None,
              work=None, n=0):
        return L.moe_route_tokens(dtype, x, i64(ld), bias, T, E, K, score, G, top, gs, 1, f, idx, w, mean, work,
                                  size_t(n), None)

    assert route(dtype=3) == INVALID and route(ld=-1) == INVALID and route(score=2) == INVALID and route(gs=-1) == INVALID
    for bad in (dict(T=-1), dict(E=0), dict(E=513), dict(K=0), dict(K=33), dict(E=3, K=4), dict(T=1 << 26, K=2),
                dict(G=0), dict(G=33, E=66), dict(G=5), dict(G=8, top=0), dict(G=8, top=9), dict(G=32, top=1, K=3)):
        assert route(**bad) == SHAPE, bad
    assert route(x=None) == INVALID and route(idx=None) == INVALID and route(w=None) == INVALID
    assert route(mean=a) == INVALID and route(mean=a, work=a, n=ws - 1) == WORKSPACE
    for bad in (dict(x=odd), dict(bias=odd), dict(idx=odd), dict(w=odd), dict(mean=odd, work=a, n=ws),
                dict(mean=a, work=vp(0x100010), n=ws)):
        assert route(**bad) == ALIGNMENT, bad
    assert route(T=0, x=None, idx=None, w=None) == 0

    def back(dtype=0, dw=a, dm=None, x=a, ld=64, idx=a, T=4, E=64, K=4, score=0, dx=a):
        return L.moe_route_tokens_backward(dtype, dw, dm, x, i64(ld), idx, T, E, K, score, 1, f, dx, None)

    assert back(dtype=-1) == INVALID and back(ld=-1) == INVALID and back(score=7) == INVALID
    assert back(E=513) == SHAPE and back(K=33) == SHAPE and back(T=-1) == SHAPE and back(E=3) == SHAPE
    for name in ("dw", "x", "idx", "dx"):
        assert back(**{name: None}) == INVALID and back(**{name: odd}) == ALIGNMENT
    assert back(dm=odd) == ALIGNMENT and back(T=0, dw=None, x=None, idx=None, dx=None) == 0


def test_fp4_refusals(L):
    def quant(dtype=0, x=a, ld=64, R=4, C=64, codes=a, scale=a):
        return L.moe_quantize_fp4(dtype, x, i64(ld), R, C, codes, scale, None)

    assert quant(dtype=3) == INVALID and quant(ld=-1) == INVALID
    for bad in (dict(R=-1), dict(C=0), dict(C=48), dict(C=(1 << 20) + 32)):
        assert quant(**bad) == SHAPE
    for name in ("x", "codes", "scale"):
        assert quant(**{name: None}) == INVALID
    assert quant(x=odd) == ALIGNMENT and quant(codes=vp(0x100008)) == ALIGNMENT and quant(R=0, x=None) == 0

    def back(dtype=0, codes=a, scale=a, R=4, C=64, out=a):
        return L.moe_dequantize_fp4(dtype, codes, scale, R, C, out, None)

    assert back(dtype=3) == INVALID and back(R=-1) == SHAPE and back(C=33) == SHAPE
    for name in ("codes", "scale", "out"):
        assert back(**{name: None}) == INVALID
    assert back(out=odd) == ALIGNMENT and back(R=0, out=None) == 0


def test_matmul_refusals(L):
    bad = [(0, 64, 0), ((1 << 20) + 1, 64, 0), (16, 48, 0), (16, 0, 0), (16, 32800, 0), (15, 64, 1)]
    for shape in bad:
        assert L.moe_matmul_fp4_prepared_bytes(*shape) == 0
        assert L.moe_matmul_fp4_prepare(*shape, a, a, a, size_t(1 << 30), None) == SHAPE
        assert L.moe_matmul_fp4(*shape, f, a, 0, a, i64(64), 4, a, size_t(1 << 30), a, None) == SHAPE
    assert L.moe_matmul_fp4_workspace_bytes(-1, 64) == 0 and L.moe_matmul_fp4_workspace_bytes(4, 33) == 0
    assert L.moe_matmul_fp4_workspace_bytes((1 << 20) + 1, 64) == 0
    sizes = [L.moe_matmul_fp4_workspace_bytes(T, 2880) for T in range(0, 700, 7)]
    assert sizes == sorted(sizes) and sizes[0] >= 4
    need, ws = L.moe_matmul_fp4_prepared_bytes(100, 96, 0), L.moe_matmul_fp4_workspace_bytes(4, 96)
    assert need >= 100 * 96 // 2

    def prepare(codes=a, scale=a, out=a, n=need):
        return L.moe_matmul_fp4_prepare(100, 96, 0, codes, scale, out, size_t(n), None)

    assert prepare(codes=None) == INVALID and prepare(scale=None) == INVALID and prepare(out=None) == INVALID
    assert prepare(n=need - 1) == WORKSPACE and prepare(out=vp(0x100010)) == ALIGNMENT

    def run(prepared=a, dtype=0, x=a, ld=96, T=4, work=a, n=ws, y=a):
        return L.moe_matmul_fp4(100, 96, 0, f, prepared, dtype, x, i64(ld), T, work, size_t(n), y, None)

    assert run(T=-1) == INVALID and run(dtype=2) == INVALID and run(ld=-1) == INVALID and run(T=(1 << 20) + 1) == SHAPE
    for name in ("prepared", "x", "work", "y"):
        assert run(**{name: None}) == INVALID and run(**{name: odd}) == ALIGNMENT
    assert run(n=ws - 1) == WORKSPACE and run(T=0, x=None, y=None, work=None) == 0


def test_python_refusals_without_a_gpu():
    x = torch.zeros(4, 64)
    u8 = torch.zeros(4, 32, dtype=torch.uint8)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: M.route_tokens(x, 2), lambda: M.quantize_fp4(x),
                 lambda: M.dequantize_fp4(u8, torch.zeros(4, 2, dtype=torch.uint8)),
                 lambda: M.route_tokens_backward(torch.zeros(4, 2), x, idx),
                 lambda: M.prepare_matmul_fp4(dict(fmt="fp4", N=4, K=64, w=u8, w_scale=torch.zeros(4, 2, dtype=torch.uint8)))):
        with pytest.raises(RuntimeError):
            call()
    for call in (lambda: M.route_tokens(x[0], 2), lambda: M.route_tokens(x.double(), 2),
                 lambda: M.prepare_matmul_fp4(dict(fmt="int4", N=4, K=64, w=u8, w_scale=u8)),
                 lambda: M.prepare_matmul_fp4(dict(fmt="fp4", N=4, K=64, w=u8, w_scale=u8)),
                 lambda: M.dequantize_fp4(u8, u8), lambda: M.dequantize_fp4(u8[:, :15], u8),
                 lambda: M.dequantize_fp4(u8, u8, torch.int32), lambda: M.quantize_fp4(x.long())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(B.MoeError):
        M.prepare_matmul_fp4(dict(fmt="fp4", N=4, K=48, w=u8, w_scale=u8))


def test_oracle_gradient_is_autograd_of_the_oracle():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 12, generator=g, dtype=torch.float64)
    dw, dm = torch.randn(5, 3, generator=g, dtype=torch.float64), torch.randn(12, generator=g, dtype=torch.float64)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx = O.choose(x, 3, score)
            v = x.clone().requires_grad_()
            s = torch.softmax(v, 1) if score == "softmax" else torch.sigmoid(v)
            w = s.gather(1, idx)
            w = 1.5 * (w / w.sum(1, keepdim=True) if renorm else w)
            loss = (w * dw).sum() + ((s / s.sum(1, keepdim=True)).mean(0) * dm).sum()
            want, = torch.autograd.grad(loss, v)
            got = O.route_backward(dw, x, idx, score, renorm, 1.5, dm)
            assert torch.allclose(got, want, rtol=1e-12, atol=1e-14)
            assert torch.allclose(O.route_weights(x, idx, score, renorm, 1.5), w.detach(), rtol=1e-13)


def test_oracle_choice_by_hand():
    x = torch.tensor([[1.0, 3.0, 3.0, -float("inf"), 2.0, 0.0]])
    assert O.choose(x, 6, "softmax").tolist() == [[1, 2, 4, 0, 5, -1]]
    bias = torch.tensor([9.0, 0.0, 0.5, 50.0, 0.0, -float("inf")])
    assert O.choose(x, 6, "sigmoid", bias).tolist() == [[0, 2, 1, 4, -1, -1]]
    # groups {0, 1}, {2, 3}, {4, 5}: the second has one expert left
    assert O.choose(x, 3, "sigmoid", None, 3, 2, "top2").tolist() == [[1, 4, 0]]
    assert O.choose(x, 3, "sigmoid", None, 3, 2, "max").tolist() == [[1, 2, 0]]


def test_oracle_format_is_the_checkpoints():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(20, 96, generator=g) * torch.exp2(torch.randint(-8, 8, (20, 96), generator=g).float())
    code, n = O.quantize_fp4(x)
    packed, scale = W._fp4_blocks(x)
    assert torch.equal((code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8), packed)
    assert torch.equal((n + 127).to(torch.uint8), scale)


def test_every_declared_symbol_is_exported(L):
    import os
    import re
    path = os.path.join(os.path.dirname(B.HERE), "include", "moe_route_fp4.h")
    names = sorted(set(re.findall(r"^\w[\w\s\*]*?\b(moe_\w+)\s*\(", open(path).read(), flags=re.M)))
    assert len(names) == 9 and "moe_route_tokens" in names and "moe_matmul_fp4" in names
    for n in names:
        getattr(L, n)
