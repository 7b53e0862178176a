"""GPU: routing, the FP4 format and the FP4 products together with the operators around
them, as a block uses them; refusals; calls from two threads and two graphs."""
import ctypes

import pytest
import torch
import torch.autograd.forward_ad as fwd

import block_scaled_moe_expert_gb300 as M
from block_scaled_moe_expert_gb300 import binding as B
from oracle import block as O
from tests import block_cases as C
from tests import parity as P
from tests.test_gpu_block_contexts import buffers, in_two_threads

pytestmark = pytest.mark.gpu

vp, i64, size_t, c_float = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


def checkpoint(seed, E, H, I, shared):
    g = C.gen(seed)
    bf16 = torch.bfloat16
    return dict(w13=C.randn(g, E, 2 * I, H, dtype=bf16, scale=0.05), w2=C.randn(g, E, H, I, dtype=bf16, scale=0.05),
                s13=C.randn(g, 2 * shared, H, dtype=bf16, scale=0.05), s2=C.randn(g, H, shared, dtype=bf16, scale=0.05),
                router=C.randn(g, E, H, scale=H ** -0.5), bias=C.randn(g, E, scale=0.05))


@pytest.mark.parametrize("T", [1, 6, 70, 300])
@pytest.mark.parametrize("activations", ["fp8", "fp4"])
def test_block_from_a_checkpoint(T, activations):
    """Weights quantised here, router, routed experts, shared expert: each step against its oracle
    on the step's own inputs."""
    E, H, I, S, K = 16, 512, 256, 384, 4
    c = checkpoint(1, E, H, I, S)
    w13, w13s = M.quantize_fp4(c["w13"])
    w2, w2s = M.quantize_fp4(c["w2"])
    weights = dict(fmt="fp4", E=E, H=H, I=I, w13=w13, w13_scale=w13s, w2=w2, w2_scale=w2s)
    experts = M.prepare_weights(weights, activations=activations)
    s_in, s_out = (dict(fmt="fp4", N=w.shape[0], K=w.shape[1], **dict(zip(("w", "w_scale"), M.quantize_fp4(w))))
                   for w in (c["s13"], c["s2"]))
    shared_in, shared_out = M.prepare_matmul_fp4(s_in, swiglu=True), M.prepare_matmul_fp4(s_out)
    n = C.randn(C.gen(2), T, H, dtype=torch.bfloat16)
    logits = n.float() @ c["router"].t()
    idx, w = M.route_tokens(logits, K, score="sigmoid", bias=c["bias"], num_groups=4, top_groups=2, scale=2.5)
    chosen = O.choose(logits, K, "sigmoid", c["bias"], 4, 2)
    assert torch.equal(idx.long(), chosen)
    routed = M.experts_forward(n, idx, w, experts)
    assert_close = P.assert_close
    assert_close(routed, P.oracle_out(n, idx, w, weights, None, act_fmt=activations), "experts")
    mid = M.matmul_fp4(n, shared_in)
    h = M.matmul_fp4(mid, shared_out)
    q, Wi = O.fp4_values(*O.quantize_fp4(n)), O.weights_4bit(s_in)
    exact = O.swiglu(O.matvec(q, Wi))
    assert float((mid.double() - exact).norm() / exact.norm()) < 2 ** -8
    q, Wo = O.fp4_values(*O.quantize_fp4(mid)), O.weights_4bit(s_out)
    C.check(h, O.matvec(q, Wo), O.matvec(q, Wo, mag=True), 4 * (S // 64 + 8) + 8)
    x = C.randn(C.gen(3), T, H, dtype=torch.bfloat16)
    r = M.norm_after(x, routed + h)
    assert r.shape == (T, H) and bool(r.isfinite().all())


def test_training_step_through_router_and_experts():
    """Gradients through router, sort, experts and back, with a balance loss, against autograd of the
    same step in 64 bits for the same choice."""
    T, H, E, K = 120, 64, 12, 3
    g = C.gen(4)
    x, target = C.randn(g, T, H), C.randn(g, T, H)
    router, we = C.randn(g, E, H, scale=H ** -0.5), C.randn(g, E, H, H, scale=H ** -0.5)
    for score in ("softmax", "sigmoid"):
        leaves = [t.clone().requires_grad_() for t in (x, router, we)]
        a, r, w = leaves
        idx, tw, mean = M.route_tokens(a @ r.t(), K, score=score, scale=1.5, mean_scores=True)
        plan = M.sort_tokens(idx, E, row_align=8)
        rows = M.permute_tokens(a, plan)
        off = plan.offsets.tolist()
        out = torch.cat([rows[off[e]:off[e + 1]] @ w[e].t() for e in range(E)] + [rows[off[E]:]])
        y = M.unpermute_tokens(out, plan, tw)
        share = plan.counts.float() / (T * K)
        loss = ((y - target) ** 2).mean() + E * (share * mean).sum()
        got = torch.autograd.grad(loss, leaves)

        doubles = [t.detach().double().requires_grad_() for t in (x, router, we)]
        a, r, w = doubles
        logits = a @ r.t()
        s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
        top = s.gather(1, idx.long())
        top = 1.5 * top / top.sum(1, keepdim=True)
        y = torch.einsum("tk,tkh->th", top, torch.einsum("tkih,th->tki", w[idx.long()], a))
        p = (s / s.sum(1, keepdim=True)).mean(0)
        loss = ((y - target.double()) ** 2).mean() + E * (share.double() * p).sum()
        want = torch.autograd.grad(loss, doubles)
        for u, v in zip(got, want):
            assert float((u.double() - v).norm() / v.norm()) < 1e-5


def test_captured_training_step():
    """Forward and backward of the router in a graph. (While an eager graph of the same leaf lives torch itself
    cannot capture a backward pass: the leaf's accumulation is tied to the stream it was made on.)"""
    x = C.randn(C.gen(5), 64, 32).requires_grad_()
    dw = C.randn(C.gen(6), 64, 4)

    def step():
        idx, w, mean = M.route_tokens(x, 4, score="sigmoid", mean_scores=True)
        return torch.autograd.grad([w, mean], [x], [dw, torch.ones_like(mean)])[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    assert torch.equal(got, want)


def test_two_graphs_with_one_workspace_in_turn():
    g = C.gen(7)
    weights = [dict(fmt="fp4", N=N, K=512, **dict(zip(("w", "w_scale"), M.quantize_fp4(C.randn(g, N, 512))))) for N in (256, 700)]
    prepared = [M.prepare_matmul_fp4(w) for w in weights]
    x = [C.randn(g, T, 512, dtype=torch.bfloat16) for T in (40, 200)]
    ws = torch.empty(max(p.workspace_bytes(200) for p in prepared), dtype=torch.uint8, device="cuda")
    want = [M.matmul_fp4(a, p) for a, p in zip(x, prepared)]
    graphs, outs = [], []
    for a, p in zip(x, prepared):
        M.matmul_fp4(a, p, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(M.matmul_fp4(a, p, workspace=ws))
        graphs.append(graph)
    for turn in (0, 1, 1, 0, 1):
        outs[turn].zero_()
        graphs[turn].replay()
        assert torch.equal(outs[turn], want[turn])


def test_calls_back_to_back_see_each_others_results():
    """Chains of dependent calls, whose kernels may start while the one in front ends."""
    g = C.gen(8)
    square = M.prepare_matmul_fp4(dict(fmt="fp4", N=768, K=768, **dict(zip(("w", "w_scale"), M.quantize_fp4(C.randn(g, 768, 768, scale=0.04))))))
    for T in (2, 8, 9, 60, 150):
        x = C.randn(g, T, 768, dtype=torch.bfloat16)
        want = x
        for _ in range(12):
            want = M.matmul_fp4(want, square)
            torch.cuda.synchronize()
        for _ in range(20):
            y = x
            for _ in range(12):
                y = M.matmul_fp4(y, square)
            assert torch.equal(y, want)


def test_products_from_two_threads():
    L, N = B.lib(), 256
    L.moe_matmul_fp4_prepared_bytes.restype = L.moe_matmul_fp4_workspace_bytes.restype = size_t
    for T in ((4, 100), (300, 40)):
        K = (2048, 512)
        prepared = [torch.zeros(L.moe_matmul_fp4_prepared_bytes(N, k, 0), dtype=torch.uint8, device="cuda") for k in K]
        x, y = buffers(300, 2048), buffers(300, N)
        n = L.moe_matmul_fp4_workspace_bytes(300, 2048)
        ws = buffers(n, dtype=torch.uint8)
        assert in_two_threads(lambda s, st: L.moe_matmul_fp4(N, K[s], 0, c_float(-1), vp(prepared[s].data_ptr()), 0,
                                                             vp(x[s].data_ptr()), i64(K[s]), T[s], vp(ws[s].data_ptr()),
                                                             size_t(n), vp(y[s].data_ptr()), st)) == [[], []]


def test_derivatives_that_are_not_there_are_refused():
    g = C.gen(9)
    x, bias = C.randn(g, 6, 64), C.randn(g, 64)
    idx, w = M.route_tokens(x, 4)
    codes, scale = M.quantize_fp4(x)
    prepared = M.prepare_matmul_fp4(dict(fmt="fp4", N=6, K=64, w=codes, w_scale=scale))
    h = x.bfloat16()
    with fwd.dual_level():
        def dual(t):
            return fwd.make_dual(t, torch.ones_like(t))
        for call in (lambda: M.route_tokens(dual(x), 4), lambda: M.route_tokens(x, 4, bias=dual(bias)),
                     lambda: M.route_tokens_backward(dual(w), x, idx), lambda: M.route_tokens_backward(w, dual(x), idx),
                     lambda: M.quantize_fp4(dual(x)), lambda: M.matmul_fp4(dual(h), prepared)):
            with pytest.raises(RuntimeError):
                call()
    for call, arg in ((lambda t: M.route_tokens(t, 4)[1] + t[:, :4], x), (lambda t: M.quantize_fp4(t)[0] + t[:, :32], x),
                      (lambda t: M.matmul_fp4(t, prepared) + t[:, :6], h)):
        call(arg)
        with pytest.raises(RuntimeError):
            torch.jit.trace(call, (arg,), check_trace=False)
    for call, arg in ((lambda t: M.quantize_fp4(t), x.clone().requires_grad_()),
                      (lambda t: M.matmul_fp4(t, prepared), h.clone().requires_grad_())):
        with pytest.raises(ValueError):
            call(arg)
        with torch.no_grad():
            call(arg)


def test_refusals():
    g = C.gen(10)
    x = C.randn(g, 6, 64)
    idx, w = M.route_tokens(x, 4)
    for kw in (dict(score="max"), dict(group_score="sum"), dict(bias=x[0].bfloat16()), dict(bias=x[0, :63])):
        with pytest.raises(ValueError):
            M.route_tokens(x, 4, **kw)
    for k, kw in ((0, {}), (33, {}), (65, {}), (4, dict(num_groups=7)), (4, dict(num_groups=8, top_groups=9)),
                  (9, dict(num_groups=8, top_groups=1)), (4, dict(num_groups=64, top_groups=8))):
        with pytest.raises(M.MoeError):
            M.route_tokens(x, k, **kw)
    with pytest.raises(M.MoeError):
        M.route_tokens(C.randn(g, 2, 513), 4)
    for call in (lambda: M.route_tokens(x.long(), 4), lambda: M.route_tokens_backward(w, x, idx.long()),
                 lambda: M.route_tokens_backward(w[:5], x, idx), lambda: M.route_tokens_backward(w.bfloat16(), x, idx),
                 lambda: M.route_tokens_backward(w, x, idx, d_mean_scores=x[0, :3]),
                 lambda: M.quantize_fp4(x[:, :48]), lambda: M.quantize_fp4(x.double())):
        with pytest.raises(ValueError):
            call()
    codes, scale = M.quantize_fp4(x)
    prepared = M.prepare_matmul_fp4(dict(fmt="fp4", N=6, K=64, w=codes, w_scale=scale))
    h = x.half()
    for call in (lambda: M.matmul_fp4(x, prepared), lambda: M.matmul_fp4(h[:, :32], prepared),
                 lambda: M.matmul_fp4(h, prepared, swiglu_limit=1.0), lambda: M.matmul_fp4(h, prepared, out=x[:, :6]),
                 lambda: M.matmul_fp4(h, prepared, workspace=h), lambda: M.dequantize_fp4(codes, scale[:, :1])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: M.matmul_fp4(h.cpu(), prepared), lambda: M.route_tokens(x, 4, bias=x[0].cpu()),
                 lambda: M.dequantize_fp4(codes, scale.cpu()), lambda: M.matmul_fp4(h, prepared, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
                 lambda: M.prepare_matmul_fp4(dict(fmt="fp4", N=6, K=64, w=codes, w_scale=scale.cpu()))):
        with pytest.raises(RuntimeError):
            call()
    # after all of that the calls work
    assert torch.equal(M.route_tokens(x, 4)[0], idx)


def test_first_calls_of_new_host_threads():
    """Threads whose first call into CUDA encodes the tensor maps of a product."""
    import threading
    g = C.gen(11)
    prepared = M.prepare_matmul_fp4(dict(fmt="fp4", N=64, K=256, **dict(zip(("w", "w_scale"), M.quantize_fp4(C.randn(g, 64, 256))))))
    x = C.randn(g, 300, 256, dtype=torch.bfloat16)
    ws = torch.empty(prepared.workspace_bytes(300), dtype=torch.uint8, device="cuda")
    want = {T: M.matmul_fp4(x[:T], prepared) for T in (2, 40, 300)}
    status, outs = {}, {T: torch.zeros_like(want[T]) for T in want}
    for T in want:
        def call(T=T):
            status[T] = B.lib().moe_matmul_fp4(64, 256, 0, c_float(-1), vp(prepared.prepared.data_ptr()), 0, vp(x.data_ptr()),
                                               i64(256), T, vp(ws.data_ptr()), size_t(ws.numel()), vp(outs[T].data_ptr()), None)
        torch.cuda.synchronize()
        t = threading.Thread(target=call)
        t.start()
        t.join()
        torch.cuda.synchronize()
    assert status == {2: 0, 40: 0, 300: 0}
    assert all(torch.equal(outs[T], want[T]) for T in want)
