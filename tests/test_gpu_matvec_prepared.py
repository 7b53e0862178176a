"""GPU: matvec directly behind the kernel that lays its weights out."""
import ctypes

import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from block_scaled_moe_expert_gb300 import binding as B
from tests import block_cases as C

pytestmark = pytest.mark.gpu

vp, i64, size_t, c_float = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float


def test_products_right_behind_their_preparation():
    """Two matrices by turns in one prepared buffer, each product enqueued right behind the layout of its
    weights: no product sees the other's. Eagerly and from a graph."""
    L, g, N, K = B.lib(), C.gen(1), 1024, 2880
    L.moe_matvec_prepared_bytes.restype = size_t
    matrices = [M.quantize_fp4(C.randn(g, N, K)) for _ in range(2)]
    n = L.moe_matvec_prepared_bytes(0, N, K, 32, 0)
    prepared = torch.empty(n, dtype=torch.uint8, device="cuda")
    for T in (1, 4, 16, 20):
        x = C.randn(g, T, K, dtype=torch.bfloat16)
        want = [M.matvec(x, M.prepare_matvec(dict(fmt="fp4", N=N, K=K, w=w, w_scale=s))) for w, s in matrices]
        outs = [torch.zeros_like(want[0]) for _ in range(20)]

        def run():
            st = vp(torch.cuda.current_stream().cuda_stream)
            for i, y in enumerate(outs):
                w, s = matrices[i % 2]
                assert L.moe_matvec_prepare(0, N, K, 32, 0, vp(w.data_ptr()), vp(s.data_ptr()), 0, None, vp(prepared.data_ptr()),
                                            size_t(n), st) == 0
                assert L.moe_matvec(0, N, K, 32, 0, c_float(-1), 0, vp(prepared.data_ptr()), 0, vp(x.data_ptr()), i64(K), T,
                                    vp(y.data_ptr()), st) == 0

        run()
        assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(outs))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for _ in range(3):
            for y in outs:
                y.zero_()
            graph.replay()
            assert all(torch.equal(y, want[i % 2]) for i, y in enumerate(outs))
