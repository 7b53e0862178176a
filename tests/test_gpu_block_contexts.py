"""GPU: the C ABI from several contexts and host threads of one process: what a
call sets up for its own launch does not fail another's."""
import ctypes
import subprocess
import sys
import threading

import pytest
import torch

from block_scaled_moe_expert_gb300 import binding as B

pytestmark = pytest.mark.gpu

vp, c_int, i64, size_t, c_float = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float

TWO_CONTEXTS = """
import ctypes, sys
cu, L = ctypes.CDLL("libcuda.so.1"), ctypes.CDLL(sys.argv[1])
vp = ctypes.c_void_p
def ok(r):
    assert r == 0, r
class Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("total", "status", "counts", "offsets", "inv", "row_slot")] + [("rows", ctypes.c_int32)]
T, E, K = 8192, 16, 4
lay = Layout()
ok(L.moe_query_sort_layout(T, E, K, 1, ctypes.byref(lay)))
ok(cu.cuInit(0))
host = (ctypes.c_int32 * (T * K))(*[i % E for i in range(T * K)])
for turn in range(2):
    ctx, idx, plan = vp(), vp(), vp()
    ok(cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0))
    ok(cu.cuMemAlloc_v2(ctypes.byref(idx), ctypes.c_size_t(4 * T * K)))
    ok(cu.cuMemAlloc_v2(ctypes.byref(plan), ctypes.c_size_t(lay.total)))
    ok(cu.cuMemcpyHtoD_v2(idx, host, ctypes.c_size_t(4 * T * K)))
    st = L.moe_sort_tokens(idx, T, E, K, 1, plan, ctypes.c_size_t(lay.total), None)
    ok(cu.cuCtxSynchronize())
    print("context", turn, "status", st)
    assert st == 0
    counts = (ctypes.c_int32 * E)()
    ok(cu.cuMemcpyDtoH_v2(counts, vp(plan.value + lay.counts), ctypes.c_size_t(4 * E)))
    assert list(counts) == [T * K // E] * E
"""


def test_large_sorts_in_a_second_context():
    """Launch limits belong to a context: each one has its own."""
    r = subprocess.run([sys.executable, "-c", TWO_CONTEXTS, B.LIB_PATH], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="one device")
def test_large_sorts_on_a_second_device():
    import block_scaled_moe_expert_gb300 as M
    for dev in range(2):
        with torch.cuda.device(dev):
            idx = (torch.arange(20000 * 7, dtype=torch.int32, device="cuda") % 60).reshape(20000, 7)
            assert M.sort_tokens(idx, 60).counts.tolist() == [-(-(140000 - e) // 60) for e in range(60)]


def in_two_threads(call):
    """call(side, stream) from two host threads at once, each on its own
    stream; the statuses that were not MOE_OK."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    refused, start = [[], []], threading.Barrier(2)

    def work(side):
        start.wait()
        for _ in range(4000):
            st = call(side, vp(streams[side].cuda_stream))
            if st:
                refused[side].append(st)

    threads = [threading.Thread(target=work, args=(s,)) for s in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return refused


def buffers(*shape, dtype=torch.bfloat16):
    return [torch.zeros(*shape, dtype=dtype, device="cuda") for _ in range(2)]


def test_norms_of_two_widths():
    L, T = B.lib(), 4
    x, y = buffers(T, 8192), buffers(T, 8192)
    H = (8192, 5504)
    assert in_two_threads(lambda s, st: L.moe_norm_before(0, vp(x[s].data_ptr()), i64(H[s]), None, 0, c_float(0), c_float(1e-6),
                                                          T, H[s], vp(y[s].data_ptr()), st)) == [[], []]


def test_norm_gradients_of_two_widths():
    L, T = B.lib(), 4
    L.moe_norm_backward_workspace_bytes.restype = size_t
    for H in ((8192, 5504), (16384, 12288)):  # the second without a ring, for its column sums
        x, dy, dx = buffers(T, H[0]), buffers(T, H[0]), buffers(T, H[0])
        w, dw = buffers(H[0]), buffers(H[0])
        n = L.moe_norm_backward_workspace_bytes(H[0])
        ws = buffers(n, dtype=torch.uint8)
        p = lambda t, s: vp(t[s].data_ptr())  # noqa: E731
        assert in_two_threads(lambda s, st: L.moe_norm_before_backward(
            0, p(dy, s), i64(H[s]), p(x, s), i64(H[s]), None, i64(0), p(w, s), 0, c_float(0), c_float(1e-6), T, H[s],
            p(dx, s), p(dw, s), p(ws, s), size_t(n), st)) == [[], []]


def test_products_of_two_depths():
    L, N = B.lib(), 256
    K = (8192, 1024)
    L.moe_matvec_prepared_bytes.restype = size_t
    prepared = [torch.zeros(L.moe_matvec_prepared_bytes(0, N, k, 32, 0), dtype=torch.uint8, device="cuda") for k in K]
    x, y = buffers(4, 8192), buffers(4, N)
    assert in_two_threads(lambda s, st: L.moe_matvec(0, N, K[s], 32, 0, c_float(-1), 0, vp(prepared[s].data_ptr()), 0,
                                                     vp(x[s].data_ptr()), i64(K[s]), 4, vp(y[s].data_ptr()), st)) == [[], []]


def test_sorts_over_two_numbers_of_experts():
    L, T, K = B.lib(), 1024, 2
    E = (512, 400)
    idx = buffers(T, K, dtype=torch.int32)
    n = 1 << 20
    plan = buffers(n, dtype=torch.uint8)
    assert in_two_threads(lambda s, st: L.moe_sort_tokens(vp(idx[s].data_ptr()), T, E[s], K, 1, vp(plan[s].data_ptr()),
                                                          size_t(n), st)) == [[], []]
