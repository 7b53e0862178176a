"""CPU: the operators around the experts forward export what their header
declares, size their buffers and refuse bad arguments without a GPU."""
import ctypes
import os
import re

import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from block_scaled_moe_expert_gb300 import binding as B
from block_scaled_moe_expert_gb300 import build as BLD
from oracle import block as O

vp, c_int, c_float, i64, size_t = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64, ctypes.c_size_t

INVALID, SHAPE, ALIGNMENT, WORKSPACE = 1, 2, 5, 6


class SortLayout(ctypes.Structure):
    _fields_ = [("total_bytes", size_t), ("status", size_t), ("counts", size_t), ("offsets", size_t),
                ("inv", size_t), ("row_slot", size_t), ("row_capacity", ctypes.c_int32)]


@pytest.fixture(scope="module")
def L():
    BLD.build()
    B._lib = None
    return B.lib()


def header_names():
    src = open(os.path.join(BLD.INCLUDE, "moe_block.h")).read()
    return sorted(set(re.findall(r"^\w[\w\s\*]*?\b(moe_\w+)\s*\(", src, flags=re.M)))


def test_every_declared_symbol_is_exported(L):
    names = header_names()
    assert len(names) == 14 and "moe_sort_tokens" in names and "moe_matvec" in names
    for n in names:
        assert hasattr(L, n), n


def sort_layout(L, T, E, K, align):
    out = SortLayout()
    return L.moe_query_sort_layout(T, E, K, align, ctypes.byref(out)), out


@pytest.mark.parametrize("T,E,K,align", [(0, 8, 2, 16), (1, 1, 1, 1), (4, 256, 8, 128), (8192, 512, 32, 256),
                                         (1000, 60, 7, 3)])
def test_sort_layout(L, T, E, K, align):
    st, lay = sort_layout(L, T, E, K, align)
    assert st == 0
    S = T * K
    assert lay.row_capacity == O.row_capacity(S, E, align) and lay.row_capacity % align == 0
    ends = [(lay.status, 4), (lay.counts, 4 * E), (lay.offsets, 4 * (E + 1)), (lay.inv, 4 * S),
            (lay.row_slot, 4 * lay.row_capacity)]
    at = 0
    for off, n in ends:
        assert off >= at and off % 256 == 0
        at = off + n
    assert at <= lay.total_bytes


@pytest.mark.parametrize("T,E,K,align", [(-1, 8, 2, 1), (1, 0, 2, 1), (1, 513, 2, 1), (1, 8, 0, 1), (1, 8, 33, 1),
                                         (1, 8, 2, 0), (1, 8, 2, 257), (1 << 25, 8, 4, 1)])
def test_unsupported_sorts_are_refused(L, T, E, K, align):
    assert sort_layout(L, T, E, K, align)[0] == SHAPE
    assert L.moe_sort_tokens(None, T, E, K, align, None, size_t(0), None) == SHAPE


def test_row_moves_check_arguments_before_the_device(L):
    a, odd = vp(0x100000), vp(0x100001)
    big = size_t(1 << 40)
    st, lay = sort_layout(L, 4, 8, 2, 16)

    def permute(dtype=0, hidden=a, ld=64, w=None, plan=a, nbytes=big, T=4, H=64, rows=a):
        return L.moe_permute_tokens(dtype, hidden, i64(ld), w, plan, nbytes, T, H, 8, 2, 16, rows, None)

    assert permute(dtype=3) == INVALID and permute(ld=-1) == INVALID
    assert permute(H=0) == SHAPE and permute(H=65537) == SHAPE and permute(T=-1) == SHAPE
    assert permute(hidden=None) == INVALID and permute(plan=None) == INVALID and permute(rows=None) == INVALID
    assert permute(nbytes=size_t(lay.total_bytes - 1)) == WORKSPACE
    assert permute(hidden=odd) == ALIGNMENT and permute(rows=odd) == ALIGNMENT and permute(plan=vp(0x100080)) == ALIGNMENT
    assert permute(T=0, hidden=None, plan=None, rows=None) == 0
    # with weights their gradient and the other operand are needed
    assert L.moe_unpermute_tokens_backward(0, a, i64(64), None, i64(64), a, a, big, 4, 64, 8, 2, 16, a, a, None) == INVALID
    assert L.moe_permute_tokens_backward(0, a, i64(64), a, i64(64), a, a, big, 4, 64, 8, 2, 16, a, None, None) == INVALID
    assert L.moe_unpermute_tokens(0, odd, i64(64), None, a, big, 4, 64, 8, 2, 16, a, None) == ALIGNMENT


def test_norms_check_arguments_before_the_device(L):
    a, odd, f = vp(0x100000), vp(0x100001), c_float(1e-6)
    L.moe_norm_backward_workspace_bytes.restype = size_t
    ws = L.moe_norm_backward_workspace_bytes(64)
    assert ws > 0 and L.moe_norm_backward_workspace_bytes(16385) == 0 and L.moe_norm_backward_workspace_bytes(0) == 0

    def before(dtype=0, x=a, ld=64, w=None, T=4, H=64, y=a):
        return L.moe_norm_before(dtype, x, i64(ld), w, 0, f, f, T, H, y, None)

    assert before(dtype=-1) == INVALID and before(ld=-2) == INVALID and before(x=None) == INVALID
    assert before(H=16385) == SHAPE and before(T=-1) == SHAPE and before(T=0, x=None, y=None) == 0
    assert before(x=odd) == ALIGNMENT and before(w=odd) == ALIGNMENT and before(y=odd) == ALIGNMENT

    def after(h=a, norm=1, w=None, nw=None, kind=0, act=0, gate=None, y=None, r=a):
        return L.moe_norm_after(0, a, i64(64), h, i64(64), norm, w, nw, 0, f, kind, act, gate, i64(64), f, f, f, f, 4,
                                64, r, y, None)

    assert after(h=None) == INVALID and after(r=None) == INVALID
    assert after(norm=0, w=a) == INVALID and after(nw=a) == INVALID        # a weight without its norm
    assert after(kind=1) == INVALID and after(gate=a) == INVALID           # a gate and its kind come together
    assert after(kind=4, gate=a) == INVALID and after(kind=1, gate=a, act=3) == INVALID
    assert after(kind=1, gate=odd) == ALIGNMENT

    def back(dr=a, dy=None, r=None, w=None, dw=None, kind=0, gate=None, dgate=None, work=a, nbytes=ws, T=4):
        return L.moe_norm_after_backward(0, dr, i64(64), dy, i64(64), a, i64(64), r, i64(64), 1, w, None, 0, f, kind, 0,
                                         gate, i64(64), f, f, f, f, T, 64, a, a, dw, dgate, None, work,
                                         size_t(nbytes), None)

    assert back(dr=None) == INVALID and back(dy=a) == INVALID and back(w=a) == INVALID and back(dw=a) == INVALID
    assert back(kind=1, gate=a) == INVALID and back(work=None) == INVALID and back(nbytes=ws - 1) == WORKSPACE
    assert back(T=0) == 0
    assert L.moe_norm_before_backward(0, a, i64(64), a, i64(64), None, i64(0), a, 0, f, f, 4, 64, a, None, a,
                                      size_t(ws), None) == INVALID


def test_gradient_without_tokens_checks_the_channel_gate(L):
    """Its d_gate is written for no tokens too, and the kernel reads the gate."""
    a, odd, f = vp(0x100000), vp(0x100001), c_float(1e-6)
    L.moe_norm_backward_workspace_bytes.restype = size_t
    ws = L.moe_norm_backward_workspace_bytes(64)

    def back(kind, gate, act=0, dgate=a, T=0):
        return L.moe_norm_after_backward(0, None, i64(64), None, i64(64), None, i64(64), None, i64(64), 1, None, None, 0, f,
                                         kind, act, gate, i64(64), f, f, f, f, T, 64, None, None, None, dgate, None, a,
                                         size_t(ws), None)

    assert back(1, None) == INVALID and back(1, odd) == ALIGNMENT
    assert back(1, a, dgate=None) == INVALID and back(1, a, dgate=odd) == ALIGNMENT
    for act in (-1, 3):
        assert back(1, a, act=act) == INVALID and back(2, None, act=act) == INVALID
    for kind in (-1, 4):
        assert back(kind, None) == INVALID and back(kind, a) == INVALID
    # gates of no elements have nothing to check
    assert back(2, None, dgate=None) == 0 and back(3, None, dgate=None) == 0 and back(0, None, dgate=None) == 0


def test_matvec_sizes_and_refusals(L):
    L.moe_matvec_prepared_bytes.restype = size_t
    for fmt, N, K, group, swiglu in [(0, 4096, 7168, 32, 1), (0, 17, 160, 32, 0), (1, 1000, 2880, 128, 0),
                                     (1, 34, 32, 64, 1)]:
        n = L.moe_matvec_prepared_bytes(fmt, N, K, group, swiglu)
        rows = -(-N // 16) * 16 if not swiglu else -(-(N // 2) // 8) * 16
        cols = -(-K // 128) * 128
        scale = 1 if fmt == 0 else 4
        assert n == rows * cols // 2 + rows * (cols // group) * scale
    for bad in [(2, 16, 64, 32, 0), (0, 0, 64, 32, 0), (0, 16, 48, 32, 0), (0, 16, 64, 64, 0), (1, 16, 64, 16, 0),
                (0, 15, 64, 32, 1), (0, 16, 32800, 32, 0), (0, (1 << 20) + 1, 64, 32, 0)]:
        assert L.moe_matvec_prepared_bytes(*bad) == 0
        assert L.moe_matvec_prepare(*bad, None, None, 0, None, None, size_t(0), None) == SHAPE
    a, odd, f = vp(0x100000), vp(0x100001), c_float(-1)
    need = L.moe_matvec_prepared_bytes(1, 16, 64, 32, 0)

    def prepare(fmt=1, codes=a, scale=a, st=0, zero=None, out=a, n=need):
        return L.moe_matvec_prepare(fmt, 16, 64, 32, 0, codes, scale, st, zero, out, size_t(n), None)

    assert prepare(codes=None) == INVALID and prepare(st=2) == INVALID and prepare(fmt=0, zero=a) == INVALID
    assert prepare(n=need - 1) == WORKSPACE and prepare(scale=odd) == ALIGNMENT and prepare(out=vp(0x100010)) == ALIGNMENT

    def run(x=a, T=2, dtype=0, y=a, K=64, ld=64):
        return L.moe_matvec(1, 16, K, 32, 0, f, 0, a, dtype, x, i64(ld), T, y, None)

    assert run(T=-1) == INVALID and run(dtype=2) == INVALID and run(ld=-1) == INVALID and run(K=65) == SHAPE
    assert run(x=None) == INVALID and run(x=odd) == ALIGNMENT and run(y=odd) == ALIGNMENT
    assert run(T=0, x=None, y=None) == 0


def test_python_refusals_without_a_gpu(L):
    x = torch.zeros(4, 64)
    for f in (lambda: M.norm_before(x), lambda: M.norm_after(x, x), lambda: M.sort_tokens(torch.zeros(4, 2, dtype=torch.int32), 8)):
        with pytest.raises(RuntimeError):
            f()
    for f in (lambda: M.norm_before(x[0]), lambda: M.norm_before(x.long()), lambda: M.sort_tokens(x, 8)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ValueError):
        M.prepare_matvec(dict(fmt="fp8", N=1, K=32))
    with pytest.raises(B.MoeError):
        M.prepare_matvec(dict(fmt="fp4", N=1, K=33, w=x, w_scale=x))
