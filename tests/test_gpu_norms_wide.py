"""GPU: wide rows with several rows to a block, so that every kernel's loop over
rows turns more than once: 16-bit rows above 8192 columns, fp32 rows above 4096,
and wide rows of odd widths and places."""
import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from oracle import block as O
from tests import block_cases as C
from tests.test_gpu_norms import steps

pytestmark = pytest.mark.gpu

EPS = 1e-5
# more rows than SMs: a block walks two to five
SHAPES = [(500, 8200), (330, 16384), (310, 16383), (620, 7168), (640, 5001), (400, 8192), (350, 12288)]


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate_kind", ["channel", "token", "element"])
def test_norms_of_wide_rows_walk_many(T, H, gate_kind, dtype):
    g = C.gen(T + H)
    x, h, dr, dy = (C.randn(g, T, H, dtype=dtype, scale=s) for s in (2.0, 3.0, 0.5, 0.5))
    w, nw = (C.randn(g, H, dtype=dtype, scale=0.5) for _ in range(2))
    gate = C.randn(g, *{"channel": (H,), "token": (T, 1), "element": (T, H)}[gate_kind], dtype=dtype)
    args = (w, gate, "tanh", 0.7, 1.3, EPS, 1.0, True)
    kw = dict(gate=gate, gate_act="tanh", alpha=0.7, beta=1.3, eps=EPS, weight_offset=1.0)
    er, mr = O.norm_after(x, h, *args), O.norm_after(x, h, *args, mag=True)
    s = 1 / torch.sqrt((er * er).mean(1, keepdim=True) + EPS)
    ey = O.norm(er, nw, EPS, 1.0)
    my = s * (nw.double() + 1.0).abs() * mr + ey.abs() * (1 + (mr * mr).mean(1, keepdim=True).sqrt() * s)
    r, y = M.norm_after(x, h, w, next_weight=nw, **kw)
    C.check(r, er, mr, steps(H), "r")
    C.check(y, ey, my, steps(H), "y")
    del er, mr, ey, my, s
    want = O.norm_after_backward(dr, h, *args, dy, r, nw, EPS)
    mags = O.norm_after_backward(dr, h, *args, dy, r, nw, EPS, mag=True)
    for hh in (h, C.strided(h, 5, 1)):
        got = M.norm_after_backward(dr, hh, w, dy=dy, r=r, next_weight=nw, **kw)
        for name, o, e, m in zip(("dx", "dh", "dw", "dgate", "dnext"), got, want, mags):
            C.check(o, e, m, 3 * steps(H, T), name)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_before_of_wide_rows_walks_many(T, H, dtype):
    g = C.gen(T + H + 1)
    x, dy, dr = (C.randn(g, T, H, dtype=dtype, scale=s) for s in (3.0, 0.5, 0.5))
    w = C.randn(g, H, dtype=torch.float32, scale=0.3)
    e = O.norm(x, w, EPS)
    for xx in (x, C.strided(x, 3)):
        C.check(M.norm_before(xx, w, EPS), e, e.abs(), steps(H), "y")
        dx, dw = M.norm_before_backward(dy, xx, w, EPS, dr=dr)
        edx, edw = O.norm_backward(dy, x, w, EPS)
        mdx, mdw = O.norm_backward(dy, x, w, EPS, mag=True)
        C.check(dx, edx + dr.double(), mdx + dr.double().abs(), steps(H), "dx")
        C.check(dw, edw, mdw, steps(H, T), "d_weight")
