"""GPU: the norms around a block, with gate, residual scale and the next norm,
and their gradients, against the 64-bit oracle."""
import itertools

import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from block_scaled_moe_expert_gb300 import binding as B
from oracle import block as O
from tests import block_cases as C

pytestmark = pytest.mark.gpu

EPS = 1e-5
SHAPES = [(1, 64), (1, 7168), (3, 1), (5, 33), (130, 512), (9, 520), (37, 1001), (700, 256), (40, 2880), (310, 4096),
          (4, 8192), (3, 8200), (2, 16384), (2, 16383)]


def steps(H, T=1):
    # a thread's own terms, the tree over the threads, the parts' sums over rows
    return H // 32 + T + 64


def gate_of(g, kind, T, H, dtype):
    shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[kind]
    return None if shape is None else C.randn(g, *shape, dtype=dtype)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_before_and_its_gradient(T, H, dtype):
    g = C.gen(T + H)
    x, dy, dr = (C.randn(g, T, H, dtype=dtype, scale=s) for s in (3.0, 0.5, 0.5))
    for wdtype, offset in ((dtype, 0.0), (torch.float32, 1.0), (None, 0.0)):
        w = None if wdtype is None else C.randn(g, H, dtype=wdtype, scale=0.3)
        y = O.norm(x, w, EPS, offset)
        C.check(M.norm_before(x, w, EPS, offset), y, y.abs(), steps(H), "y")
        for res in (None, dr):
            dx, dw = M.norm_before_backward(dy, x, w, EPS, offset, dr=res)
            edx, edw = O.norm_backward(dy, x, w, EPS, offset)
            mdx, mdw = O.norm_backward(dy, x, w, EPS, offset, mag=True)
            if res is not None:
                edx, mdx = edx + res.double(), mdx + res.double().abs()
            C.check(dx, edx, mdx, steps(H), "dx")
            assert (dw is None) == (w is None)
            if w is not None:
                assert dw.dtype == w.dtype
                C.check(dw, edw, mdw, steps(H, T), "d_weight")


CASES = list(itertools.product(["none", "channel", "token", "element"], ["none", "sigmoid", "tanh"], [True, False],
                               [True, False]))


def after_case(T, H, dtype, i):
    """One of the combinations of gate, activation, norm and next norm."""
    kind, act, has_norm, nxt = CASES[i % len(CASES)]
    g = C.gen(100 * T + H + i)
    x, h, dr, dy = (C.randn(g, T, H, dtype=dtype, scale=s) for s in (2.0, 3.0, 0.5, 0.5))
    wdtype = torch.float32 if i % 3 == 0 else dtype
    w = C.randn(g, H, dtype=wdtype, scale=0.5) if has_norm and i % 5 else None
    nw = C.randn(g, H, dtype=wdtype, scale=0.5) if nxt and i % 7 else None
    gate = gate_of(g, kind, T, H, dtype)
    kw = dict(gate=gate, gate_act=act, alpha=0.7 if i % 2 else 1.0, beta=1.3 if i % 4 == 1 else 1.0, eps=EPS,
              weight_offset=1.0 if i % 2 else 0.0, norm=has_norm, next_weight=nw)
    return x, h, dr, dy, w, nw, gate, kw, nxt


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_after_and_its_gradient(T, H, dtype):
    first = SHAPES.index((T, H)) * 3
    for i in range(first, first + (len(CASES) if (T, H) in ((9, 520), (37, 1001), (130, 512)) else 6)):
        x, h, dr, dy, w, nw, gate, kw, nxt = after_case(T, H, dtype, i)
        off, act, a, b = kw["weight_offset"], kw["gate_act"], kw["alpha"], kw["beta"]
        args = (w, gate, act, a, b, EPS, off, kw["norm"])
        er, mr = O.norm_after(x, h, *args), O.norm_after(x, h, *args, mag=True)
        out = M.norm_after(x, h, w, next_norm=nxt, next_eps=EPS / 2, **kw)
        r, y = out if nxt else (out, None)
        C.check(r, er, mr, steps(H), ("r", i))
        if nxt:
            ey = O.norm(er, nw, EPS / 2, off)
            # r's rounding errors reach y by its own term and by the row's scale
            s = 1 / torch.sqrt((er * er).mean(1, keepdim=True) + EPS / 2)
            wn = 1.0 if nw is None else (nw.double() + off).abs()
            spread = (mr * mr).mean(1, keepdim=True).sqrt() * s
            C.check(y, ey, s * wn * mr + ey.abs() * (1 + spread), steps(H), ("y", i))
        bk = dict(dy=dy, r=r, next_w=nw, next_eps=EPS / 2) if nxt else {}
        want = O.norm_after_backward(dr, h, *args, **bk)
        mags = O.norm_after_backward(dr, h, *args, **bk, mag=True)
        kw.pop("next_weight")
        got = M.norm_after_backward(dr, h, w, dy=dy if nxt else None, r=r if nxt else None, next_weight=nw,
                                    next_eps=EPS / 2, **kw)
        have = (True, True, w is not None, gate is not None, nw is not None)
        over_tokens = (False, False, True, gate is not None and gate.dim() == 1, True)
        for name, o, e, m, there, summed in zip(("dx", "dh", "dw", "dgate", "dnext"), got, want, mags, have,
                                                over_tokens):
            assert (o is not None) == there, (name, i)
            if there:
                # G's, the statistics' and the sums' roundings one after another
                C.check(o, e.expand(o.shape), m.expand(o.shape), 3 * steps(H, T if summed else 1), (name, i))


def test_sums_over_many_tokens_repeat_bit_for_bit():
    x, h, dr, dy, w, nw, gate, kw, _ = after_case(5000, 1024, torch.bfloat16, 21)
    g = C.gen(3)
    w, nw, gate = (C.randn(g, 1024, dtype=torch.bfloat16) for _ in range(3))
    r = C.randn(g, 5000, 1024, dtype=torch.bfloat16)
    runs = [M.norm_after_backward(dr, h, w, gate=gate, dy=dy, r=r, next_weight=nw) for _ in range(3)]
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))
    want = O.norm_after_backward(dr, h, w, gate, "none", 1.0, 1.0, 1e-6, 0.0, True, dy, r, nw, 1e-6)
    mags = O.norm_after_backward(dr, h, w, gate, "none", 1.0, 1.0, 1e-6, 0.0, True, dy, r, nw, 1e-6, mag=True)
    for o, e, m in zip(runs[0], want, mags):
        C.check(o, e, m, 3 * steps(1024, 5000))


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("T,H", [(1003, 1001), (2500, 37), (640, 2049), (900, 4091), (333, 8185), (320, 8190)])
def test_odd_widths_over_many_tokens(T, H, dtype):
    """Every row starts at another place of a 16-byte chunk, and a block walks
    several rows; strided operands start elsewhere than contiguous ones."""
    x, h, dr, dy, w, nw, gate, kw, _ = after_case(T, H, dtype, 44)  # element gate, norm, next norm
    assert gate.shape == (T, H) and w is not None and nw is not None
    args = (w, gate, kw["gate_act"], kw["alpha"], kw["beta"], EPS, kw["weight_offset"], True)
    er, mr = O.norm_after(x, h, *args), O.norm_after(x, h, *args, mag=True)
    s = 1 / torch.sqrt((er * er).mean(1, keepdim=True) + EPS)
    ey = O.norm(er, nw, EPS, kw["weight_offset"])
    my = s * (nw.double() + kw["weight_offset"]).abs() * mr + ey.abs() * (1 + (mr * mr).mean(1, keepdim=True).sqrt() * s)
    r = None
    for xs, hs in ((x, h), (C.strided(x, 3), h), (x, C.strided(h, 8, 1))):
        r, y = M.norm_after(xs, hs, w, **kw)
        C.check(r, er, mr, steps(H))
        C.check(y, ey, my, steps(H))
    kw.pop("next_weight")
    want = O.norm_after_backward(dr, h, *args, dy, r, nw, EPS)
    mags = O.norm_after_backward(dr, h, *args, dy, r, nw, EPS, mag=True)
    for ds, hs in ((dr, h), (C.strided(dr, 5), h), (dr, C.strided(h, 16, 2))):
        got = M.norm_after_backward(ds, hs, w, dy=dy, r=r, next_weight=nw, **kw)
        for o, e, m in zip(got, want, mags):
            C.check(o, e, m, 3 * steps(H, T))


@pytest.mark.parametrize("H", [512, 1024, 1000, 1001])
def test_strided_misaligned_and_broadcast_rows(H):
    g = C.gen(H)
    T = 21
    x, h, dr, dy, gate = (C.randn(g, T, H, dtype=torch.bfloat16) for _ in range(5))
    w = C.randn(g, H + 1, dtype=torch.bfloat16)
    views = [C.strided(t, pad, lead) for t, pad, lead in zip((x, h, dr, dy, gate), (8, 3, 16, 1, 5), (0, 1, 8, 0, 2))]
    want_r, want_y = M.norm_after(x, h, w[1:].clone(), gate=gate, gate_act="tanh", next_norm=True)
    r, y = M.norm_after(views[0], views[1], w[1:], gate=views[4], gate_act="tanh", next_norm=True)
    # the order of a row's sum depends on the vector width
    C.check(r, want_r.double(), O.norm_after(x, h, w[1:], gate, "tanh", 1, 1, 1e-6, 0, True, mag=True) * 2 ** 17, 1)
    C.check(y, want_y.double(), want_y.double().abs() * 2 ** 17, 1)
    got = M.norm_after_backward(views[2], views[1], w[1:], gate=views[4], gate_act="tanh", dy=views[3], r=want_r)
    args = (w[1:], gate, "tanh", 1.0, 1.0, 1e-6, 0.0, True, dy, want_r, None, 1e-6)
    for o, e, m in zip(got[:4], O.norm_after_backward(dr, h, *args), O.norm_after_backward(dr, h, *args, mag=True)):
        C.check(o, e, m, 3 * steps(H, T))
    ones = x[:1].expand(T, H)
    assert torch.equal(M.norm_before(ones), M.norm_before(ones.contiguous()))
    assert torch.equal(M.norm_before(x.t().contiguous().t()), M.norm_before(x))
    token = C.randn(g, T, 3, dtype=torch.bfloat16)[:, 1:2]  # a strided token gate
    assert torch.equal(M.norm_after(x, h, gate=token), M.norm_after(x, h, gate=token.contiguous()))


def test_offsets_beyond_32_bits():
    """Rows whose element offsets pass 2^31: the last rows as a call of their own."""
    T, H, n = 263000, 8192, 40
    assert T * H > 2 ** 31
    g = C.gen(6)
    tail = C.randn(g, n, H, dtype=torch.bfloat16)
    w = C.randn(g, H, dtype=torch.bfloat16)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[-n:] = tail
    r, y = M.norm_after(x, x, w, next_weight=w)
    want_r, want_y = M.norm_after(tail, tail, w, next_weight=w)
    assert torch.equal(r[-n:], want_r) and torch.equal(y[-n:], want_y)
    assert int(torch.count_nonzero(y[:-n])) == 0
    del y
    dx, dh, dw, _, dn = M.norm_after_backward(x, x, w, dy=x, r=r, next_weight=w)
    want = M.norm_after_backward(tail, tail, w, dy=tail, r=want_r, next_weight=w)
    assert torch.equal(dx[-n:], want[0]) and torch.equal(dh[-n:], want[1])
    # the same terms, shared out to other blocks
    args = (w, None, "none", 1.0, 1.0, 1e-6, 0.0, True, tail, want_r, w, 1e-6)
    mags = O.norm_after_backward(tail, tail, *args, mag=True)
    for o, e, m in zip((dw, dn), O.norm_after_backward(tail, tail, *args)[2::2], mags[2::2]):
        C.check(o, e, m, 3 * steps(H, T))


def test_no_tokens():
    for H in (64, 33):
        x = torch.zeros(0, H, dtype=torch.bfloat16, device="cuda")
        w = torch.ones(H, device="cuda")
        assert M.norm_before(x, w).shape == (0, H)
        dx, dw = M.norm_before_backward(x, x, w)
        assert dx.shape == (0, H) and (dw == 0).all()
        r, y = M.norm_after(x, x, w, gate=w.to(x.dtype), next_weight=w)
        got = M.norm_after_backward(x, x, w, gate=w.to(x.dtype), dy=x, r=r, next_weight=w)
        assert y.shape == (0, H) and all((t == 0).all() for t in got)


def test_zero_rows_and_special_values():
    x = torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda")
    x[1, 5], x[2, 7] = float("inf"), float("nan")
    x[3] = 1.0
    y = M.norm_before(x)
    assert (y[0] == 0).all()                       # eps keeps a zero row finite
    assert y[1, 5].isnan() and (y[1, :5] == 0).all()  # inf * rsqrt(inf) = inf * 0
    assert y[2].isnan().all() and y[3].isfinite().all()
    dx, dw = M.norm_before_backward(x[[0, 3]], x[[0, 3]], torch.ones(512, device="cuda"))
    assert dx.isfinite().all() and dw.isfinite().all()


@pytest.mark.parametrize("kind,act", [("channel", "none"), ("token", "sigmoid"), ("element", "tanh")])
def test_autograd_is_the_gradient(kind, act):
    """Against the oracle's autograd, and against central differences."""
    T, H = 7, 48
    g = C.gen(11)
    x, h, w, nw = (C.randn(g, *s) for s in ((T, H), (T, H), (H,), (H,)))
    gate = gate_of(g, kind, T, H, torch.float32)
    pr, py = C.randn(g, T, H), C.randn(g, T, H)
    leaves = [t.requires_grad_() for t in (x, h, w, gate, nw)]

    def loss(x, h, w, gate, nw):
        b = M.norm_before(x, w, 1e-3)
        r, y = M.norm_after(x, h + b, w, gate=gate, gate_act=act, alpha=0.5, beta=0.8, eps=1e-3, next_weight=nw)
        return ((r * pr).double() + (y * py).double()).sum()

    loss(*leaves).backward()
    wide = [t.detach().double().requires_grad_() for t in leaves]
    x64, h64, w64, g64, n64 = wide
    r = O.norm_after(x64, h64 + O.norm(x64, w64, 1e-3), w64, g64, act, 0.5, 0.8, 1e-3, 0.0, True)
    ((r * pr.double()) + O.norm(r, n64, 1e-3) * py.double()).sum().backward()
    for t, u in zip(leaves, wide):
        # the gradients' terms are of the order of their norm; T H terms of
        # fp32 roundings through three norms
        scale = torch.full_like(u.grad, float(u.grad.abs().max()) + 1.0)
        C.check(t.grad, u.grad, scale, 8 * (T + H))
    for i, t in enumerate(leaves):
        d = torch.randn_like(t)
        step = 2.0 ** -7
        with torch.no_grad():
            moved = [list(leaves), list(leaves)]
            moved[0][i], moved[1][i] = t + step * d, t - step * d
            diff = float(loss(*moved[0]) - loss(*moved[1])) / (2 * step)
            def wide_loss(ts):
                x, h, w, gate, nw = [v.detach().double() for v in ts]
                r = O.norm_after(x, h + O.norm(x, w, 1e-3), w, gate, act, 0.5, 0.8, 1e-3, 0.0, True)
                return float((r * pr.double() + O.norm(r, nw, 1e-3) * py.double()).sum())
            # what the difference itself is off by, in 64 bits, and the roundings of T H terms over the step
            exact = float((wide[i].grad * d.double()).sum())
            cut = abs((wide_loss(moved[0]) - wide_loss(moved[1])) / (2 * step) - exact)
        assert abs(diff - float((t.grad.double() * d.double()).sum())) <= cut + T * H * 32 * 2.0 ** -24 / step


def test_autograd_with_only_one_output_used():
    g = C.gen(2)
    x, h = (C.randn(g, 5, 64).requires_grad_() for _ in range(2))
    r, y = M.norm_after(x, h, next_norm=True)
    y.sum().backward()
    want = O.norm_after_backward(torch.zeros(5, 64, device="cuda"), h.detach(), None, None, "none", 1.0, 1.0, 1e-6, 0.0,
                                 True, torch.ones(5, 64, device="cuda"), r.detach(), None, 1e-6)
    # r is rounded to fp32 between the passes
    C.check(x.grad, want[0], torch.full_like(want[0], 64.0), 64)
    C.check(h.grad, want[1], torch.full_like(want[1], 64.0), 64)


def test_replay_in_a_graph():
    g = C.gen(4)
    x, h, dr = (C.randn(g, 300, 2048, dtype=torch.bfloat16) for _ in range(3))
    w = C.randn(g, 2048)
    want = [*M.norm_after(x, h, w, next_weight=w), *M.norm_before_backward(dr, x, w)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [*M.norm_after(x, h, w, next_weight=w), *M.norm_before_backward(dr, x, w)]
    for t in got:
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad in (x.double(), x[0], x.to(torch.int32)):
        with pytest.raises(ValueError):
            M.norm_before(bad)
    for bad in (w[:-1], w.half(), x):
        with pytest.raises(ValueError):
            M.norm_before(x, bad)
    with pytest.raises(ValueError):
        M.norm_after(x, x[:3])
    with pytest.raises(ValueError):
        M.norm_after(x, x.float())
    with pytest.raises(ValueError):
        M.norm_after(x, x, w, norm=False)
    with pytest.raises(ValueError):
        M.norm_after(x, x, w, next_weight=w.to(x.dtype))
    with pytest.raises(ValueError):
        M.norm_after(x, x, next_weight=w, next_norm=False)
    for bad in (w, x[:, :5], x[:3, :1], x[0, :5]):
        with pytest.raises(ValueError):
            M.norm_after(x, x, gate=bad)
    with pytest.raises(ValueError):
        M.norm_after(x, x, gate=x, gate_act="relu")
    with pytest.raises(ValueError):
        M.norm_after_backward(x, x, dy=x)
    with pytest.raises(ValueError):
        M.norm_after_backward(x, x, next_weight=w)
    with pytest.raises(B.MoeError):
        M.norm_before(torch.zeros(1, 16385, device="cuda"))
    with pytest.raises(RuntimeError):
        M.norm_before(x.cpu())
    with pytest.raises(RuntimeError):
        M.norm_before(x, w.cpu())
    with pytest.raises(ValueError):
        M.norm_before(x.float().requires_grad_(), out=torch.empty(4, 64, device="cuda"))
