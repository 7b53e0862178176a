"""GPU: tokens sorted by expert and back, and the gradients, against the
64-bit oracle."""
import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from block_scaled_moe_expert_gb300 import binding as B
from oracle import block as O
from tests import block_cases as C

pytestmark = pytest.mark.gpu


def routing(T, E, K, skip=0.0, seed=0, hot=None):
    g = C.gen(seed)
    idx = torch.stack([torch.randperm(max(E, K), generator=g, device="cuda")[:K] % E for _ in range(min(T, 64))]) \
        if T else torch.zeros(0, K, device="cuda")
    idx = idx.repeat(-(-T // 64), 1)[:T].to(torch.int32) if T else idx.to(torch.int32)
    if hot is not None:
        idx[:] = hot
    if skip:
        idx[torch.rand(T, K, generator=g, device="cuda") < skip] = -1
    w = torch.rand(T, K, generator=g, device="cuda") + 0.1
    return idx.contiguous(), w


SORTS = [  # T, E, K, align, skip, hot expert
    (0, 8, 2, 16, 0, None), (1, 1, 1, 1, 0, None), (1, 256, 8, 128, 0, None), (1, 512, 32, 256, 0, None),
    (3, 8, 2, 1, 1.0, None), (33, 7, 3, 5, 0.2, None), (2000, 512, 2, 1, 0, None), (513, 8, 8, 128, 0.05, None),
    (4096, 5, 1, 16, 0, None), (4097, 3, 1, 1, 0, 2), (5000, 512, 4, 128, 0.1, None), (20000, 60, 7, 3, 0.05, None),
    (9000, 256, 1, 256, 0, 255),
]


@pytest.mark.parametrize("T,E,K,align,skip,hot", SORTS)
def test_sort_is_the_stable_grouping(T, E, K, align, skip, hot):
    idx, _ = routing(T, E, K, skip, seed=T + E, hot=hot)
    plan = M.sort_tokens(idx, E, row_align=align)
    counts, offsets, inv, row_slot = O.sort_tokens(idx.cpu(), E, align)
    assert plan.row_capacity == len(row_slot)
    assert plan.counts.tolist() == counts and plan.offsets.tolist() == offsets
    assert plan.inv.reshape(-1).tolist() == inv and plan.row_slot.tolist() == row_slot
    assert B.device_status(plan.buffer) == 0


def test_sort_flags_ids_out_of_range_and_the_next_sort_clears():
    for T in (9, 6000):
        idx, _ = routing(T, 8, 2)
        idx[T // 2, 1], idx[T - 1, 0] = 8, -2
        plan = M.sort_tokens(idx, 8, row_align=4)
        counts, offsets, inv, row_slot = O.sort_tokens(idx.cpu(), 8, 4)
        assert plan.inv.reshape(-1).tolist() == inv and plan.row_slot.tolist() == row_slot
        assert B.device_status(plan.buffer) == B.MOE_DEV_BAD_EXPERT_ID
        assert B.device_status(plan.buffer) == 0


def test_sort_fills_the_capacity_it_reports():
    # one slot an expert: every group is one row and row_align - 1 of padding
    idx = torch.arange(8, dtype=torch.int32, device="cuda").reshape(4, 2)
    plan = M.sort_tokens(idx, 8, row_align=7)
    assert int(plan.offsets[-1]) == plan.row_capacity == 56


ROWS = [  # T, H, E, K, align, skip
    (1, 64, 8, 2, 1, 0), (1, 7168, 256, 8, 16, 0), (5, 1, 4, 3, 2, 0), (3, 33, 8, 8, 1, 0.5), (65, 2880, 128, 4, 128, 0.1),
    (700, 520, 16, 9, 8, 0.05), (600, 1001, 60, 5, 1, 0.1), (17, 2048, 64, 32, 4, 0.2), (4, 256, 4, 2, 8, 1.0),
]


def make(T, H, E, K, align, skip, dtype, seed=5):
    idx, w = routing(T, E, K, skip, seed=seed)
    plan = M.sort_tokens(idx, E, row_align=align)
    g = C.gen(seed + 1)
    return plan, w, C.randn(g, T, H, dtype=dtype), C.randn(g, plan.row_capacity, H, dtype=dtype)


@pytest.mark.parametrize("dtype", C.DTYPES)
@pytest.mark.parametrize("T,H,E,K,align,skip", ROWS)
def test_rows_there_and_back(T, H, E, K, align, skip, dtype):
    plan, w, x, rows = make(T, H, E, K, align, skip, dtype)
    inv, cap = plan.inv, plan.row_capacity
    rows[plan.row_slot < 0] = float("nan")  # rows of no slot are never read
    dot_steps = H // 256 + 32
    assert torch.equal(M.permute_tokens(x, plan).double(), O.place(x, None, inv, cap))
    placed = O.place(x, w, inv, cap)
    C.check(M.permute_tokens(x, plan, w), placed, placed.abs(), 1, "permute, weighted")
    for ww in (None, w):
        C.check(M.unpermute_tokens(rows, plan, ww), O.gather(rows, ww, inv), O.gather(rows, ww, inv, mag=True), K + 1,
                "unpermute")
        dx, dw = M.permute_tokens_backward(rows, plan, x, ww)
        C.check(dx, O.gather(rows, ww, inv), O.gather(rows, ww, inv, mag=True), K + 1, "d_hidden")
        drows, dw2 = M.unpermute_tokens_backward(x, plan, rows, ww)
        placed = O.place(x, ww, inv, cap)
        C.check(drows, placed, placed.abs(), 1, "d_rows")
        assert (drows[plan.row_slot < 0] == 0).all()
        if ww is None:
            assert dw is None and dw2 is None
        else:
            d, mag = O.dots(x, rows, inv), O.dots(x, rows, inv, mag=True)
            C.check(dw, d, mag, dot_steps, "d_topk_w of permute")
            C.check(dw2, d, mag, dot_steps, "d_topk_w of unpermute")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,lead", [(8, 0), (3, 0), (5, 1), (16, 8)])
def test_strided_and_misaligned_rows(pad, lead, dtype):
    plan, w, x, rows = make(37, 136, 8, 3, 4, 0.1, dtype)
    xs, rs = C.strided(x, pad, lead), C.strided(rows, pad, lead)
    assert torch.equal(M.permute_tokens(xs, plan, w), M.permute_tokens(x, plan, w))
    assert torch.equal(M.unpermute_tokens(rs, plan, w), M.unpermute_tokens(rows, plan, w))
    for a, b in zip(M.unpermute_tokens_backward(xs, plan, rs, w) + M.permute_tokens_backward(rs, plan, xs, w),
                    M.unpermute_tokens_backward(x, plan, rows, w) + M.permute_tokens_backward(rows, plan, x, w)):
        if a.dtype == dtype and a.dim() == 2 and a.shape[1] == 136:
            assert torch.equal(a, b)
        else:  # the dots' order depends on the vector width
            C.check(a, b.double(), torch.full_like(b, 136.0, dtype=torch.float64), 64)
    one = x[:1].expand(37, 136)  # row stride 0
    assert torch.equal(M.permute_tokens(one, plan), M.permute_tokens(one.contiguous(), plan))
    assert torch.equal(M.permute_tokens(x.t().contiguous().t(), plan), M.permute_tokens(x, plan))


def test_special_values_move_unchanged():
    plan, w, x, _ = make(4, 64, 4, 2, 1, 0, torch.bfloat16)
    x[0, 0], x[1, 1], x[2, 2], x[3, 3] = float("inf"), float("-inf"), float("nan"), -0.0
    rows = M.permute_tokens(x, plan)
    assert torch.equal(rows.view(torch.int16), x[(plan.row_slot // 2).long()].view(torch.int16))
    out = M.unpermute_tokens(M.permute_tokens(x, plan, w), plan)
    assert out[0, 0] == float("inf") and out[1, 1] == float("-inf") and out[2, 2].isnan()
    assert int(out.isnan().sum()) == 1


def test_a_plan_of_another_call_moves_nothing_out_of_range():
    """Slots whose row is outside the rows count as skipped."""
    T, H, E, K = 9, 72, 4, 3
    plan, w, x, rows = make(T, H, E, K, 2, 0, torch.float32)
    want_drows, want_dw = M.unpermute_tokens_backward(x, plan, rows, w)
    keep = torch.ones(T, K, dtype=torch.bool, device="cuda")
    for (t, k), row in (((0, 0), plan.row_capacity), ((3, 2), 2 ** 31 - 1), ((8, 1), -2 ** 31), ((5, 0), -7)):
        lost = int(plan.inv[t, k])
        plan.inv[t, k] = row
        keep[t, k] = False
        want_drows[lost] = 0
        plan.row_slot[lost] = -1
    inv = torch.where(keep, plan.inv, torch.full_like(plan.inv, -1))
    C.check(M.unpermute_tokens(rows, plan, w), O.gather(rows, w, inv), O.gather(rows, w, inv, mag=True), K + 1)
    drows, dw = M.unpermute_tokens_backward(x, plan, rows, w)
    assert torch.equal(drows, want_drows) and torch.equal(dw, torch.where(keep, want_dw, torch.zeros_like(want_dw)))


def test_offsets_beyond_32_bits():
    """Rows whose element offsets pass 2^31 (8 GB of rows)."""
    H, T, K, E = 65536, 8224, 4, 4
    idx = torch.arange(K, dtype=torch.int32, device="cuda").repeat(T, 1)
    plan = M.sort_tokens(idx, E)
    assert plan.row_capacity * H > 2 ** 31
    x = torch.empty(T, H, dtype=torch.float16, device="cuda")
    x.copy_(torch.arange(T, device="cuda")[:, None] % 97)
    x[:, 1] = 5
    rows = M.permute_tokens(x, plan)
    assert torch.equal(rows[3 * T:], x) and torch.equal(rows[T:2 * T], x)
    out = M.unpermute_tokens(rows, plan)
    assert torch.equal(out[-3:], 4 * x[-3:]) and torch.equal(out[:3], 4 * x[:3])


def test_autograd_is_the_gradient():
    """Through permute (weighted) and unpermute (weighted), against autograd of
    the same products on the oracle's order and against differences."""
    T, H, E, K = 19, 40, 6, 3
    plan, w, x, _ = make(T, H, E, K, 4, 0.2, torch.float32)
    g = C.gen(9)
    mix = C.randn(g, plan.row_capacity, H)
    probe = C.randn(g, T, H)
    x.requires_grad_(), w.requires_grad_()

    def loss(x, w):
        rows = M.permute_tokens(x, plan, w)
        return (M.unpermute_tokens(rows * mix, plan, w) * probe).double().sum()

    loss(x, w).backward()
    x64, w64 = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    out = 0.0
    for k in range(K):
        ok = plan.inv[:, k] >= 0
        r = plan.inv[:, k].clamp(min=0).long()
        out = out + torch.where(ok[:, None], x64 * mix.double()[r] * w64[:, k:k + 1] ** 2, torch.zeros(1, device="cuda"))
    (out * probe.double()).sum().backward()
    mag = (mix.abs().max() ** 2 * probe.abs().max() * x.abs().max()).double()
    C.check(x.grad, x64.grad, torch.full_like(x64.grad, float(mag)), 4 * K)
    C.check(w.grad, w64.grad, torch.full_like(w64.grad, float(mag) * H), 4 * H)
    # differences: the loss is quadratic in w and linear in x, so the central
    # difference has rounding errors only: 2^-24 of the terms, over the step
    for t, d in ((x, torch.randn_like(x)), (w, torch.randn_like(w))):
        step = 2.0 ** -4
        with torch.no_grad():
            args = [(x + step * d, w), (x - step * d, w)] if t is x else [(x, w + step * d), (x, w - step * d)]
            diff = (loss(*args[0]) - loss(*args[1])) / (2 * step)
            terms = float(sum((M.unpermute_tokens((M.permute_tokens(a.abs(), plan, b.abs()) * mix.abs()), plan,
                                                  b.abs()) * probe.abs()).sum() for a, b in args))
        assert abs(float(diff) - float((t.grad.double() * d.double()).sum())) <= 16 * 2.0 ** -24 * terms / step


def test_plan_and_rows_on_another_stream_and_in_a_graph():
    plan_in, w, x, _ = make(130, 512, 16, 4, 8, 0.1, torch.bfloat16)
    idx = torch.where(plan_in.inv >= 0, plan_in.inv, -1)  # any int32 tensor of the shape
    idx = (idx % 16).to(torch.int32).contiguous()
    want = M.unpermute_tokens(M.permute_tokens(x, M.sort_tokens(idx, 16, 8), w), M.sort_tokens(idx, 16, 8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan = M.sort_tokens(idx, 16, 8)
        out = M.unpermute_tokens(M.permute_tokens(x, plan, w), plan)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = M.sort_tokens(idx, 16, 8)
        out = M.unpermute_tokens(M.permute_tokens(x, plan, w), plan)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


def test_refusals():
    plan, w, x, rows = make(4, 64, 4, 2, 1, 0, torch.bfloat16)
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        M.sort_tokens(idx.long(), 4)
    with pytest.raises(ValueError):
        M.permute_tokens(x[:3], plan)
    with pytest.raises(ValueError):
        M.permute_tokens(x.to(torch.float64), plan)
    with pytest.raises(ValueError):
        M.unpermute_tokens(rows[:-1], plan)
    with pytest.raises(ValueError):
        M.permute_tokens(x, plan, w.double())
    with pytest.raises(ValueError):
        M.unpermute_tokens_backward(x, plan, None, w)
    with pytest.raises(ValueError):
        M.unpermute_tokens_backward(x, plan, rows.float(), w)
    with pytest.raises(ValueError):
        M.permute_tokens(x, plan, out=torch.empty_like(rows.float()))
    with pytest.raises(B.MoeError):
        M.sort_tokens(idx, 0)
    with pytest.raises(B.MoeError):
        M.sort_tokens(idx, 513)
    with pytest.raises(B.MoeError):
        M.sort_tokens(idx, 4, row_align=257)
    with pytest.raises(RuntimeError):
        M.sort_tokens(idx.cpu(), 4)
    with pytest.raises(RuntimeError):
        M.permute_tokens(x.cpu(), plan)
