"""GPU: the router's choice of experts, its weights and mean scores, and their
gradient against the 64-bit oracle.

Bounds. A weight is made of exponentials of x - most (one rounding: relative error
|x - most| 2^-24 of the exponential, 2^-22 of the exponential itself with its fast
form), a sum of positive terms and a quotient: relative error below
(2 D + 32) 2^-23 with D the largest |x - most|. A mean adds the roundings of a sum
of positive terms, fewer than 64 on any path for the sizes here. A gradient has
the same factors, so twice that of the magnitude of its terms, and its rounding.
"""
import math

import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from oracle import block as O
from tests import block_cases as C

pytestmark = pytest.mark.gpu


def logits_of(seed, T, E, dtype=torch.float32, scale=1.5):
    g = C.gen(seed)
    return C.randn(g, T, E, dtype=dtype, scale=scale), C.randn(g, E, scale=0.1)


def check(logits, K, score="softmax", bias=None, groups=1, top_groups=1, group_score="top2", renorm=True, scale=1.0,
          mean=True):
    out = M.route_tokens(logits, K, score=score, bias=bias, num_groups=groups, top_groups=top_groups,
                         group_score=group_score, renormalize=renorm, scale=scale, mean_scores=mean)
    idx = O.choose(logits, K, score, bias, groups, top_groups, group_score)
    assert out[0].dtype == torch.int32 and out[1].dtype == torch.float32
    assert torch.equal(out[0].long(), idx)
    w = O.route_weights(logits, idx, score, renorm, scale)
    x = logits.double()
    D = float((x.amax(1, keepdim=True) - x).nan_to_num(0, 0, 0).max()) if x.numel() else 0.0
    tol = (2 * min(D, 90.0) + 32) * 2.0 ** -23
    assert torch.equal(out[1].isnan(), w.isnan())
    err = (out[1].double() - w).abs().nan_to_num(0)
    assert bool((err <= tol * w.abs().nan_to_num(0) + 1e-37).all()), float((err / w.abs()).nan_to_num(0).max() / tol)
    if mean:
        p = O.scores(logits, score)[1].mean(0) if logits.shape[0] else torch.zeros_like(out[2], dtype=torch.float64)
        assert out[2].shape == (logits.shape[1],)
        assert torch.equal(out[2].isnan(), p.isnan())
        err = (out[2].double() - p).abs().nan_to_num(0)
        assert bool((err <= (2 * tol + 64 * 2.0 ** -24) * p.nan_to_num(0) + 1e-37).all())
    return out


@pytest.mark.parametrize("E,K", [(1, 1), (2, 2), (7, 3), (8, 2), (8, 8), (31, 31), (32, 32), (60, 5), (64, 6),
                                 (96, 7), (128, 4), (160, 8), (256, 8), (300, 20), (384, 32), (512, 1), (511, 9)])
@pytest.mark.parametrize("dtype", C.DTYPES)
def test_choice_and_weights(E, K, dtype):
    for T in (1, 77, 1030):
        x, bias = logits_of(E + K + T, T, E, dtype)
        check(x, K, "softmax", renorm=True)
        check(x, K, "softmax", renorm=False, scale=1.5)
        check(x, K, "sigmoid", bias, renorm=True, scale=2.5)
        check(x, K, "sigmoid", renorm=False, mean=False)
        check(x, K, "softmax", bias, renorm=False, mean=False)


@pytest.mark.parametrize("E,groups,top_groups,K", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 32, 5, 10), (96, 3, 2, 7),
                                                   (510, 17, 4, 9), (512, 2, 1, 32), (60, 5, 5, 5), (24, 12, 2, 4),
                                                   (32, 32, 8, 8), (512, 16, 3, 8), (384, 6, 2, 8)])
@pytest.mark.parametrize("group_score", ["top2", "max"])
def test_groups(E, groups, top_groups, K, group_score):
    for dtype in (torch.float32, torch.bfloat16):
        x, bias = logits_of(E + groups, 600, E, dtype)
        for score in ("softmax", "sigmoid"):
            check(x, K, score, bias, groups, top_groups, group_score, scale=2.5)
            check(x, K, score, None, groups, top_groups, group_score, renorm=False, mean=False)


def test_many_tokens_choose_as_64_bits_do():
    """fp32 scores would choose otherwise for some of these."""
    x, bias = logits_of(5, 200000, 256)
    check(x, 8, "sigmoid", bias, 8, 4, "top2", scale=2.5)
    check(x, 8, "softmax", bias, renorm=False)
    x, bias = logits_of(6, 100000, 128, torch.bfloat16)
    check(x, 4, "softmax", None)
    check(x, 6, "sigmoid", torch.zeros_like(bias))


def test_biased_scores_nearer_than_fp32_holds():
    """A bias that cancels the scores: all keys within a few fp32 steps of each other."""
    for score in ("sigmoid", "softmax"):
        for E, K, groups in ((256, 8, 1), (64, 12, 4), (60, 7, 1)):
            x, _ = logits_of(E, 1, E)
            s = O.scores(x, score)[0][0]
            bias = (0.75 - s).float()
            near = x + 1e-6 * torch.arange(50, device="cuda")[:, None] * C.randn(C.gen(1), 50, E)
            check(near, K, score, bias, groups, max(1, groups // 2))


def test_ties_go_to_the_lowest_index():
    for E, K in ((256, 8), (60, 9), (8, 3)):
        zero = torch.zeros(5, E, device="cuda")
        zero[1, 3] = -0.0
        zero[2] = 3.0
        for bias in (None, torch.zeros(E, device="cuda")):
            for score in ("softmax", "sigmoid"):
                idx = check(zero, K, score, bias)[0]
                assert idx.tolist() == [list(range(K))] * 5
    same = torch.zeros(3, 64, device="cuda")
    idx = check(same, 4, "sigmoid", None, 8, 2)[0]
    assert idx.tolist() == [[0, 1, 2, 3]] * 3


def test_saturated_scores():
    """Logits where sigmoids reach 1 or leave fp32's range; 64 bits hold them."""
    x, bias = logits_of(9, 200, 64)
    check(x * 6 - 20, 6, "sigmoid", bias)
    check(x - 100, 6, "sigmoid", None)           # e^-100: below fp32, the ratios are not
    check(x - 300, 6, "sigmoid", None, renorm=True)
    check(x * 30, 6, "softmax", None)
    check(x + 20, 6, "sigmoid", None)


def test_masked_experts():
    """-inf: never chosen; tokens with fewer available experts than K, and with none."""
    x, bias = logits_of(10, 64, 60)
    n = torch.arange(64, device="cuda") % 20
    x = torch.where(torch.rand(64, 60, generator=C.gen(4), device="cuda").argsort(1).argsort(1) < n[:, None], x, -math.inf)
    x[0] = -math.inf
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            out = check(x, 8, score, None, renorm=renorm)
            assert bool((out[0][0] == -1).all()) and bool((out[1][0] == 0).all())
            check(x, 8, score, bias, renorm=renorm)
            check(x, 8, score, bias, 6, 2, renorm=renorm)
            check(x, 8, score, None, 6, 2, "max", renorm=renorm)
    closed = bias.clone()
    closed[::2] = -math.inf  # experts taken out of service
    closed[1] = float("nan")
    out = check(x, 8, "sigmoid", closed)
    assert not bool(((out[0] >= 0) & ((out[0] % 2 == 0) | (out[0] == 1))).any())
    lowest = torch.where(x == -math.inf, torch.finfo(torch.float32).min, x)  # a mask of the lowest value: last, but available
    check(lowest, 8, "softmax", None)


def test_nan_and_infinite_logits():
    x, bias = logits_of(11, 12, 32)
    x[3, 5] = float("nan")
    x[7] = float("nan")
    for score in ("softmax", "sigmoid"):
        idx, w, mean = M.route_tokens(x, 4, score=score, bias=bias, mean_scores=True)
        assert torch.equal(idx.long(), O.choose(torch.where(x.isnan(), -math.inf, x), 4, score, bias))
        bad = w.isnan().all(1)
        assert bad.tolist() == [t in (3, 7) for t in range(12)] and bool(mean.isnan().all())
    y = logits_of(12, 4, 32)[0]
    y[1, 9] = math.inf
    idx, w = M.route_tokens(y, 4, score="sigmoid")
    assert int(idx[1, 0]) == 9 and abs(float(w[1].sum()) - 1) < 1e-6


def test_strides_offsets_and_empty_batches():
    x, bias = logits_of(13, 90, 256, torch.bfloat16)
    want = M.route_tokens(x, 8, bias=bias, mean_scores=True)
    for pad, lead in ((8, 0), (1, 1), (3, 5)):
        got = M.route_tokens(C.strided(x, pad, lead), 8, bias=bias, mean_scores=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = M.route_tokens(x.t().contiguous().t(), 8, bias=bias, mean_scores=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    row = M.route_tokens(x[:1].expand(5, 256), 8, bias=bias)
    assert torch.equal(row[0], want[0][:1].expand(5, 8))
    idx, w, mean = M.route_tokens(x[:0], 8, mean_scores=True)
    assert idx.shape == (0, 8) and w.shape == (0, 8) and bool((mean == 0).all())
    assert M.route_tokens_backward(w, x[:0], idx, d_mean_scores=mean).shape == (0, 256)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,K", [(8, 2), (8, 8), (60, 5), (128, 4), (256, 8), (300, 17), (512, 32), (3, 1)])
def test_gradient(score, renorm, E, K):
    for dtype in C.DTYPES:
        for T, with_mean in ((1, True), (333, False), (700, True)):
            x, bias = logits_of(E + K + T, T, E, dtype)
            g = C.gen(T)
            dw, dmean = C.randn(g, T, K), C.randn(g, E) if with_mean else None
            idx = O.choose(x, K, score, bias).int()
            check_gradient(dw, x, idx, score, renorm, 1.5, dmean)


def check_gradient(dw, x, idx, score, renorm, scale, dmean):
    got = M.route_tokens_backward(dw, x, idx, score=score, renormalize=renorm, scale=scale, d_mean_scores=dmean)
    args = (dw, x, idx, score, renorm, scale, dmean)
    exact, mag = O.route_backward(*args), O.route_backward(*args, mag=True)
    D = float((x.double().amax(1, keepdim=True) - x.double()).nan_to_num(0, 0, 0).max())
    assert got.dtype == x.dtype
    C.check(got, exact, mag, 4 * (2 * min(D, 90.0) + 32 + idx.shape[1]), f"{score} {renorm}")


def test_gradient_of_skipped_foreign_and_repeated_experts():
    x, _ = logits_of(20, 40, 60)
    idx = torch.randint(0, 60, (40, 6), generator=C.gen(2), device="cuda", dtype=torch.int32)
    idx[::3, 2] = -1
    idx[1::3, 0] = 60
    idx[5] = -1
    idx[7] = 11
    x[9, 10:] = -math.inf
    idx[9] = torch.tensor([0, 1, 2, 3, -1, -1], dtype=torch.int32)
    dw, dmean = C.randn(C.gen(3), 40, 6), C.randn(C.gen(4), 60)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for dm in (None, dmean):
                check_gradient(dw, x, idx, score, renorm, 2.0, dm)
    x[9] = -math.inf
    idx[9] = -1
    got = M.route_tokens_backward(dw, x, idx, d_mean_scores=dmean)
    assert bool((got[9] == 0).all()) and not bool(got.isnan().any())


def test_gradient_against_differences():
    """In 64 bits, of the weights that the kernel's choice has: steps of 1e-5 with an error of their square."""
    x, bias = logits_of(21, 3, 20)
    g = C.gen(5)
    a, b = C.randn(g, 3, 4).double(), C.randn(g, 20).double()
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            idx = M.route_tokens(x, 4, score=score, bias=bias)[0].long()

            def loss(v):
                return (float((a * O.route_weights(v, idx, score, renorm, 1.5)).sum())
                        + float((b * O.scores(v, score)[1].mean(0)).sum()))

            got = M.route_tokens_backward(a.float(), x, idx.int(), score=score, renormalize=renorm, scale=1.5,
                                          d_mean_scores=b.float()).double()
            for t in range(3):
                for e in range(20):
                    step = torch.zeros_like(x, dtype=torch.float64)
                    step[t, e] = 1e-5
                    d = (loss(x.double() + step) - loss(x.double() - step)) / 2e-5
                    assert abs(d - float(got[t, e])) < 1e-5


def test_autograd():
    for score, with_bias in (("softmax", False), ("sigmoid", True)):
        x, bias = logits_of(22, 50, 64, torch.bfloat16)
        x.requires_grad_()
        idx, w, mean = M.route_tokens(x, 4, score=score, bias=bias if with_bias else None, mean_scores=True, scale=2.0)
        assert not idx.requires_grad and w.requires_grad and mean.requires_grad
        g = C.gen(6)
        dw, dm = C.randn(g, 50, 4), C.randn(g, 64)
        got, = torch.autograd.grad([w, mean], [x], [dw, dm], retain_graph=True)
        want = M.route_tokens_backward(dw, x.detach(), idx, score=score, scale=2.0, d_mean_scores=dm)
        assert torch.equal(got, want)
        only, = torch.autograd.grad([mean], [x], [dm], retain_graph=True)
        assert torch.equal(only, M.route_tokens_backward(torch.zeros_like(dw), x.detach(), idx, score=score, scale=2.0,
                                                         d_mean_scores=dm))
        only, = torch.autograd.grad([w], [x], [dw])
        assert torch.equal(only, M.route_tokens_backward(dw, x.detach(), idx, score=score, scale=2.0))


def test_captured_and_repeated_calls_give_the_same_bits():
    x, bias = logits_of(23, 3000, 128, torch.bfloat16)
    dw, dm = C.randn(C.gen(7), 3000, 4), C.randn(C.gen(8), 128)

    def call():
        out = M.route_tokens(x, 4, score="sigmoid", bias=bias, mean_scores=True)
        return (*out, M.route_tokens_backward(dw, x, out[0], score="sigmoid", d_mean_scores=dm))

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    keep = x.clone()
    x.copy_(torch.randn_like(x))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, call()))
    x.copy_(keep)


def test_tied_groups():
    """Routers of zeros and of a few values: groups and experts that tie exactly, in every kind of call."""
    g = C.gen(24)
    for x in (torch.zeros(700, 64, device="cuda"), torch.randint(-1, 2, (700, 64), generator=g, device="cuda").float(),
              torch.randint(0, 2, (700, 64), generator=g, device="cuda").float() * 0.25):
        bias = torch.randint(0, 3, (64,), generator=g, device="cuda").float() * 0.125
        for dtype in (torch.float32, torch.bfloat16):
            for b in (None, torch.zeros_like(bias), bias):
                for score in ("softmax", "sigmoid"):
                    for group_score in ("top2", "max"):
                        check(x.to(dtype), 6, score, b, 8, 3, group_score, mean=False)
                    check(x.to(dtype), 6, score, b, mean=False)
