"""GPU: routing where groups have no available expert or an infinite value, and
near ties between the others, against the 64-bit oracle."""
import math

import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from oracle import block as O
from tests import block_cases as C
from tests.test_gpu_route_tokens import check, logits_of

pytestmark = pytest.mark.gpu

STEP = 1.0 + 2.0 ** -23


def near_ties(seed, T, E, groups, score, shut=()):
    """Logits and a bias that cancels the scores: the groups' two best within a few fp32 steps of all the others',
    the rest of a group in clear steps below. shut: experts with logits of -inf."""
    x, _ = logits_of(seed, 1, E)
    x[:, list(shut)] = -math.inf
    below = torch.arange(E, device="cuda") % (E // groups) // 2
    bias = (0.75 - O.scores(x, score)[0][0] - 0.01 * below).float()
    return x + 1e-6 * C.randn(C.gen(seed + 1), T, E), bias


SHAPES = [(256, 8, 4), (64, 4, 2), (96, 3, 1), (32, 16, 5), (512, 16, 12)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["top2", "max"])
@pytest.mark.parametrize("E,groups,top_groups", SHAPES)
def test_near_ties_beside_masked_groups(E, groups, top_groups, score, group_score):
    size, K = E // groups, 2 * top_groups
    for shut in ([groups - 1], [0], list(range(0, groups, 4))[: groups - top_groups - 1]):
        experts = [g * size + i for g in shut for i in range(size)]
        x, bias = near_ties(E + groups, 3000, E, groups, score, experts)
        check(x, K, score, bias, groups, top_groups, group_score, mean=False)
        x, bias = near_ties(E + groups, 3000, E, groups, score)
        for low in (-math.inf, torch.finfo(torch.float32).min):
            closed = bias.clone()
            closed[experts] = low
            check(x, K, score, closed, groups, top_groups, group_score, mean=False)


def test_groups_of_the_lowest_bias_come_before_masked_ones():
    """Sums of two biases of the type's lowest value pass its range; such groups are available all the same."""
    low = torch.finfo(torch.float32).min
    x, _ = logits_of(3, 50, 64)
    for score in ("softmax", "sigmoid"):
        for masked in ((0, 1), (5, 2), (0, 7)):
            bias = torch.full((64,), low, device="cuda")
            bias[24:32] = 0.0
            for g in masked:
                bias[8 * g:8 * g + 8] = -math.inf
            for top_groups in (2, 3, 6, 7):
                check(x, 8, score, bias, 8, top_groups, "top2", mean=False)


def test_neighbouring_logits_beside_a_masked_group():
    """Maxima of two groups one fp32 step apart, the lower group's index the lower one."""
    x = torch.full((4, 32), -1.0, device="cuda")
    x[:, 3], x[:, 9] = 1.0, STEP
    x[1, 24:] = -math.inf
    x[2, 16:] = -math.inf
    x[3, 31] = -math.inf
    for score in ("softmax", "sigmoid"):
        assert check(x, 1, score, None, 4, 1, "max", mean=False)[0].tolist() == [[9]] * 4


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["top2", "max"])
def test_near_ties_beside_an_infinite_group(score, group_score):
    """A bias of +inf takes its expert's group first; the rest is as near as before."""
    for E, groups, top_groups in SHAPES:
        x, bias = near_ties(E, 3000, E, groups, score)
        for first in ([5], [5, E - 1], [5, 6, E - 1]):
            b = bias.clone()
            b[first] = math.inf
            check(x, 2 * top_groups, score, b, groups, top_groups, group_score, mean=False)


def test_neighbouring_logits_beside_an_infinite_one():
    """By the logits: the second group of two, whose maxima are one fp32 step apart."""
    x = torch.full((3, 32), -1.0, device="cuda")
    x[:, 3], x[:, 9], x[:, 30] = 1.0, STEP, math.inf
    x[1, 31] = math.inf
    idx, w = M.route_tokens(x, 2, score="sigmoid", num_groups=4, top_groups=2, group_score="max")
    assert idx.tolist() == [[30, 9], [30, 31], [30, 9]]
    assert torch.allclose(w.sum(1), torch.ones(3, device="cuda"))
    idx, w = M.route_tokens(x[:, :31].contiguous(), 2, score="sigmoid")
    assert idx.tolist() == [[30, 9]] * 3


def test_infinite_logits_under_softmax():
    """A logit of +inf has no softmax: the token's weights and the mean scores are NaN, as its scores are; where
    scores choose, the choice is that without its expert (like a NaN's), where logits do, it is the largest."""
    for dtype in C.DTYPES:
        x, bias = logits_of(11, 40, 64, dtype)
        x[3, 5] = x[6, 60] = x[9, 0] = math.inf
        x[9, 1] = math.inf
        x[12] = math.inf
        bad = torch.zeros(40, dtype=torch.bool, device="cuda")
        bad[[3, 6, 9, 12]] = True
        rest = torch.where(x == math.inf, -math.inf, x.float())
        for renorm in (True, False):
            for b, groups, top in ((bias, 1, 1), (bias, 8, 3), (bias, 4, 4), (None, 8, 3)):
                for group_score in ("top2", "max"):
                    if b is None and group_score == "max":
                        continue
                    idx, w, mean = M.route_tokens(x, 6, bias=b, num_groups=groups, top_groups=top, group_score=group_score,
                                                  renormalize=renorm, mean_scores=True)
                    assert torch.equal(idx.long(), O.choose(rest, 6, "softmax", b, groups, top, group_score))
                    assert torch.equal(w.isnan().all(1), bad) and torch.equal(w.isnan().any(1), bad)
                    assert bool(mean.isnan().all())
                    want = O.route_weights(rest, idx.long(), "softmax", renorm, 1.0)[~bad]
                    assert torch.allclose(w[~bad].double(), want, rtol=1e-5, atol=1e-30)
            idx, w, mean = M.route_tokens(x, 6, renormalize=renorm, mean_scores=True)
            assert idx[3, 0] == 5 and idx[6, 0] == 60 and idx[9, :2].tolist() == [0, 1]
            assert torch.equal(w.isnan().all(1), bad) and torch.equal(w.isnan().any(1), bad) and bool(mean.isnan().all())


def neighbours(value, low, high, count):
    """Index pairs (i, j) of `value` [N] that are next to each other in order and between low and high apart."""
    order = value.argsort()
    gap = value[order][1:] - value[order][:-1]
    at = ((gap >= low) & (gap <= high)).nonzero().flatten()
    at = at[:: max(1, at.numel() // count)][:count]
    assert at.numel() >= count // 2
    return order[at], order[at + 1]


def test_bias_that_cancels_the_score():
    """bias = -score in fp32 leaves keys of 1e-8, whose error is that of the scores: neighbours 1e-15 to 8e-15
    apart, 5 to 40 times the error of their 64-bit values (a sigmoid 2^-53, a sum that is exact)."""
    x = C.randn(C.gen(30), 400000, scale=1.5)
    s = O.scores(x[:, None], "sigmoid")[0][:, 0]
    i, j = neighbours(s - s.float().double(), 1e-15, 8e-15, 320)
    for a, b in ((i, j), (j, i)):
        # 16 pairs a call, each pair's expert with the smaller or the larger key first
        for k in range(0, i.numel() - 15, 16):
            row = x[torch.stack([a[k:k + 16], b[k:k + 16]], 1).flatten()][None]
            bias = -O.scores(row, "sigmoid")[0][0].float()
            for K in (31, 32):
                check(row, K, "sigmoid", bias, mean=False)
            row, bias = torch.cat([row, row], 1), torch.cat([bias, bias - 0.25])
            check(row, 31, "sigmoid", bias, mean=False)
            check(row, 20, "sigmoid", bias, 2, 1, "max", mean=False)


def test_softmax_bias_that_cancels_the_score():
    """The same for scores of some 1/64 that share a sum: 1e-17 to 1e-15 apart, 64-bit values good to 1e-17 / 5."""
    x = C.randn(C.gen(31), 60000, 64)
    s = O.scores(x, "softmax")[0]
    top = (s - s.float().double()).sort(1, descending=True)[0][:, :33]
    gap = (top[:, :-1] - top[:, 1:]).amin(1)
    rows = ((gap >= 1e-17) & (gap <= 1e-15)).nonzero().flatten()[:80]
    assert rows.numel() == 80
    for r in rows.tolist():
        check(x[r:r + 1], 32, "softmax", -s[r].float(), mean=False)


def test_equal_experts_do_not_hide_a_larger_one():
    """Experts with the same logit at the border of the choice, and one a step of fp32 above them further on."""
    for E in (32, 60, 256, 512):
        for K in (1, 2, 5):
            for dtype, step in ((torch.float32, STEP), (torch.float32, 1.0 + 2.0 ** -22), (torch.bfloat16, 1.0 + 2.0 ** -7)):
                x = torch.full((6, E), -1.0, device="cuda")
                x[:5, : E // 2 : 2] = 1.0
                for t, at in enumerate((E - 1, E // 2, E // 2 - 1, 1)):
                    x[t, at] = step
                x[4, E - 7:] = step
                x = x.to(dtype)
                for score in ("softmax", "sigmoid"):
                    check(x, K, score, None, mean=False)
                    check(x, K, score, torch.zeros(E, device="cuda"), mean=False)
                    check(x, min(K, E // 2), score, None, 2, 1, "max", mean=False)
                    check(x, min(K, E // 2), score, torch.full((E,), 0.25, device="cuda"), 4, 2, "top2", mean=False)


def test_group_sums_that_cancel():
    """Groups whose two best biased scores cancel to 1e-8: sums 3e-15 to 2e-14 apart, 64-bit ones good to 5e-16."""
    x = C.randn(C.gen(32), 200000, 2, scale=1.5)
    s = O.scores(x, "sigmoid")[0]
    low = -(0.5 + s.sum(1)).float()
    i, j = neighbours(s.sum(1) + 0.5 + low.double(), 3e-15, 2e-14, 200)
    bias = torch.stack([torch.full_like(low, 0.5), low], 1)
    for a, b in ((i, j), (j, i)):
        rows, biases = torch.cat([x[a], x[b]], 1), torch.cat([bias[a], bias[b]], 1)
        for r in range(rows.shape[0]):
            check(rows[r:r + 1], 1, "sigmoid", biases[r], 2, 1, "top2", mean=False)


def test_softmax_group_sums_that_cancel():
    """The same for 32 groups of two whose scores share a sum, with the border between two near ones."""
    x = C.randn(C.gen(33), 400000, 64)
    s = O.scores(x, "softmax")[0].view(-1, 32, 2)
    low = -(0.5 + s.sum(2)).float()
    value, order = (s.sum(2) + 0.5 + low.double()).sort(1, descending=True)
    gap = (value[:, :-1] - value[:, 1:])[:, :16]
    rows, at = ((gap >= 2e-15) & (gap <= 2e-14)).nonzero(as_tuple=True)
    assert rows.numel() >= 20
    for r, p in list(zip(rows.tolist(), at.tolist()))[:80]:
        bias = torch.stack([torch.full_like(low[r], 0.5), low[r]], 1).flatten()
        check(x[r:r + 1], 2 * (p + 1), "softmax", bias, 32, p + 1, "top2", mean=False)


def test_saturated_scores_with_a_bias():
    """Sigmoids next to 1 whose biased keys share a pair of floats while 64 bits tell them apart: steps of
    5 and more units of 2^-52. The larger logits have the larger indices."""
    steps = torch.tensor([32.0, 33.0, 34.0], device="cuda")
    for b in (0.1, 0.7, -0.3, 0.9):
        bias = torch.full((24,), b, device="cuda")
        x = steps.repeat_interleave(8)[None] + 0.0
        for K in (4, 12, 23):
            check(x, K, "sigmoid", bias, mean=False)
            check(x.flip(1), K, "sigmoid", bias, mean=False)
        check(x, 4, "sigmoid", bias, 3, 1, "max", mean=False)
        check(x, 4, "sigmoid", bias, 3, 1, "top2", mean=False)
        check(x, 4, "sigmoid", bias, 6, 3, "top2", mean=False)


@pytest.mark.parametrize("E,groups,top_groups", [(510, 17, 4), (512, 16, 5), (512, 1, 1), (256, 8, 3), (60, 1, 1)])
def test_sums_whose_terms_all_round_down(E, groups, top_groups):
    """Softmax sums of one term of 1 a lane and terms just below the half of its last place, which fp32 drops: scores
    come out too large by a step for every term. Biases put small scores next to large ones, from half of that to
    twice it away."""
    size = E // groups
    x = torch.full((400, E), math.log(0.99 * 2.0 ** -24), device="cuda")
    x[:, :: size if groups > 1 else 8] = 0.0
    s = O.scores(x[:1], "softmax")[0][0]
    small = s < 0.5 * s.max()
    shift = torch.linspace(-4, 4, E, device="cuda", dtype=torch.float64)[torch.randperm(E, generator=C.gen(34), device="cuda")]
    bias = torch.where(small, s.max() - s, 0.0) + s.max() * E * 2.0 ** -24 * shift
    bias = torch.where(torch.arange(E, device="cuda") % size < 5, bias, bias - 0.1).float()
    noise = torch.where(x == 0, 0.0, C.randn(C.gen(35), 400, E, scale=1e-3))
    for group_score in ("top2", "max"):
        check(x - noise.abs(), 8, "softmax", bias, groups, top_groups, group_score, mean=False)


def test_mean_scores_of_many_tokens():
    """The error of a mean does not grow with the number of tokens: 64 roundings of 2^-24 for thousands of tokens a
    lane, beside those of a score, the same in every row: 4 + 3 D of an exponential (2^-22 and its argument's), as much
    again and 21 of the sum over the experts, 3 of the quotient (a sigmoid's own 8 are fewer). Rows share their memory,
    so that there may be many."""
    for E, T, values in ((256, 1 << 22, (0.0, 0.3, -0.2)), (512, 1 << 21, (0.1, -0.05, 0.2)), (8, 1 << 25, (0.0, 0.7, -0.4))):
        row = torch.tensor(values, device="cuda").repeat(E // 3 + 1)[:E]
        for score in ("softmax", "sigmoid"):
            mean = M.route_tokens(row.expand(T, E), 1, score=score, mean_scores=True)[2].double()
            p = O.scores(row[None], score)[1][0]
            D = float(row.max() - row.min())
            tol = (2 * (4 + 3 * D) + 24 + 64) * 2.0 ** -24
            assert bool(((mean - p).abs() <= tol * p).all()), float(((mean - p).abs() / p).max() / tol)
