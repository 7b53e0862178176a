"""GPU: the example block, and its decode step against the 64-bit oracles."""
import importlib.util
import os

import pytest
import torch

import block_scaled_moe_expert_gb300 as M
from oracle import block as O
from tests import block_cases as C

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block_example", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_lowers_the_loss_the_same_way_each_time(example):
    losses = example.train()
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert losses[0] == example.train(steps=1)[0]


def test_training_step_reaches_every_parameter(example):
    block = example.TrainBlock(128, 64, 4, 2)
    r, y = block(C.randn(C.gen(3), 64, 128, dtype=torch.bfloat16))
    (r.float().square().mean() + y.float().square().mean() * y.float().mean()).backward()
    for name, p in block.named_parameters():
        assert p.grad is not None and p.grad.isfinite().all() and p.grad.abs().max() > 0, name


def test_decode_block_is_its_operators(example):
    block = example.DecodeBlock(512, 256, 16, 2)
    x = C.randn(C.gen(5), 4, 512, dtype=torch.bfloat16)
    r, y = block(x)
    # the block's own intermediate results through the oracle of each step
    n = M.norm_before(x, block.norm_in)
    e = O.norm(x, block.norm_in, 1e-6)
    C.check(n, e, e.abs(), 80)
    idx, w = example.route(n @ block.router.t(), 2)
    h = M.experts_forward(n, idx, w, block.experts) + M.matvec(M.matvec(n, block.shared_in), block.shared_out)
    er = O.norm_after(x, h, block.norm_out, None, "none", 1.0, 1.0, 1e-6, 0.0, True)
    mr = O.norm_after(x, h, block.norm_out, None, "none", 1.0, 1.0, 1e-6, 0.0, True, mag=True)
    C.check(r, er, mr, 80)
    ey = O.norm(er, block.norm_next, 1e-6)
    s = 1 / torch.sqrt((er * er).mean(1, keepdim=True) + 1e-6)
    C.check(y, ey, s * mr + ey.abs() * (1 + (mr * mr).mean(1, keepdim=True).sqrt() * s), 80)
