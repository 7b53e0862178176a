"""One MoE block from its operators, training and decoding.

    python examples/moe_block.py

The block is norm -> router -> experts -> gated norm + residual, with a shared
expert beside the routed ones at decode:

* training (`TrainBlock`): bf16 experts as products over the sorted rows; the
  sort, the rows' way there and back, both norms and their gradients are the
  package's (sort_tokens, permute_tokens, unpermute_tokens, norm_before,
  norm_after), through autograd;
* decoding (`DecodeBlock`): FP4 experts by experts_forward, the shared expert by
  matvec on FP4 weights with the SwiGLU applied, norm_after with the next
  block's norm in the same pass.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import block_scaled_moe_expert_gb300 as M  # noqa: E402
from block_scaled_moe_expert_gb300 import workloads as W  # noqa: E402


def route(logits, k):
    """Top-k experts and softmax weights over them."""
    top, idx = torch.topk(logits.float(), k, dim=1)
    return idx.to(torch.int32), torch.softmax(top, dim=1)


class TrainBlock(torch.nn.Module):
    def __init__(self, H, I, E, K, seed=0):
        super().__init__()
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(*shape):
            w = torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5
            return torch.nn.Parameter(w.to(torch.bfloat16))

        self.E, self.K = E, K
        self.router, self.w13, self.w2 = weight(E, H), weight(E, 2 * I, H), weight(E, H, I)
        self.gate = weight(1, H)
        self.norm_in, self.norm_out, self.norm_next = (torch.nn.Parameter(torch.ones(H, device="cuda"))
                                                       for _ in range(3))

    def experts(self, rows, offsets):
        """SwiGLU experts over the groups of rows."""
        out = []
        for e in range(self.E):
            r = rows[offsets[e]:offsets[e + 1]]
            gate, up = (r @ self.w13[e].t()).chunk(2, dim=1)
            out.append((torch.nn.functional.silu(gate) * up) @ self.w2[e].t())
        return torch.cat(out + [rows[offsets[self.E]:]])

    def forward(self, x):
        y = M.norm_before(x, self.norm_in)
        idx, w = route(y @ self.router.t(), self.K)
        plan = M.sort_tokens(idx, self.E, row_align=16)
        rows = M.permute_tokens(y, plan)
        h = M.unpermute_tokens(self.experts(rows, plan.offsets.tolist()), plan, w)
        gate = y @ self.gate.t()  # one logit a token
        return M.norm_after(x, h, self.norm_out, gate=gate, gate_act="sigmoid", alpha=0.5,
                            next_weight=self.norm_next)


class DecodeBlock:
    def __init__(self, H, I, E, K, seed=0):
        wl = W.Workload("decode_block", 1, H, I, E, K, "fp4", "softmax", seed=seed)
        self.K = K
        self.experts = M.prepare_weights(W.make_weights(wl, "cuda"))
        shared = W.make_weights(W.scaled(wl, E=1, K=1, seed=seed + 1), "cuda")
        self.shared_in = M.prepare_matvec(dict(fmt="fp4", N=2 * I, K=H, w=shared["w13"][0],
                                               w_scale=shared["w13_scale"][0]), swiglu=True)
        self.shared_out = M.prepare_matvec(dict(fmt="fp4", N=H, K=I, w=shared["w2"][0], w_scale=shared["w2_scale"][0]))
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 2)
        self.router = (torch.randn(E, H, generator=g, device="cuda") * H ** -0.5).to(torch.bfloat16)
        self.norm_in, self.norm_out, self.norm_next = (torch.ones(H, device="cuda") for _ in range(3))

    def __call__(self, x):
        y = M.norm_before(x, self.norm_in)
        idx, w = route(y @ self.router.t(), self.K)
        h = M.experts_forward(y, idx, w, self.experts)
        h += M.matvec(M.matvec(y, self.shared_in), self.shared_out)
        return M.norm_after(x, h, self.norm_out, next_weight=self.norm_next)


def train(steps=5, T=512, H=256, I=128, E=8, K=2):
    """Losses of a few steps that fit the block's output to a target."""
    block = TrainBlock(H, I, E, K)
    opt = torch.optim.SGD(block.parameters(), lr=0.3)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    x, target = (torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        r, y = block(x)
        loss = ((y - target).float() ** 2).mean()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def decode(steps=4, T=4, H=512, I=256, E=16, K=2):
    """The residual stream after a few passes through one block."""
    block = DecodeBlock(H, I, E, K)
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    for _ in range(steps):
        x, y = block(x)
    return x, y


if __name__ == "__main__":
    print("training losses:", [f"{v:.4f}" for v in train()])
    x, y = decode()
    print("decoded rows:", tuple(x.shape), "rms", f"{float((x.float() ** 2).mean().sqrt()):.4f}")
