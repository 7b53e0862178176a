"""Timing cases of the operators around the experts forward.

Three families: tokens sorted by expert and back (sort_tokens, permute_tokens,
unpermute_tokens and their gradients), the norms before and after a block with
its gate and residual scale (norm_before, norm_after and their gradients), and
matrix-vector products with 4-bit weights (matvec). `run` computes a case with
elementary torch operations in 32 bits, or, where `own` is true, through the
package's entry points; `exact` computes it in 64 bits from the definitions.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ESIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _named(name, **case):
    return case if name is None else dict(name=name, **case)


def _route(name, op, T, H, E, K, dtype, align, weighted, skip):
    return _named(name, op=op, T=T, H=H, E=E, K=K, dtype=dtype, align=align, weighted=weighted, skip=skip)


def _norm(name, op, T, H, dtype, wdtype, gate, act, post, nxt, alpha, beta):
    return _named(name, op=op, T=T, H=H, dtype=dtype, wdtype=wdtype, gate=gate, act=act, post=post, next=nxt,
                  alpha=alpha, beta=beta)


def _mv(name, T, N, K, fmt, group, zero, swiglu, dtype):
    return _named(name, op="matvec", T=T, N=N, K=K, fmt=fmt, group=group, zero=zero, swiglu=swiglu, dtype=dtype)


def listed():
    return [
        # one decode step of a few sequences: the call's latency
        _route("dispatch_decode", "dispatch", 4, 7168, 256, 8, "bf16", 1, False, 0.0),
        # a prefill or training batch into groups of whole 128-row tiles, with skipped slots
        _route("dispatch_prefill", "dispatch", 8192, 7168, 256, 8, "bf16", 128, False, 0.05),
        # the way back of a large batch, routing weights applied
        _route("combine_prefill", "combine", 8192, 2880, 128, 4, "bf16", 128, True, 0.0),
        # training: the gradient of the way back, rows and weights
        _route("combine_backward_train", "combine_backward", 4096, 4096, 8, 2, "bf16", 16, True, 0.0),
        # training in 32 bits with an odd width and weights applied on the way in
        _route("dispatch_backward_odd", "dispatch_backward", 3001, 1001, 60, 5, "fp32", 1, True, 0.1),
        # one token's norm before the block
        _norm("norm_before_decode", "norm_before", 1, 7168, "bf16", "fp32", "none", "none", True, False, 1.0, 1.0),
        # after the block of a prefill: norm, channel gate, residual scale and the next block's norm in one pass
        _norm("norm_after_prefill", "norm_after", 8192, 7168, "bf16", "bf16", "channel", "none", True, True, 0.5,
              1.0),
        # its training direction, a gate logit for each token
        _norm("norm_after_backward_train", "norm_after_backward", 8192, 4096, "bf16", "bf16", "token", "sigmoid",
              True, True, 0.7, 0.9),
        # training: an odd width in fp16
        _norm("norm_before_backward_odd", "norm_before_backward", 2777, 2881, "fp16", "fp32", "none", "none", True,
              False, 1.0, 1.0),
        # the shared expert's gate and up product of one token, SwiGLU applied
        _mv("matvec_shared_expert", 1, 4096, 7168, "fp4", 32, False, True, "bf16"),
        # an output head of one token: the longest stream of weights
        _mv("matvec_head", 1, 131072, 4096, "fp4", 32, False, False, "bf16"),
        # a dense product for the sequences of a small batch, zero points, odd number of rows
        _mv("matvec_batch_int4", 7, 28671, 4096, "int4", 128, True, False, "fp16"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n % 1024 == 0 and n < hi else n  # round sizes are in the list


def _width(rng, lo, hi):
    """A row width: an odd multiple of 64 or of 8, or any odd number."""
    step = rng.choice([64, 64, 8, 1])
    n = _log_int(rng, lo, hi) // step
    return max(n | 1, 1) * step


def draw(rng):
    """Another case of the ranges: tokens 1..16384, widths 64..8192, 8..512 experts, 1..8 of them a token."""
    op = rng.choice(["dispatch", "combine", "dispatch_backward", "combine_backward", "norm_before", "norm_after",
                     "norm_before_backward", "norm_after_backward", "matvec", "matvec"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "matvec":
        K = 32 * (_log_int(rng, 128, 16384) // 32 | 1)
        N = min(_log_int(rng, 64, 65536), (1 << 28) // K)
        fmt = rng.choice(["fp4", "fp4", "int4"])
        swiglu = rng.random() < 0.3
        group = 32 if fmt == "fp4" else rng.choice([32, 64, 128])
        zero = fmt == "int4" and rng.random() < 0.5
        return _mv(None, rng.choice([1, 1, 2, 3, 5, 8, 13, 16]), N // 2 * 2 if swiglu else N, K, fmt, group, zero,
                   swiglu, rng.choice(["bf16", "fp16"]))
    T, H = _log_int(rng, 1, 16384), _width(rng, 64, 8192)
    if op.startswith("norm"):
        T = max(1, min(T, (3 << 24) // H))
        after = op.startswith("norm_after")
        gate = rng.choice(["none", "channel", "token", "element"]) if after else "none"
        act = rng.choice(["none", "sigmoid", "tanh"]) if gate != "none" else "none"
        nxt = after and rng.random() < 0.5
        post = rng.random() < 0.8 if after else True
        return _norm(None, op, T, H, dtype, rng.choice([dtype, "fp32"]), gate, act, post, nxt,
                     rng.choice([1.0, 0.25]) if after else 1.0, rng.choice([1.0, 0.8]) if after else 1.0)
    E = rng.choice([8, 16, 60, 64, 128, 256, 512])
    K = rng.randint(1, 8)
    align = rng.choice([1, 16, 128])
    while _capacity(T * K, E, align) * H * ESIZE[dtype] > 1 << 30:
        T = T // 2 + 1
        H = (H // 2 | 1) if H > 4096 else H
    weighted = rng.random() < 0.5 if op.startswith("dispatch") else rng.random() < 0.9
    return _route(None, op, T, H, E, K, dtype, align, weighted, rng.choice([0.0, 0.05]))


def _capacity(S, E, align):
    return (S + min(E, S) * (align - 1)) // align * align


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# ------------------------------------------------------------------- inputs

def _routing(case, seed):
    """Router choices over experts of uneven popularity: K distinct a token, some slots skipped; softmax weights."""
    g = _gen(seed, 1)
    T, E, K = case["T"], case["E"], case["K"]
    logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    top, idx = torch.topk(logits, K, dim=1)
    idx = idx.to(torch.int32)
    if case["skip"] > 0:
        drop = torch.rand(T, K, generator=g, device="cuda") < case["skip"]
        idx = torch.where(drop, torch.full_like(idx, -1), idx)
    return idx.contiguous(), torch.softmax(top, dim=1).contiguous()


def _route_inputs(case, seed):
    g = _gen(seed, 2)
    dt, T, H = DTYPES[case["dtype"]], case["T"], case["H"]
    M = _capacity(T * case["K"], case["E"], case["align"])
    idx, w = _routing(case, seed)
    s = dict(idx=idx, w=w if case["weighted"] else None)
    op = case["op"]
    if op in ("dispatch", "dispatch_backward"):
        s["hidden"] = _randn(g, T, H, dtype=dt)
    if op in ("combine", "combine_backward"):
        s["rows"] = _randn(g, M, H, dtype=dt)
    if op == "dispatch_backward":
        s["drows"] = _randn(g, M, H, dtype=dt, scale=0.1)
    if op == "combine_backward":
        s["dout"] = _randn(g, T, H, dtype=dt, scale=0.1)
    return s


def _norm_inputs(case, seed):
    g = _gen(seed, 3)
    dt, wt, T, H = DTYPES[case["dtype"]], DTYPES[case["wdtype"]], case["T"], case["H"]
    after, back = "after" in case["op"], "backward" in case["op"]

    def weight():
        return (1.0 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(wt)

    s = dict(weight=weight() if case["post"] else None)
    s["next_weight"] = weight() if case["next"] else None
    shape = {"none": None, "channel": (H,), "token": (T, 1), "element": (T, H)}[case["gate"]]
    s["gate"] = None if shape is None else _randn(g, *shape, dtype=dt)
    if after:
        s["h"] = _randn(g, T, H, dtype=dt, scale=3.0)
    if back:
        s["dr" if after else "dy"] = _randn(g, T, H, dtype=dt, scale=0.1)
        if case["next"]:
            s["dy"] = _randn(g, T, H, dtype=dt, scale=0.1)
            s["r"] = _randn(g, T, H, dtype=dt, scale=2.0)
        if not after:
            s["x"] = _randn(g, T, H, dtype=dt, scale=2.0)
    else:
        s["x"] = _randn(g, T, H, dtype=dt, scale=2.0)
    return s


def _matvec_inputs(case, seed):
    g = _gen(seed, 4)
    N, K, G = case["N"], case["K"], -(-case["K"] // case["group"])
    s = dict(x=_randn(g, case["T"], K, dtype=DTYPES[case["dtype"]]))
    s["w"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    if case["fmt"] == "fp4":
        s["w_scale"] = torch.randint(117, 122, (N, G), generator=g, device="cuda", dtype=torch.uint8)
    else:
        s["w_scale"] = (0.004 + 0.012 * torch.rand(N, G, generator=g, device="cuda")).to(DTYPES[case["dtype"]])
    s["w_zero"] = None
    if case["zero"]:
        s["w_zero"] = torch.randint(6, 11, (N, G), generator=g, device="cuda", dtype=torch.uint8)
    return s


def _inputs(case, seed):
    if case["op"] == "matvec":
        return _matvec_inputs(case, seed)
    return _norm_inputs(case, seed) if case["op"].startswith("norm") else _route_inputs(case, seed)


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:
        import block_scaled_moe_expert_gb300 as M
        state["M"] = M
        if case["op"] == "matvec":
            weights = dict(fmt=case["fmt"], N=case["N"], K=case["K"], w=state["w"], w_scale=state["w_scale"])
            if case["fmt"] == "int4":
                weights.update(group=case["group"], w_zero=state["w_zero"])
            state["prepared"] = M.prepare_matvec(weights, swiglu=case["swiglu"])
    if case["op"] in ("combine", "combine_backward", "dispatch_backward"):
        # the plan of the same step's sort
        state["plan"] = (state["M"].sort_tokens(state["idx"], case["E"], row_align=case["align"]) if own
                         else _plain_sort(state["idx"], case["E"], case["align"]))
    return state


# --------------------------------------------------------------- plain forms

def _plain_sort(idx, E, align):
    """(counts, offsets, inv, row_slot) of the stable grouping by expert."""
    T, K = idx.shape
    S = T * K
    key = idx.reshape(-1).long()
    key = torch.where((key >= 0) & (key < E), key, torch.full_like(key, E))
    order = torch.argsort(key, stable=True)
    count = torch.zeros(E + 1, dtype=torch.long, device=idx.device).index_add_(0, key, torch.ones_like(key))
    padded = (count[:E] + align - 1) // align * align
    offsets = torch.zeros(E + 1, dtype=torch.long, device=idx.device)
    offsets[1:] = torch.cumsum(padded, 0)
    start = torch.cumsum(count, 0) - count
    skey = key[order]
    row = offsets[skey] + torch.arange(S, device=idx.device) - start[skey]
    row = torch.where(skey < E, row, torch.full_like(row, -1))
    inv = torch.empty(S, dtype=torch.long, device=idx.device)
    inv[order] = row
    M = _capacity(S, E, align)
    slots = torch.full((M + 1,), -1, dtype=torch.long, device=idx.device)
    slots[torch.where(row >= 0, row, torch.full_like(row, M))] = order
    i32 = torch.int32
    return count[:E].to(i32), offsets.to(i32), inv.to(i32).reshape(T, K), slots[:M].to(i32)


def _gather_rows(rows, inv_k):
    """fp32 rows of one k's slots; zeros where the slot is skipped."""
    r = rows[inv_k.clamp(min=0).long()].float()
    return torch.where((inv_k >= 0)[:, None], r, torch.zeros_like(r))


def _place_rows(x, w, plan, M, dtype):
    """rows[inv[t, k]] = w[t, k] x[t], zeros elsewhere."""
    slot = plan[3].long()
    K = plan[2].shape[1]
    r = x[slot.clamp(min=0) // K].float()
    if w is not None:
        r = r * w.reshape(-1)[slot.clamp(min=0)][:, None]
    return torch.where((slot >= 0)[:, None], r, torch.zeros_like(r)).to(dtype)


def _sum_rows(rows, w, plan):
    out = 0.0
    for k in range(plan[2].shape[1]):
        r = _gather_rows(rows, plan[2][:, k])
        out = out + (r if w is None else r * w[:, k:k + 1])
    return out.to(rows.dtype)


def _row_dots(x, rows, plan):
    xf = x.float()
    return torch.stack([(xf * _gather_rows(rows, plan[2][:, k])).sum(1) for k in range(plan[2].shape[1])], dim=1)


EPS = 1e-6


def _act(name, v):
    return torch.sigmoid(v) if name == "sigmoid" else torch.tanh(v) if name == "tanh" else v


def _act_grad(name, a):
    """Derivative of the gate's activation from its value."""
    return a * (1 - a) if name == "sigmoid" else 1 - a * a if name == "tanh" else torch.ones_like(a)


def _plain_norm(v, w):
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return y if w is None else y * w.float()


def _plain_norm_backward(dy, v, w):
    inv = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    n = v * inv
    dn = dy * w.float()
    return inv * (dn - n * (dn * n).mean(1, keepdim=True)), (dy * n).sum(0).to(w.dtype)


def _plain_norm_after(s, c):
    z = s["h"].float()
    if c["post"]:
        z = _plain_norm(z, s["weight"])
    if s["gate"] is not None:
        z = z * _act(c["act"], s["gate"].float())
    r = c["beta"] * s["x"].float() + c["alpha"] * z
    if not c["next"]:
        return r.to(s["x"].dtype)
    return r.to(s["x"].dtype), _plain_norm(r, s["next_weight"]).to(s["x"].dtype)


def _plain_norm_after_backward(s, c):
    dt = s["h"].dtype
    G, dnext = s["dr"].float(), None
    if c["next"]:
        d, dnext = _plain_norm_backward(s["dy"].float(), s["r"].float(), s["next_weight"])
        G = G + d
    h = s["h"].float()
    z = _plain_norm(h, s["weight"]) if c["post"] else h
    dz, dgate = c["alpha"] * G, None
    if s["gate"] is not None:
        a = _act(c["act"], s["gate"].float())
        full = dz * z * _act_grad(c["act"], a)
        dgate = (full if c["gate"] == "element" else full.sum(0) if c["gate"] == "channel"
                 else full.sum(1, keepdim=True)).to(dt)
        dz = dz * a
    dh, dweight = dz, None
    if c["post"]:
        dh, dweight = _plain_norm_backward(dz, h, s["weight"])
    return (c["beta"] * G).to(dt), dh.to(dt), dweight, dgate, dnext


def _plain_matvec(s, c):
    lo, hi = (s["w"] & 15).int(), (s["w"] >> 4).int()
    u = torch.stack([lo, hi], dim=2).reshape(c["N"], c["K"])
    if c["fmt"] == "fp4":
        W = torch.tensor(E2M1, device="cuda")[u]
        scale = torch.pow(2.0, s["w_scale"].float() - 127.0)
    else:
        W = u.float()
        zero = 8.0 if s["w_zero"] is None else _per_column(s["w_zero"].float(), c)
        W = W - zero
        scale = s["w_scale"].float()
    y = s["x"].float() @ (W * _per_column(scale, c)).t()
    if c["swiglu"]:
        g, up = y[:, :c["N"] // 2], y[:, c["N"] // 2:]
        y = g * torch.sigmoid(g) * up
    return y.to(s["x"].dtype)


def _per_column(v, c):
    return v.repeat_interleave(c["group"], dim=1)[:, :c["K"]]


# ----------------------------------------------------------------------- run

def _present(out):
    """The outputs that the case has: no weight, gate or norm, no gradient of it."""
    return tuple(o for o in out if o is not None) if isinstance(out, tuple) else out


def run(state):
    c, s = state["case"], state
    return _present(_run_own(s["M"], s, c, c["op"]) if own else _run_plain(s, c, c["op"]))


def _run_plain(s, c, op):
    if op == "dispatch":
        plan = _plain_sort(s["idx"], c["E"], c["align"])
        return (_place_rows(s["hidden"], s["w"], plan, plan[3].numel(), s["hidden"].dtype),) + plan
    if op == "combine":
        return _sum_rows(s["rows"], s["w"], s["plan"])
    if op == "dispatch_backward":
        dx = _sum_rows(s["drows"], s["w"], s["plan"])
        return dx, _row_dots(s["hidden"], s["drows"], s["plan"]) if c["weighted"] else None
    if op == "combine_backward":
        drows = _place_rows(s["dout"], s["w"], s["plan"], s["rows"].shape[0], s["rows"].dtype)
        return drows, _row_dots(s["dout"], s["rows"], s["plan"]) if c["weighted"] else None
    if op == "norm_before":
        return _plain_norm(s["x"].float(), s["weight"]).to(s["x"].dtype)
    if op == "norm_before_backward":
        dx, dw = _plain_norm_backward(s["dy"].float(), s["x"].float(), s["weight"])
        return dx.to(s["x"].dtype), dw
    if op == "norm_after":
        return _plain_norm_after(s, c)
    if op == "norm_after_backward":
        return _plain_norm_after_backward(s, c)
    return _plain_matvec(s, c)


def _run_own(M, s, c, op):
    if op == "dispatch":
        plan = M.sort_tokens(s["idx"], c["E"], row_align=c["align"])
        return M.permute_tokens(s["hidden"], plan, s["w"]), plan.counts, plan.offsets, plan.inv, plan.row_slot
    if op == "combine":
        return M.unpermute_tokens(s["rows"], s["plan"], s["w"])
    if op == "dispatch_backward":
        return M.permute_tokens_backward(s["drows"], s["plan"], s["hidden"], s["w"])
    if op == "combine_backward":
        return M.unpermute_tokens_backward(s["dout"], s["plan"], s["rows"], s["w"])
    if op == "norm_before":
        return M.norm_before(s["x"], s["weight"], eps=EPS)
    if op == "norm_before_backward":
        return M.norm_before_backward(s["dy"], s["x"], s["weight"], eps=EPS)
    if op == "norm_after":
        return M.norm_after(s["x"], s["h"], s["weight"], gate=s["gate"], gate_act=c["act"], alpha=c["alpha"],
                            beta=c["beta"], eps=EPS, norm=c["post"], next_weight=s["next_weight"])
    if op == "norm_after_backward":
        return M.norm_after_backward(s["dr"], s["h"], s["weight"], gate=s["gate"], gate_act=c["act"],
                                     alpha=c["alpha"], beta=c["beta"], eps=EPS, norm=c["post"], dy=s.get("dy"),
                                     r=s.get("r"), next_weight=s["next_weight"])
    return M.matvec(s["x"], s["prepared"])


# ---------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "matvec":
        es, G = ESIZE[c["dtype"]], -(-c["K"] // c["group"])
        scale = 1 if c["fmt"] == "fp4" else 2 + (1 if c["zero"] else 0)
        out = c["N"] // 2 if c["swiglu"] else c["N"]
        return dict(bytes=c["N"] * c["K"] // 2 + c["N"] * G * scale + c["T"] * (c["K"] + out) * es,
                    flops=2 * c["T"] * c["N"] * c["K"])
    es = ESIZE[c["dtype"]]
    if c["op"].startswith("norm"):
        n = c["T"] * c["H"]
        rows = {"norm_before": 2, "norm_after": 3, "norm_before_backward": 3, "norm_after_backward": 3}[c["op"]]
        if c["op"] == "norm_after_backward":  # dy, r and dx; without the next norm dx is beta dr
            rows += 3 if c["next"] else c["beta"] != 1.0
        elif c["next"]:
            rows += 1
        if c["gate"] == "element":
            rows += 2 if "backward" in c["op"] else 1
        cols = (c["post"] + c["next"]) * ESIZE[c["wdtype"]] + (c["gate"] == "channel") * es
        tokens = c["T"] * es * (c["gate"] == "token")
        twice = 2 if "backward" in c["op"] else 1
        return dict(bytes=rows * n * es + twice * (cols * c["H"] + tokens),
                    flops=n * (4 + 4 * c["post"] + 4 * c["next"]) * twice)
    S = c["T"] * c["K"]
    M = _capacity(S, c["E"], c["align"])
    valid = int(S * (1 - c["skip"]))
    x, wbytes = c["T"] * c["H"] * es, 4 * S if c["weighted"] else 0
    if c["op"] == "dispatch":
        return dict(bytes=4 * S + x + M * c["H"] * es + 4 * (S + M + 2 * c["E"] + 1) + wbytes,
                    flops=valid * c["H"] if c["weighted"] else S)
    if c["op"] == "combine":
        return dict(bytes=valid * c["H"] * es + x + 4 * S + wbytes, flops=2 * valid * c["H"])
    if c["op"] == "dispatch_backward":
        return dict(bytes=valid * c["H"] * es + x * (2 if c["weighted"] else 1) + 4 * S + 2 * wbytes,
                    flops=(4 if c["weighted"] else 1) * valid * c["H"])
    return dict(bytes=(M + (valid if c["weighted"] else 0)) * c["H"] * es + x + 4 * S + 2 * wbytes,
                flops=(3 if c["weighted"] else 1) * valid * c["H"])


# --------------------------------------------------------------------- exact

def _exact_sort(idx, E, align):
    """Slot by slot over the experts, in numpy."""
    T, K = idx.shape
    flat = idx.cpu().numpy().reshape(-1)
    M = _capacity(T * K, E, align)
    counts, offsets = np.zeros(E, np.int32), np.zeros(E + 1, np.int32)
    inv, row_slot = np.full(T * K, -1, np.int32), np.full(M, -1, np.int32)
    for e in range(E):
        slots = np.flatnonzero(flat == e)
        counts[e] = len(slots)
        inv[slots] = offsets[e] + np.arange(len(slots))
        row_slot[offsets[e]:offsets[e] + len(slots)] = slots
        offsets[e + 1] = offsets[e] + math.ceil(len(slots) / align) * align
    return [torch.from_numpy(a).cuda() for a in (counts, offsets, inv.reshape(T, K), row_slot)]


def _exact_route(c, s):
    counts, offsets, inv, row_slot = _exact_sort(s["idx"], c["E"], c["align"])
    T, K, H, M = c["T"], c["K"], c["H"], row_slot.numel()
    t, k = torch.nonzero(inv >= 0, as_tuple=True)
    row = inv[t, k].long()
    w = torch.ones(T, K, dtype=torch.float64, device="cuda") if s["w"] is None else s["w"].double()

    def placed(x):
        out = torch.zeros(M, H, dtype=torch.float64, device="cuda")
        out[row] = x.double()[t] * w[t, k][:, None]
        return out

    def summed(rows):
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(K):
            m = k == j
            out[t[m]] += rows[row[m]].double() * w[t[m], j][:, None]
        return out

    def dots(x, rows):
        if s["w"] is None:
            return None
        d = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        for j in range(K):
            m = k == j
            d[t[m], j] = torch.einsum("th,th->t", x[t[m]].double(), rows[row[m]].double())
        return d

    if c["op"] == "dispatch":
        return placed(s["hidden"]), counts, offsets, inv, row_slot
    if c["op"] == "combine":
        return summed(s["rows"])
    if c["op"] == "dispatch_backward":
        return summed(s["drows"]), dots(s["hidden"], s["drows"])
    return placed(s["dout"]), dots(s["dout"], s["rows"])


def _exact_norm(c, s):
    d = {k: (v.double() if torch.is_tensor(v) else v) for k, v in s.items()}

    def stat(v):
        return 1.0 / torch.sqrt(torch.einsum("th,th->t", v, v) / c["H"] + EPS)

    def normed(v, w):
        return torch.einsum("th,t,h->th", v, stat(v), w)

    def back(dy, v, w):
        inv = stat(v)
        inner = torch.einsum("th,h,th->t", dy, w, v)
        dv = inv[:, None] * w * dy - (inv ** 3 * inner / c["H"])[:, None] * v
        return dv, torch.einsum("th,th,t->h", dy, v, inv)

    if c["op"] == "norm_before":
        return normed(d["x"], d["weight"])
    if c["op"] == "norm_before_backward":
        return back(d["dy"], d["x"], d["weight"])
    gate, slope = 1.0, 0.0
    if c["gate"] != "none":
        v = d["gate"]
        gate = {"none": v, "sigmoid": 1 / (1 + torch.exp(-v)), "tanh": torch.tanh(v)}[c["act"]]
        slope = {"none": torch.ones_like(v), "sigmoid": torch.exp(-v) / (1 + torch.exp(-v)) ** 2,
                 "tanh": torch.cosh(v) ** -2}[c["act"]]
    z = normed(d["h"], d["weight"]) if c["post"] else d["h"]
    if c["op"] == "norm_after":
        r = c["alpha"] * gate * z + c["beta"] * d["x"]
        return (r, normed(r, d["next_weight"])) if c["next"] else r
    G, dnext = d["dr"], None
    if c["next"]:
        dv, dnext = back(d["dy"], d["r"], d["next_weight"])
        G = G + dv
    dgate = None
    if c["gate"] != "none":
        dgate = c["alpha"] * G * z * slope
        dgate = dgate.sum(0) if c["gate"] == "channel" else dgate.sum(1, keepdim=True) if c["gate"] == "token" else dgate
    dh, dweight = c["alpha"] * gate * G, None
    if c["post"]:
        dh, dweight = back(dh, d["h"], d["weight"])
    return c["beta"] * G, dh, dweight, dgate, dnext


def _exact_matvec(c, s):
    table = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    x = s["x"].double()
    out = torch.empty(c["T"], c["N"], dtype=torch.float64, device="cuda")
    column = torch.arange(c["K"], device="cuda") // c["group"]
    for n0 in range(0, c["N"], 4096):  # a few rows of weights at a time
        w = s["w"][n0:n0 + 4096]
        code = torch.empty(w.shape[0], c["K"], dtype=torch.long, device="cuda")
        code[:, 0::2], code[:, 1::2] = w & 15, w >> 4
        scale = s["w_scale"][n0:n0 + 4096]
        if c["fmt"] == "fp4":
            value = torch.ldexp(table[code], (scale.int() - 127)[:, column])
        else:
            zero = torch.full_like(scale, 8) if s["w_zero"] is None else s["w_zero"][n0:n0 + 4096]
            value = (code.double() - zero.double()[:, column]) * scale.double()[:, column]
        out[:, n0:n0 + 4096] = torch.einsum("tk,nk->tn", x, value)
    if not c["swiglu"]:
        return out
    gate, up = out.chunk(2, dim=1)
    return gate / (1 + torch.exp(-gate)) * up


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "matvec":
        return _exact_matvec(case, s)
    return _present(_exact_norm(case, s) if case["op"].startswith("norm") else _exact_route(case, s))
