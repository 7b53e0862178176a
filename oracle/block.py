"""64-bit oracle of the operators around the experts forward (torch, any device).

Every function takes the operands as tensors and computes in float64 from the
definitions. The functions with a `mag` argument return, when it is true, the
same expression with every term taken by its absolute value and every
difference as a sum: what rounding errors in the terms are measured by.
"""
import math

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ------------------------------------------------------------ tokens by expert

def row_capacity(S, E, align):
    return (S + min(E, S) * (align - 1)) // align * align


def sort_tokens(topk_idx, E, align):
    """(counts, offsets, inv, row_slot) as int lists, slot by slot."""
    flat = [int(v) for v in topk_idx.reshape(-1).tolist()]
    S = len(flat)
    groups = [[] for _ in range(E)]
    for s, e in enumerate(flat):
        if 0 <= e < E:
            groups[e].append(s)
    row_slot, inv, offsets = [-1] * row_capacity(S, E, align), [-1] * S, [0]
    for g in groups:
        for i, s in enumerate(g):
            row_slot[offsets[-1] + i] = s
            inv[s] = offsets[-1] + i
        offsets.append(offsets[-1] + math.ceil(len(g) / align) * align)
    return [len(g) for g in groups], offsets, inv, row_slot


def place(x, w, inv, M):
    """rows[inv[t, k]] = w[t, k] x[t], zeros elsewhere."""
    T, K = inv.shape
    out = torch.zeros(M, x.shape[1], dtype=torch.float64, device=x.device)
    for k in range(K):
        ok = inv[:, k] >= 0
        v = x.double()[ok]
        out[inv[ok, k].long()] = v if w is None else v * w.double()[ok, k:k + 1]
    return out


def gather(rows, w, inv, mag=False):
    """out[t] = sum_k w[t, k] rows[inv[t, k]]."""
    out = torch.zeros(inv.shape[0], rows.shape[1], dtype=torch.float64, device=rows.device)
    for k in range(inv.shape[1]):
        ok = inv[:, k] >= 0
        v = rows[inv[ok, k].long()].double()
        v = v if w is None else v * w.double()[ok, k:k + 1]
        out[ok] += v.abs() if mag else v
    return out


def dots(x, rows, inv, mag=False):
    """<x[t], rows[inv[t, k]]>, 0 for skipped slots."""
    out = torch.zeros(inv.shape, dtype=torch.float64, device=rows.device)
    for k in range(inv.shape[1]):
        ok = inv[:, k] >= 0
        v = x.double()[ok] * rows[inv[ok, k].long()].double()
        out[ok, k] = (v.abs() if mag else v).sum(1)
    return out


# --------------------------------------------------------- norms around a block

def _scale(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def _w(w, offset):
    return 1.0 if w is None else w.double() + offset


def norm(v, w, eps, offset=0.0):
    v = v.double()
    return v * _scale(v, eps) * _w(w, offset)


def gate_value(gate, act):
    if gate is None:
        return 1.0
    g = gate.double()
    return torch.sigmoid(g) if act == "sigmoid" else torch.tanh(g) if act == "tanh" else g


def gate_slope(gate, act):
    """d act / d gate, from the gate's distance from 0: 1 - g has no bits left
    where g has come near 1. Never negative: its own magnitude."""
    e = torch.exp(-gate.double().abs() * (2 if act == "tanh" else 1))
    if act == "none":
        return torch.ones_like(e)
    return e / (1 + e) ** 2 * (4 if act == "tanh" else 1)


def norm_after(x, h, w, gate, act, alpha, beta, eps, offset, has_norm, mag=False):
    z = norm(h, w, eps, offset) if has_norm else h.double()
    if mag:
        return abs(beta) * x.double().abs() + (alpha * gate_value(gate, act) * z).abs()
    return beta * x.double() + alpha * gate_value(gate, act) * z


def norm_backward(d, v, w, eps, offset=0.0, mag=False):
    """(gradient at v, gradient of w) of N(v; w) for d."""
    d, v = d.double(), v.double()
    inv = _scale(v, eps)
    u = d * _w(w, offset)
    if mag:
        d, v, u = d.abs(), v.abs(), u.abs()
    inner = (u * v).mean(1, keepdim=True)
    dv = inv * u + v * inv ** 3 * inner if mag else inv * u - v * inv ** 3 * inner
    return dv, (d * v * inv).sum(0)


def norm_after_backward(dr, h, w, gate, act, alpha, beta, eps, offset, has_norm, dy=None, r=None, next_w=None,
                        next_eps=None, mag=False):
    """(dx, dh, dw, dgate, dnext_w)."""
    G, dnext = dr.double(), None
    if mag:
        G = G.abs()
    if dy is not None:
        d, dnext = norm_backward(dy, r, next_w, next_eps, offset, mag)
        G = G + d
    g = gate_value(gate, act)
    z = norm(h, w, eps, offset) if has_norm else h.double()
    if mag:
        z, alpha, beta = z.abs(), abs(alpha), abs(beta)
        g = g if gate is None else g.abs()
    dgate = None
    if gate is not None:
        full = alpha * G * z * gate_slope(gate, act)
        dgate = full.sum(0) if gate.dim() == 1 else full.sum(1, keepdim=True) if gate.shape[1] == 1 else full
    dz, dw = alpha * g * G, None
    dh = dz * torch.ones_like(h, dtype=torch.float64)
    if has_norm:
        dh, dw = norm_backward(dz, h, w, eps, offset, mag)
    return beta * G, dh, dw, dgate, dnext


# ------------------------------------------------- products with 4-bit weights

def weights_4bit(weights):
    """float64 [N, K] of a prepare_matvec dict."""
    N, K, code = weights["N"], weights["K"], weights["w"]
    u = torch.stack([code & 15, code >> 4], dim=2).reshape(N, K).long()
    group = 32 if weights["fmt"] == "fp4" else weights["group"]
    column = torch.arange(K, device=code.device) // group
    if weights["fmt"] == "fp4":
        e = weights["w_scale"].long()
        scale = torch.where(e == 255, torch.full_like(e, float("nan"), dtype=torch.float64),
                            torch.ldexp(torch.ones_like(e, dtype=torch.float64), e - 127))
        value = torch.tensor(E2M1, dtype=torch.float64, device=code.device)[u]
    else:
        scale = weights["w_scale"].double()
        zero = weights.get("w_zero")
        value = u.double() - (8.0 if zero is None else zero.double()[:, column])
    return value * scale[:, column]


def matvec(x, W, mag=False):
    return x.double().abs() @ W.abs().t() if mag else x.double() @ W.t()


def swiglu(y, limit=None):
    gate, up = y.chunk(2, dim=1)
    if limit is not None:
        gate, up = gate.clamp(max=limit), up.clamp(-limit, limit)
    return gate * torch.sigmoid(gate) * up
