"""The block operators' definitions in 64 bits, for the GPU tests.

Inputs are tensors of any type; every function works on float64 copies. The
gradients come from differentiating the forward definitions.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24                                              # half a step of fp32, relative
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16)}   # of a rounding


def scores(l, score):
    if score == "sigmoid":
        return torch.sigmoid(l)
    m = l.max(dim=1, keepdim=True).values
    z = torch.where(l > -math.inf, torch.exp(l - torch.where(m > -math.inf, m, 0.0)), 0.0)
    total = z.sum(dim=1, keepdim=True)
    return torch.where(total > 0, z / torch.where(total > 0, total, 1.0), 0.0)


def route(logits, bias, K, score="sigmoid", groups=1, topk_groups=1, group_top=1, renorm=True,
          scale=1.0):
    """idx [T, K] int64 and w [T, K]: one row and one pick at a time, ties to the lower index."""
    l = logits.double().cpu()
    T, E = l.shape
    s = scores(l, score)
    c = s + (bias.double().cpu() if bias is not None else 0.0)
    c = torch.where(l == -math.inf, -math.inf, c)
    size = E // groups
    idx = torch.zeros((T, K), dtype=torch.int64)
    for t in range(T):
        row = c[t].tolist()
        value = [sum(sorted(row[g * size:(g + 1) * size], reverse=True)[:group_top])
                 for g in range(groups)]
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:topk_groups]
        allowed = [e for g in sorted(kept) for e in range(g * size, (g + 1) * size)]
        idx[t] = torch.tensor(sorted(allowed, key=lambda e: (-row[e], e))[:K])
    return idx, weights(l, idx, score, renorm, scale)


def weights(l, idx, score, renorm, scale):
    """The weights of given choices; `l` float64 (may require a gradient). Ratios of
    renormalised scores too small for 64 bits are not looked at here."""
    w = scores(l, score).gather(1, idx)
    if renorm:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    return w * scale


def route_backward(logits, idx, d_w, score, renorm, scale):
    l = logits.double().cpu().requires_grad_(True)
    w = weights(l, idx.long().cpu(), score, renorm, scale)
    (g,) = torch.autograd.grad(w, l, d_w.double().cpu())
    return torch.where(l == -math.inf, 0.0, g).detach()


def rms(v, w, eps):
    return v / torch.sqrt((v * v).mean(dim=-1, keepdim=True) + eps) * w


def widen(gate, kind):
    if kind == "none":
        return 1.0
    return gate.unsqueeze(1) if kind == "token" else gate


def block(y, w_post, gate, kind, alpha, eps):
    u = y if w_post is None else rms(y, w_post, eps)
    return alpha * widen(gate, kind) * u


def block_norm(h, y, w_post, gate, kind, w_pre, alpha, eps):
    """(h', x); entries that are not asked for are None."""
    d = [t.double() if t is not None else None for t in (h, y, w_post, gate, w_pre)]
    h, y, w_post, gate, w_pre = d
    h_out = h + block(y, w_post, gate, kind, alpha, eps) if y is not None else h
    return (h_out if y is not None else None,
            rms(h_out, w_pre, eps) if w_pre is not None else None)


def block_norm_backward(d_h_out, d_x, h_out, y, w_post, gate, kind, w_pre, alpha, eps):
    """Gradients at the stored h', as a dict."""
    def leaf(t):
        return None if t is None else t.double().clone().requires_grad_(True)
    out = {}
    g = d_h_out.double() if d_h_out is not None else torch.zeros_like(h_out.double())
    if w_pre is not None:
        a, w = leaf(h_out), leaf(w_pre)
        into, out["d_w_pre"] = torch.autograd.grad(rms(a, w, eps), [a, w], d_x.double())
        g = g + into
    out["d_h"] = g
    if y is not None:
        leaves = {"d_y": leaf(y), "d_w_post": leaf(w_post), "d_gate": leaf(gate)}
        v = block(leaves["d_y"], leaves["d_w_post"], leaves["d_gate"], kind, alpha, eps)
        names = [k for k, t in leaves.items() if t is not None]
        out.update(zip(names, torch.autograd.grad(v, [leaves[k] for k in names], g)))
    return out


def act(z, name):
    return {"none": lambda v: v, "silu": lambda v: v * torch.sigmoid(v),
            "gelu": lambda v: 0.5 * v * torch.special.erfc(-v * math.sqrt(0.5))}[name](z)


def linear(x, w, bias, residual, name):
    """(y, z)"""
    z = x.double() @ w.double().t()
    if bias is not None:
        z = z + bias.double()
    y = act(z, name)
    return (y + residual.double() if residual is not None else y), z


def act_backward(dy, pre, name):
    if name == "none":
        return dy.double()
    z = pre.double().clone().requires_grad_(True)
    (g,) = torch.autograd.grad(act(z, name), z, dy.double())
    return g
