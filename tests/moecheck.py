"""The mixture-of-experts layer in 64 bits (torch float64 on the tensors' device), with elementwise error bounds.

The kernels carry an activation as two 16-bit parts: what they leave out is at most 2^-16 of it (bf16: two
half-steps of 2^-8 multiply) or 2^-20 (fp16 parts, 2^-11 each, with room for the smallest elements of a row); sums
run in fp32 over chains of well under 128 additions, each off by at most 2^-23 of the running magnitude.  So a product
W v is off by at most (part + 2^-16) |W| |v|, and errors of v pass through |W|.  Elementary functions are off by a few
units of 2^-24.  An fp32 value below 2^-126 is a multiple of 2^-149, so an activation or an output of that size is off
by up to TINY whatever it was computed from.
"""
from __future__ import annotations

import torch

FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
PART = {"bf16": 2.0 ** -16, "mxfp4": 2.0 ** -20}
SUM = 2.0 ** -16
TINY = 2.0 ** -149


def widen(w, scale):
    if scale is None:
        return w.double()
    lut = torch.tensor(FP4 + tuple(-v for v in FP4), dtype=torch.float64, device=w.device)
    b = w.long()
    v = lut[torch.stack((b & 15, b >> 4), -1).flatten(-2)]
    s = torch.where(scale == 255, float("nan"), torch.exp2(scale.double() - 127.0))
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def route(x, gamma, router_w, bias, topk, n_shared, score, scale, eps):
    """t, ids, weights and the smallest gap between a selected expert and the next one of each token, relative to its
    largest score (fp32 scores are off by about 1e-6 of that)."""
    t = x.double()
    if gamma is not None:
        t = t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps) * gamma.double()
    z = t @ router_w.double().T
    weigh = torch.sigmoid(z) if score == "sigmoid" else z
    rank = weigh if bias is None else weigh + bias.double()
    order = torch.sort(rank, dim=-1, descending=True, stable=True)
    ids = order.indices[:, :topk]
    gaps = (order.values[:, :-1] - order.values[:, 1:]) / rank.abs().amax(-1, keepdim=True)
    gap = gaps[:, :topk].amin(-1) if gaps.shape[1] else torch.ones(len(t), dtype=torch.float64, device=t.device)
    if score == "sigmoid":
        w = torch.gather(weigh, 1, ids)
        w = w / w.sum(-1, keepdim=True)
    else:
        w = torch.softmax(torch.gather(rank, 1, ids), -1)
    w = w * scale
    E = router_w.shape[0]
    more = torch.arange(E, E + n_shared, device=ids.device).expand(len(t), n_shared)
    return t, torch.cat((ids, more), 1), torch.cat((w, torch.ones_like(more, dtype=torch.float64)), 1), gap


def experts(t, ids, w1, s1, b1, w2, s2, b2, weight_dtype, act, alpha, beta, limit, interleaved):
    """Slots y [T, S, H] in 64 bits and their bounds."""
    T, S = ids.shape
    H = w2.shape[1]
    y = torch.empty((T, S, H), dtype=torch.float64, device=t.device)
    bound = torch.empty_like(y)
    rel = PART[weight_dtype] + SUM
    for e in torch.unique(ids).tolist():
        at = (ids == e).nonzero()
        m1 = widen(w1[e], None if s1 is None else s1[e])
        m2 = widen(w2[e], None if s2 is None else s2[e])
        v = t[at[:, 0]]
        h = v @ m1.T + (0 if b1 is None else b1[e].double())
        dh = rel * (v.abs() @ m1.abs().T) + 2.0 ** -22 * h.abs()
        if act == "relu2":
            a = torch.clamp(h, min=0.0) ** 2
            da = (2 * torch.clamp(h, min=0.0) + dh) * dh + 2.0 ** -22 * a
        else:
            half = h.shape[1] // 2
            cut = (lambda m: (m[:, 0::2], m[:, 1::2])) if interleaved else (lambda m: (m[:, :half], m[:, half:]))
            (g, u), (dg, du) = cut(h), cut(dh)
            if limit > 0:
                g, u = torch.clamp(g, max=limit), torch.clamp(u, -limit, limit)
            silu = g * torch.sigmoid(alpha * g)
            a = silu * (u + beta)
            slope = 1.0 + 0.28 * max(1.0, abs(alpha))  # |d silu / d g| <= sigmoid + |alpha g| sigmoid' < 1.28
            da = slope * dg * ((u + beta).abs() + du) + silu.abs() * du + 2.0 ** -20 * a.abs()
        da = da + TINY
        out = a @ m2.T + (0 if b2 is None else b2[e].double())
        dy = da @ m2.abs().T + rel * ((a.abs() + da) @ m2.abs().T) + 2.0 ** -22 * out.abs() + TINY
        y[at[:, 0], at[:, 1]] = out
        bound[at[:, 0], at[:, 1]] = dy
    return y, bound
