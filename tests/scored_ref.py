"""Plain 64-bit routing by scores, a token at a time: scores, choice, groups,
top-k and weights as include/moe.h defines them (moe_router_t)."""
import numpy as np
import torch


def scores(L, sigmoid):
    L = np.asarray(L, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-L))
        m = np.nanmax(L) if not np.isnan(L).all() else -np.inf
        if m == -np.inf:
            return np.zeros_like(L) if not np.isnan(L).any() else np.full_like(L, np.nan)
        e = np.exp(L - m)
        return e / e.sum()


def log_scores(L, sigmoid):
    """log s, which holds where s itself leaves 64 bits."""
    L = np.asarray(L, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if sigmoid:
            return np.minimum(L, 0.0) - np.log1p(np.exp(-np.abs(L)))
        m = np.max(L)
        return L - m - np.log(np.exp(L - m).sum()) if m > -np.inf else np.full_like(L, -np.inf)


def shares(log_s):
    """s over their sum; zeros where every s is 0."""
    m = np.max(log_s)
    if m == -np.inf:
        return np.zeros_like(log_s)
    e = np.exp(log_s - m)
    return e / e.sum()


def ranked(q, ids):
    """ids by descending q, equal ones by ascending id, NaN last."""
    q = np.asarray(q, np.float64)
    nan = np.isnan(q)
    return [ids[i] for i in np.lexsort((ids, np.where(nan, 0.0, -q), nan))]


def select(L, bias, k, sigmoid, G, Gk, top2):
    """The chosen experts of one token."""
    s = scores(L, sigmoid)
    E = len(s)
    q = s if bias is None else s + np.asarray(bias, np.float64)
    # without a bias the experts' order is that of the logits
    order = np.asarray(L, np.float64) if bias is None else q
    kept = range(G)
    if Gk < G:
        n = E // G
        u = []
        for g in range(G):
            best = ranked((order if not top2 else q)[g * n:(g + 1) * n], list(range(g * n, (g + 1) * n)))
            of = q if top2 or bias is not None else order
            u.append(of[best[0]] + of[best[1]] if top2 and n > 1 else of[best[0]])
        kept = sorted(ranked(u, list(range(G)))[:Gk])
    ids = [e for g in kept for e in range(g * (E // G), (g + 1) * (E // G))]
    return ranked(order[ids], ids)[:k]


def select_many(L, bias, k, sigmoid, G, Gk, top2):
    """The same for a batch [T, E] of finite logits, in torch on its device."""
    T, E = L.shape
    L = L.double()
    s = 1.0 / (1.0 + torch.exp(-L)) if sigmoid else torch.softmax(L, -1)
    q = s if bias is None else s + bias.double()
    order = L if bias is None else q
    if Gk < G:
        best = torch.sort((q if top2 else order).view(T, G, -1), dim=-1, descending=True).values
        u = best[..., :2].sum(-1) if top2 else best[..., 0]
        kept = torch.sort(u, dim=-1, descending=True, stable=True).indices[:, :Gk]
        there = torch.zeros(T, G, dtype=torch.bool, device=L.device).scatter_(1, kept, True)
        order = order.masked_fill(~there.repeat_interleave(E // G, 1), float("-inf"))
    return torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :k]


def weights(L, idx, sigmoid, renorm, scale):
    """torch, 64 bits, differentiable in L [T, E]."""
    s = torch.sigmoid(L) if sigmoid else torch.softmax(L, -1)
    w = s.gather(1, idx)
    return scale * (w / w.sum(-1, keepdim=True) if renorm else w)
