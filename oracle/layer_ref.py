"""CPU oracle of the layer operators: expert routing with scores, layer norm, token embedding and the
distillation head.  TEST INFRASTRUCTURE ONLY; float64 numpy, the definitions as include/moe_scores.h,
moe_norm.h, moe_embed.h and moe_distill.h write them.  It shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def _f64(a) -> np.ndarray:
    return np.asarray(a, dtype=np.float64)


# ------------------------------------------------------------------------------------------ layer norm
def norm_forward(x, weight, bias, eps):
    x = _f64(x)
    mean = x.mean(axis=1)
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    rstd = 1 / np.sqrt(var + eps)
    xh = (x - mean[:, None]) * rstd[:, None]
    y = xh * (1 if weight is None else _f64(weight)) + (0 if bias is None else _f64(bias))
    return y, mean, rstd


def norm_backward(x, weight, dy, eps):
    xh, _, rstd = norm_forward(x, None, None, eps)
    dy = _f64(dy)
    t = dy * (1 if weight is None else _f64(weight))
    dx = rstd[:, None] * (t - t.mean(axis=1, keepdims=True) - xh * (t * xh).mean(axis=1, keepdims=True))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


# ------------------------------------------------------------------------------------------ embedding
def embed_backward(ids, dy, V, scale, padding=-1, into=None):
    g = np.zeros((V, dy.shape[1]))
    for n, i in enumerate(np.asarray(ids)):
        if 0 <= i < V and i != padding:
            g[i] += _f64(dy[n])
    return scale * g + (0 if into is None else _f64(into))


# ------------------------------------------------------------------------------------------ scores
def scores(l, kind):
    """s [N, E]; a row of -inf alone scores 0."""
    l = _f64(l)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-l))
        m = l.max(axis=1, keepdims=True)
        e = np.exp(l - np.where(np.isinf(m), 0, m))
        total = e.sum(axis=1, keepdims=True)
        return np.where(total > 0, e / np.where(total > 0, total, 1), 0)


def route(l, bias, k, groups=1, topk_groups=1, kind="softmax", renormalize=True, scale=1.0, group_top=2):
    """(idx [N, k], weights [N, k], counts [E])."""
    s = scores(l, kind)
    N, E = s.shape
    # without a bias the choice is the logits' own order
    c = _f64(l) if bias is None else s + _f64(bias)
    value = s if bias is None else c
    idx = np.zeros((N, k), np.int64)
    for n in range(N):
        open_ = np.ones(E, bool)
        if groups > 1:
            size = E // groups
            gs = [np.sort(value[n, g * size:(g + 1) * size])[::-1][:group_top].sum() for g in range(groups)]
            best = sorted(range(groups), key=lambda g: (-gs[g], g))[:topk_groups]
            open_ = np.isin(np.arange(E) // size, best)
        cand = sorted(np.flatnonzero(open_), key=lambda e: (-c[n, e], e))
        idx[n] = cand[:k]
    w = np.take_along_axis(s, idx, axis=1)
    if renormalize:
        total = w.sum(axis=1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1), 0)
    return idx, scale * w, np.bincount(idx.ravel(), minlength=E)


def route_backward(l, idx, dw, kind, renormalize, scale):
    s = scores(l, kind)
    N, E = s.shape
    dw = _f64(dw)
    ds = np.zeros((N, E))
    c = np.take_along_axis(s, idx, axis=1)
    total = c.sum(axis=1, keepdims=True) if renormalize else np.ones((N, 1))
    total = np.where(total > 0, total, 1)
    inner = (dw * c).sum(axis=1, keepdims=True) / total if renormalize else 0.0
    np.put_along_axis(ds, idx, scale * (dw - inner) / total, axis=1)
    if kind == "sigmoid":
        return ds * s * scores(-_f64(l), "sigmoid")
    return s * (ds - (ds * s).sum(axis=1, keepdims=True))


# ------------------------------------------------------------------------------------------ distillation
def teacher(t_idx, t_logits, V, tau):
    """q [N, V] (rows without entries: zeros) and sum q log q [N] over the entries."""
    N = t_idx.shape[0]
    q, ent = np.zeros((N, V)), np.zeros(N)
    for n in range(N):
        there = [j for j, i in enumerate(t_idx[n]) if 0 <= i < V and t_logits[n, j] > -np.inf]
        if not there:
            continue
        t = _f64(t_logits[n, there]) / tau
        p = np.exp(t - t.max())
        p /= p.sum()
        for j, pj in zip(there, p):
            q[n, t_idx[n, j]] += pj
        ent[n] = (p[p > 0] * np.log(p[p > 0])).sum()
    return q, ent


def distill(X, W, t_idx, t_logits, tau, dloss):
    """(loss [N], lse [N], dX, dW)."""
    X, W = _f64(X), _f64(W)
    z = X @ W.T / tau
    m = z.max(axis=1, keepdims=True)
    lse = (m + np.log(np.exp(z - m).sum(axis=1, keepdims=True)))[:, 0]
    q, ent = teacher(t_idx, t_logits, W.shape[0], tau)
    loss = tau * tau * (ent + q.sum(axis=1) * lse - (q * z).sum(axis=1))
    d = (np.exp(z - lse[:, None]) * q.sum(axis=1, keepdims=True) - q) * (tau * _f64(dloss))[:, None]
    return loss, lse, d @ W, d.T @ X
