"""The router's definition in 64 bits, token by token, for its tests. CPU only; no code of the library."""
from __future__ import annotations

import math

import numpy as np


def scores(logits, score):
    """64-bit scores of one token; experts with logit +infinity share softmax's sum."""
    l = np.asarray(logits, np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    top = np.nanmax(l) if not np.isnan(l).all() else np.nan
    if not top > -np.inf:
        return np.zeros_like(l)
    with np.errstate(invalid="ignore"):
        e = np.where(l == top, 1.0, np.exp(l - top))
    return e / e.sum()


def choose(logits, r, bias=None):
    """Chosen experts of one token, in order; fewer than num_topk where no more are open."""
    l = np.asarray(logits, np.float64)
    E, G = r.num_experts, r.num_groups
    grouped = r.topk_groups < G
    open_ = l > -np.inf
    if bias is not None:
        open_ &= np.asarray(bias, np.float64) > -np.inf
    s = scores(np.where(np.isnan(l), -np.inf, l), r.score)
    c = l if bias is None else s + np.asarray(bias, np.float64)  # without a bias the scores' order is the logits'
    if grouped:
        value, by = [], s if bias is None and r.group_top == 2 else c
        for g in range(G):
            v = sorted((by[e] for e in range(g * E // G, (g + 1) * E // G) if open_[e]), reverse=True)
            value.append(-math.inf if not v else v[0] if r.group_top == 1 or len(v) == 1 else v[0] + v[1])
        kept = sorted(range(G), key=lambda g: (-value[g], g))[:r.topk_groups]
        open_ = open_ & np.isin(np.arange(E) // (E // G), kept)
    return sorted(np.flatnonzero(open_), key=lambda e: (-c[e], e))[:r.num_topk]


def weights(logits, picked, r):
    """64-bit weights of the picked experts."""
    l = np.asarray(logits, np.float64)
    if not len(picked):
        return np.zeros(0)
    if np.isnan(l).any():
        return np.full(len(picked), np.nan)
    if r.renormalize:  # scaled so that none underflows
        x = l[picked]
        if r.score == "sigmoid":
            low = np.minimum(x, 0.0)
            s = np.exp(low - low.max()) / (1.0 + np.exp(-np.abs(x)))
        else:
            with np.errstate(invalid="ignore"):
                s = np.where(x == x.max(), 1.0, np.exp(x - x.max()))
        s = s / s.sum()
    else:
        s = scores(l, r.score)[picked]
    return s * float(np.float32(r.scale))


def route(logits, r, bias=None):
    T, k = len(logits), r.num_topk
    idx, w = np.full((T, k), -1, np.int64), np.zeros((T, k))
    for t in range(T):
        p = choose(logits[t], r, bias)
        idx[t, :len(p)] = p
        w[t, :len(p)] = weights(logits[t], p, r)
        if np.isnan(np.asarray(logits[t], np.float64)).any():
            w[t] = np.nan
    return idx, w


def gradient(d, logits, idx, r):
    """64-bit gradient of the weights in the logits [T, E], by the chain rule over w = scale s_j / (sum of the chosen or 1)."""
    T, E = np.shape(logits)
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        l = np.asarray(logits[t], np.float64)
        picked, g = [], []
        for j, e in enumerate(idx[t]):
            if 0 <= e < E and e not in picked:
                picked.append(int(e))
                g.append(float(d[t][j]) * float(np.float32(r.scale)))
        if not picked:
            continue
        g, s = np.array(g), scores(l, r.score)
        sp = s[picked]
        total = sp.sum() if r.renormalize else 1.0
        ds = (g - (g @ sp) / total) / total if r.renormalize else g           # of the chosen scores
        mag = (np.abs(g) + (np.abs(g) @ sp) / total) / total if r.renormalize else np.abs(g)
        if r.score == "sigmoid":
            out[t, picked], size[t, picked] = ds * sp * (1 - sp), mag * sp * (1 - sp)
        elif r.renormalize:  # the other experts' parts cancel
            out[t, picked], size[t, picked] = ds * sp, mag * sp
        else:
            full, big = np.zeros(E), np.zeros(E)
            full[picked], big[picked] = g, np.abs(g)
            out[t], size[t] = s * (full - g @ sp), s * (big + np.abs(g) @ sp)
    return out, size
