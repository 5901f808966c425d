"""CPU oracle of the choice of experts, fp64 numpy (TEST INFRASTRUCTURE ONLY: imported by tests/,
never by the library): token by token from the definition."""
from __future__ import annotations

import math

import numpy as np

SUM_EPS = 1e-20


def scores(l, score: str):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    if np.all(l == -np.inf):
        return np.zeros_like(l)
    with np.errstate(invalid="ignore"):
        e = np.exp(l - l.max())
    return e / e.sum()


def low(v):
    return np.where(np.isnan(v), -np.inf, v)


def group_scores(l, bias, score, groups, group_score):
    s = scores(l, score)
    key = low(l if bias is None else s + bias)
    val = low(s) if bias is None and group_score == "top2" else key
    two = -np.sort(-val.reshape(groups, -1), axis=1)[:, :2]
    return two.sum(axis=1) if group_score == "top2" else two[:, 0]


def choose(l, bias, k, score, groups, topk_groups, group_score, best=None):
    """The chosen experts of one token; best: the groups that take part, where they are known."""
    E = len(l)
    s = scores(l, score)
    key = low(l if bias is None else s + bias)
    keep = np.ones(E, bool)
    if topk_groups < groups:
        if best is None:
            g = group_scores(l, bias, score, groups, group_score)
            best = np.argsort(-g, kind="stable")[:topk_groups]
        keep = np.repeat(np.isin(np.arange(groups), best), E // groups)
    order = [int(e) for e in np.argsort(-key, kind="stable") if keep[e]]
    return np.array(order[:k])


def weights(l, idx, score, renormalise, scale):
    if renormalise and score == "softmax":
        c = l[idx]
        if np.all(c == -np.inf):
            return np.zeros(len(idx))
        e = np.exp(c - c.max())
        return scale * e / e.sum()
    w = scores(l, score)[idx]
    return scale * (w / (w.sum() + SUM_EPS) if renormalise else w)


def forward(logits, bias, k, score="softmax", groups=1, topk_groups=1, group_score="max",
            renormalise=True, scale=1.0):
    logits = np.asarray(logits, np.float64)
    idx = np.stack([choose(l, bias, k, score, groups, topk_groups, group_score) for l in logits])
    w = np.stack([weights(l, i, score, renormalise, scale) for l, i in zip(logits, idx)])
    return idx, w


def backward(logits, idx, g, score="softmax", renormalise=True, scale=1.0):
    """dlogits through the weights of the experts idx (those outside are dropped)."""
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    d = np.zeros((T, E))
    for t in range(T):
        j = [j for j, e in enumerate(idx[t]) if 0 <= e < E]
        e, gt = np.asarray(idx[t])[j].astype(int), np.asarray(g[t], np.float64)[j]
        l = logits[t]
        if score == "softmax" and renormalise:
            c = l[e]
            if len(c) == 0 or np.all(c == -np.inf):
                continue
            q = np.exp(c - c.max())
            q /= q.sum()
            np.add.at(d[t], e, scale * q * (gt - q @ gt))
            continue
        s = scores(l, score)
        ds = scale * gt
        if renormalise:
            n = s[e].sum() + SUM_EPS
            ds = scale * (gt - (gt @ s[e]) / n) / n
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                np.add.at(d[t], e, ds * s[e] / (1.0 + np.exp(l[e])))
        else:
            np.add.at(d[t], e, ds * s[e])
            d[t] -= s * (ds @ s[e])
    return d
