"""CPU oracle of the operators around the MoE layer in a training step, fp64 numpy (TEST
INFRASTRUCTURE ONLY: imported by tests/, never by the library): layer normalisation with
its backward, the router's balance and z losses with their logit gradient, the global
gradient norm with clipping.  Plain per-row and per-sequence loops over the definitions.
"""
from __future__ import annotations

from typing import Dict, Optional, Sequence

import numpy as np


# ----------------------------------------------------------------------- layer norm
def norm_forward(x, weight, bias, eps: float) -> Dict[str, np.ndarray]:
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    xc = x - mean[:, None]
    rstd = 1.0 / np.sqrt((xc * xc).mean(axis=1) + eps)
    xh = xc * rstd[:, None]
    y = xh * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return dict(y=y, mean=mean, rstd=rstd, xh=xh)


def norm_backward(dy, x, weight, eps: float, dx_add=None) -> Dict[str, np.ndarray]:
    f = norm_forward(x, weight, None, eps)
    dy = np.asarray(dy, np.float64)
    g = dy * np.asarray(weight, np.float64)
    xh, rstd = f["xh"], f["rstd"]
    dx = np.empty_like(g)
    for t in range(g.shape[0]):
        dx[t] = rstd[t] * (g[t] - g[t].mean() - xh[t] * (g[t] * xh[t]).mean())
    if dx_add is not None:
        dx = dx + np.asarray(dx_add, np.float64)
    return dict(dx=dx, dweight=(dy * xh).sum(axis=0), dbias=dy.sum(axis=0))


# --------------------------------------------------------------------- balance loss
def _members(logits, G, seq_offsets, mask):
    """Indices of every sequence's counting tokens."""
    T = logits.shape[0]
    off = [0, T] if seq_offsets is None else [int(v) for v in seq_offsets]
    out = []
    for s in range(G):
        out.append([t for t in range(off[s], off[s + 1])
                    if (mask is None or mask[t]) and not np.all(logits[t] == -np.inf)])
    return out


def softmax(row) -> np.ndarray:
    e = np.exp(row - row.max())
    return e / e.sum()


def lse(row) -> float:
    m = row.max()
    return float(m + np.log(np.exp(row - m).sum()))


def balance_forward(logits, topk_idx, G: int = 1, seq_offsets=None, mask=None) -> Dict:
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    k = topk_idx.shape[1]
    rows = _members(logits, G, seq_offsets, mask)
    counts = np.zeros((G, E), np.int64)
    seq_loss = np.zeros(G)
    lses = np.zeros(T)
    for s, r in enumerate(rows):
        P = np.zeros(E)
        for t in r:
            P += softmax(logits[t])
            lses[t] = lse(logits[t])
            for e in topk_idx[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        n = len(r)
        if n:
            seq_loss[s] = np.sum(E / (k * n) * counts[s] * (P / n))
    tokens = np.array([len(r) for r in rows], np.int64)
    live, N = int((tokens > 0).sum()), int(tokens.sum())
    z = float((lses ** 2).sum()) / N if N else 0.0
    return dict(losses=np.array([seq_loss.sum() / live if live else 0.0, z]), seq_loss=seq_loss,
                counts=counts, tokens=tokens, lse=lses)


def balance_backward(logits, topk_idx, dlosses, G: int = 1, seq_offsets=None, mask=None
                     ) -> np.ndarray:
    logits = np.asarray(logits, np.float64)
    T, E = logits.shape
    k = topk_idx.shape[1]
    f = balance_forward(logits, topk_idx, G, seq_offsets, mask)
    live, N = int((f["tokens"] > 0).sum()), int(f["tokens"].sum())
    d = np.zeros((T, E))
    for s, r in enumerate(_members(logits, G, seq_offsets, mask)):
        for t in r:
            p = softmax(logits[t])
            n = len(r)
            c = dlosses[0] * E / (k * n * n * live) * f["counts"][s]
            d[t] = p * (c - p @ c) + dlosses[1] * 2.0 * f["lse"][t] / N * p
    return d


# --------------------------------------------------------------------- clipping
def grad_norm(grads: Sequence[np.ndarray]) -> float:
    """sqrt of the sum of squares (scaled by the largest, so that no square overflows)."""
    big = max((float(np.abs(np.asarray(g, np.float64)).max(initial=0.0)) for g in grads),
              default=0.0)
    if not big > 0.0 or not np.isfinite(big):
        return big
    return big * float(np.sqrt(sum(((np.asarray(g, np.float64) / big) ** 2).sum()
                                   for g in grads)))


def grad_clip(grads: Sequence[np.ndarray], max_norm: float, eps: float = 1e-6,
              norm: Optional[float] = None):
    n = grad_norm(grads) if norm is None else norm
    coef = min(1.0, max_norm / (n + eps)) if n + eps > 0 else 1.0
    return n, [np.asarray(g, np.float64) * coef for g in grads]
