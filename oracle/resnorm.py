"""CPU oracle of the norms before and after a block with its gate and residual scale, fp64 numpy
(TEST INFRASTRUCTURE ONLY: imported by tests/, never by the library)."""
from __future__ import annotations

import numpy as np


def _gate(gate, kind):
    if kind is None:
        return 1.0
    return gate if kind == "channel" else gate[:, None]


def forward(x, f, w_post, gate, w_pre, kind, scale, eps):
    r = {}
    out = x
    if f is not None:
        u = f
        if w_post is not None:
            r["rstd_f"] = ((f ** 2).mean(axis=1) + eps) ** -0.5
            u = f * r["rstd_f"][:, None] * w_post
        out = x + scale * _gate(gate, kind) * u
    r["out"] = out
    if w_pre is not None:
        r["rstd_out"] = ((out ** 2).mean(axis=1) + eps) ** -0.5
        r["n"] = out * r["rstd_out"][:, None] * w_pre
    return r


def backward(dout, dn, out, f, w_post, gate, w_pre, kind, scale, rstd_f, rstd_out):
    """The gradients from the kept reciprocal norms, row by row."""
    T, H = (out if out is not None else f).shape
    D = np.zeros((T, H)) if dout is None else dout.copy()
    r = {}
    if w_pre is not None:
        oh = out * rstd_out[:, None]
        v = dn * w_pre
        for t in range(T):
            D[t] += rstd_out[t] * (v[t] - oh[t] * (oh[t] @ v[t]) / H)
        r["pre_weight"] = (dn * oh).sum(axis=0)
    r["dx"] = D
    if f is None:
        return r
    fh = f if w_post is None else f * rstd_f[:, None]
    u = fh if w_post is None else fh * w_post
    du = scale * _gate(gate, kind) * D
    if kind is not None:
        r["gate"] = scale * (u * D).sum(axis=0 if kind == "channel" else 1)
    if w_post is None:
        r["df"] = du * np.ones((T, H))
        return r
    r["post_weight"] = (du * fh).sum(axis=0)
    q = du * w_post
    r["df"] = np.stack([rstd_f[t] * (q[t] - fh[t] * (fh[t] @ q[t]) / H) for t in range(T)])
    return r
