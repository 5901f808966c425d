"""MoEBlock: the expert layer as a training step runs it, x + MoE(LayerNorm(x)), or between RMS
norms with a gate and a residual scale.

  n = LayerNorm(x);  topk = Router(n);  losses = BalanceLoss(router logits, topk)
  out = x + MoELayer(n, topk)

and its backward: the layer's dx, the router's (with the auxiliary losses' logit gradient)
added to it, the norm's backward joined with the residual path's gradient.  Every step but the
residual's addition (under RMS norms that one too) is one of the library's operators; this module
holds the buffers that pass between them.  The layer gives its output in bf16, so out is rounded
twice: where the layer stores it and where the residual is added (one half ulp of MoE(n) beside one
of out).
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch

from .layer import MoELayer, MoERouter
from .resnorm import MoEResidualNorm
from .train import MoEBalanceLoss, MoELayerNorm

PARAMS = ("norm_weight", "norm_bias", "W_router", "W_gate", "W_up", "W_down")
RMS_PARAMS = ("norm_weight", "post_weight", "gate", "next_weight", "W_router", "W_gate", "W_up",
              "W_down")


class MoEBlock:
    """One pre-norm MoE block of T tokens (in `sequences` sequences), with its parameters
    passed in as a dict of bf16 tensors: norm_weight, norm_bias [H], W_router [E, H],
    W_gate, W_up [E, I, H], W_down [E, H, I].

    select: options of the router's choice of experts (MoERouter's); the forward then takes the
    balance bias.

    norm="rms": RMS norms without a bias, and what today's blocks have behind them:
      n = norm_weight x rstd;  f = MoELayer(n, topk)
      out = x + scale gate post_weight f rstd_f;  next = next_weight out rstd_out
    in one pass over out (MoEResidualNorm).  Of its parameters post_weight, gate and next_weight [H] are
    each left out where the block has none (post_norm, gate, next_norm); `next` is the norm in front
    of the following block, which takes it as its n and has no norm_weight of its own (first=False)."""

    def __init__(self, T: int, H: int, I: int, E: int, k: int, prec: str = "bf16",
                 sequences: int = 1, device: Optional[torch.device] = None,
                 recompute: bool = False, select: Optional[dict] = None, norm: str = "layer",
                 post_norm: bool = True, gate: bool = False, next_norm: bool = False,
                 first: bool = True, scale: float = 1.0):
        if norm not in ("layer", "rms"):
            raise ValueError(f"norm must be 'layer' or 'rms', got {norm!r}")
        self.rms, self.first, self.next_norm = norm == "rms", first, next_norm
        if self.rms:
            self.norm = MoEResidualNorm(T, H, post=False, device=device) if first else None
            self.join = MoEResidualNorm(T, H, post=post_norm, gate="channel" if gate else None,
                                        pre=next_norm, scale=scale, device=device)
            self.join_params = {k: n for k, n, has in (
                ("post_weight", "post_weight", post_norm), ("gate", "gate", gate),
                ("pre_weight", "next_weight", next_norm)) if has}
        elif gate or next_norm or not first or scale != 1.0:
            raise ValueError("gate, next_norm, first and scale: with norm='rms'")
        else:
            self.norm = MoELayerNorm(T, H, device=device)
        self.router = MoERouter(T, H, E, k, device=device, select=select)
        self.balance = MoEBalanceLoss(T, E, k, sequences, device=device)
        self.layer = MoELayer(T, H, I, E, k, prec, device=device, recompute=recompute)
        self._kept = None

    @staticmethod
    def init_params(H: int, I: int, E: int, seed: int = 0, std: float = 0.02,
                    device="cuda", rms: bool = False) -> Dict[str, torch.Tensor]:
        """rms: all parameters that a block with norm="rms" can have."""
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def w(*shape):
            return (std * torch.randn(shape, generator=gen, device=device)).to(torch.bfloat16)
        ones = [torch.ones(H, dtype=torch.bfloat16, device=device) for _ in range(4 if rms else 1)]
        if rms:
            return dict(zip(RMS_PARAMS, ones), W_router=w(E, H), W_gate=w(E, I, H),
                        W_up=w(E, I, H), W_down=w(E, H, I))
        return dict(norm_weight=ones[0],
                    norm_bias=torch.zeros(H, dtype=torch.bfloat16, device=device),
                    W_router=w(E, H), W_gate=w(E, I, H), W_up=w(E, I, H), W_down=w(E, H, I))

    def forward(self, x: torch.Tensor, params: Dict[str, torch.Tensor], seq_offsets=None,
                mask=None, bias=None, n=None) -> Tuple[torch.Tensor, ...]:
        """(out [T, H], losses [2] fp32: balance and z, counts [sequences, E] int32), with next_norm
        the next block's n behind them; losses and counts are the balance loss's own tensors, which
        the next forward overwrites.  bias [E] fp32: the router's (with select).  n: the block in
        front's next (with first=False)."""
        p = params
        if (n is None) != self.first:
            raise ValueError("n: the block in front's next, with first=False")
        if not self.rms:
            n = self.norm.forward(x, p["norm_weight"], p["norm_bias"])
        elif self.first:
            n = self.norm.forward(x, pre_weight=p["norm_weight"])[1]
        self._kept = None  # (from here on the handles hold parts of this forward)
        idx, w = self.router.forward(n, p["W_router"], bias=bias)
        losses, counts = self.balance.forward(self.router.logits, idx, seq_offsets, mask)
        f = self.layer.forward(n, idx, w, p["W_gate"], p["W_up"], p["W_down"])
        kept = (x, n, idx, w, seq_offsets, mask)
        if not self.rms:
            self._kept = kept
            return f.add_(x), losses, counts
        out, following = self.join.forward(x, f, **{k: p[v] for k, v in self.join_params.items()})
        self._kept = (*kept, f, out)
        return (out, losses, counts, following) if self.next_norm else (out, losses, counts)

    def backward(self, dout: Optional[torch.Tensor], params: Dict[str, torch.Tensor],
                 dlosses: torch.Tensor, dnext: Optional[torch.Tensor] = None
                 ) -> Tuple[torch.Tensor, ...]:
        """(dx, gradients of the parameters) of the last forward; dlosses [2] fp32 on the
        device: the gradients of the balance and the z loss (their coefficients).  With next_norm
        dnext is the gradient of next (dout may then be None); with first=False dn stands behind
        dx and the gradients: that of the forward's n, the block in front's dnext."""
        if dnext is not None and not self.next_norm:
            raise ValueError("dnext: this block gives no next (next_norm)")
        if self._kept is None:
            raise RuntimeError("backward needs a forward first")
        x, n, idx, w, seq_offsets, mask, *rest = self._kept
        p = params
        grads, df = {}, dout
        if self.rms:
            f, out = rest
            dres, df, g = self.join.backward(dout, dnext, out if self.next_norm else None, f,
                                             **{k: p[v] for k, v in self.join_params.items()})
            grads = {self.join_params[k]: v for k, v in g.items()}
        dn, dWg, dWu, dWd, dtw = self.layer.backward(df, p["W_gate"], p["W_up"], p["W_down"],
                                                     x=n)
        daux = self.balance.backward(self.router.logits, dlosses, seq_offsets, mask)
        dWr = self.router.backward(n, p["W_router"], idx, w, dtw, dn, dlogits_aux=daux)
        weights = dict(W_router=dWr, W_gate=dWg, W_up=dWu, W_down=dWd)
        if not self.rms:
            dx, dgamma, dbeta = self.norm.backward(dn, x, p["norm_weight"], dx_add=dout)
            return dx, dict(norm_weight=dgamma, norm_bias=dbeta, **weights)
        if not self.first:
            return dres, {**grads, **weights}, dn
        dx, _, g = self.norm.backward(dres, dn, x, pre_weight=p["norm_weight"])
        return dx, {"norm_weight": g["pre_weight"], **grads, **weights}
