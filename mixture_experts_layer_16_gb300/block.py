"""MoEBlock: the expert layer as a training step runs it, x + MoE(LayerNorm(x)).

  n = LayerNorm(x);  topk = Router(n);  losses = BalanceLoss(router logits, topk)
  out = x + MoELayer(n, topk)

and its backward: the layer's dx, the router's (with the auxiliary losses' logit gradient)
added to it, the norm's backward joined with the residual path's gradient.  Every step but the
residual's addition is one of the library's operators; this module holds the buffers that pass
between them.  The layer gives its output in bf16, so out is rounded twice: where the layer stores
it and where the residual is added (one half ulp of MoE(n) beside one of out).
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch

from .layer import MoELayer, MoERouter
from .train import MoEBalanceLoss, MoELayerNorm

PARAMS = ("norm_weight", "norm_bias", "W_router", "W_gate", "W_up", "W_down")


class MoEBlock:
    """One pre-norm MoE block of T tokens (in `sequences` sequences), with its parameters
    passed in as a dict of bf16 tensors: norm_weight, norm_bias [H], W_router [E, H],
    W_gate, W_up [E, I, H], W_down [E, H, I]."""

    def __init__(self, T: int, H: int, I: int, E: int, k: int, prec: str = "bf16",
                 sequences: int = 1, device: Optional[torch.device] = None,
                 recompute: bool = False):
        self.norm = MoELayerNorm(T, H, device=device)
        self.router = MoERouter(T, H, E, k, device=device)
        self.balance = MoEBalanceLoss(T, E, k, sequences, device=device)
        self.layer = MoELayer(T, H, I, E, k, prec, device=device, recompute=recompute)
        self._kept = None

    @staticmethod
    def init_params(H: int, I: int, E: int, seed: int = 0, std: float = 0.02,
                    device="cuda") -> Dict[str, torch.Tensor]:
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def w(*shape):
            return (std * torch.randn(shape, generator=gen, device=device)).to(torch.bfloat16)
        return dict(norm_weight=torch.ones(H, dtype=torch.bfloat16, device=device),
                    norm_bias=torch.zeros(H, dtype=torch.bfloat16, device=device),
                    W_router=w(E, H), W_gate=w(E, I, H), W_up=w(E, I, H), W_down=w(E, H, I))

    def forward(self, x: torch.Tensor, params: Dict[str, torch.Tensor], seq_offsets=None,
                mask=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        """(out [T, H], losses [2] fp32: balance and z, counts [sequences, E] int32); losses and
        counts are the balance loss's own tensors, which the next forward overwrites."""
        p = params
        n = self.norm.forward(x, p["norm_weight"], p["norm_bias"])
        idx, w = self.router.forward(n, p["W_router"])
        losses, counts = self.balance.forward(self.router.logits, idx, seq_offsets, mask)
        out = self.layer.forward(n, idx, w, p["W_gate"], p["W_up"], p["W_down"]).add_(x)
        self._kept = (x, n, idx, w, seq_offsets, mask)
        return out, losses, counts

    def backward(self, dout: torch.Tensor, params: Dict[str, torch.Tensor],
                 dlosses: torch.Tensor) -> Tuple[torch.Tensor, Dict[str, torch.Tensor]]:
        """(dx, gradients of the parameters) of the last forward; dlosses [2] fp32 on the
        device: the gradients of the balance and the z loss (their coefficients)."""
        if self._kept is None:
            raise RuntimeError("backward needs a forward first")
        x, n, idx, w, seq_offsets, mask = self._kept
        p = params
        dn, dWg, dWu, dWd, dtw = self.layer.backward(dout, p["W_gate"], p["W_up"], p["W_down"],
                                                     x=n)
        daux = self.balance.backward(self.router.logits, dlosses, seq_offsets, mask)
        dWr = self.router.backward(n, p["W_router"], idx, w, dtw, dn, dlogits_aux=daux)
        dx, dgamma, dbeta = self.norm.backward(dn, x, p["norm_weight"], dx_add=dout)
        return dx, dict(norm_weight=dgamma, norm_bias=dbeta, W_router=dWr, W_gate=dWg, W_up=dWu,
                        W_down=dWd)
