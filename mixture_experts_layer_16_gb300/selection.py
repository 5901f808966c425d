"""MoESelect: the choice of experts from a router's logits in its other forms (scores by softmax or
sigmoid, a balance bias, groups, renormalised weights or not), and its backward.

MoERouter has plain top-k with a softmax over the chosen, and takes these forms as options; this
handle is the choice alone, for logits that come from elsewhere.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import binding as B
from .layer import _need
from .train import _device, _dtype, _on, _plain, _stream


class MoESelect:
    """The k best of E experts for each of T tokens.

    score: "softmax" over all experts or "sigmoid" of each logit.  The experts are ranked by
    score + bias (the bias of the forward call, [E] fp32, or none: it acts on the choice alone and
    has no gradient).  groups, topk_groups: of so many groups of consecutive experts only the
    best take part, by their largest key (group_score "max") or by the sum of their two largest
    ("top2").  renormalise: the chosen weights add up to 1 before `scale`.  Equal keys go to the lower
    index; the order is that of the keys in exact arithmetic.

    dtype: of the logits; grad_dtype: of their gradient, dtype itself (the default) or "bf16"."""

    def __init__(self, T: int, E: int, k: int, score: str = "softmax", groups: int = 1,
                 topk_groups: int = 1, group_score: str = "max", renormalise: bool = True,
                 scale: float = 1.0, dtype: str = "fp32", grad_dtype: Optional[str] = None,
                 device: Optional[torch.device] = None):
        grad_dtype = dtype if grad_dtype is None else grad_dtype
        if score not in B.SCORE:
            raise ValueError(f"score must be one of {tuple(B.SCORE)}, got {score!r}")
        if group_score not in B.GROUP_SCORE:
            raise ValueError(f"group_score must be one of {tuple(B.GROUP_SCORE)}, "
                             f"got {group_score!r}")
        self.dtype, self.grad_dtype = _dtype(dtype), _dtype(grad_dtype)
        if self.grad_dtype not in (self.dtype, torch.bfloat16):
            raise ValueError(f"grad_dtype must be {dtype!r} or 'bf16', got {grad_dtype!r}")
        T, E, k, groups, topk_groups = int(T), int(E), int(k), int(groups), int(topk_groups)
        if not (1 <= T < 1 << 31 and 1 <= E <= 1024 and 1 <= k <= 32):
            raise ValueError(f"T, E, k: got {T}, {E}, {k}, allowed up to 2^31 - 1, 1024, 32")
        if not (1 <= groups <= 32 and E % groups == 0 and 1 <= topk_groups <= groups):
            raise ValueError(f"groups: {E} experts cannot be cut into {groups} groups (at most 32), "
                             f"of which {topk_groups} are kept")
        if k > E // groups * topk_groups:
            raise ValueError(f"k: {k} experts chosen of {E // groups * topk_groups}")
        if not abs(scale) < float("inf"):
            raise ValueError(f"scale must be finite, got {scale}")
        self.T, self.E, self.k = T, E, k
        self.device = _device(device)
        self.shape = B.Select(T, E, k, B.DTYPE[dtype], B.DTYPE[grad_dtype], B.SCORE[score], groups,
                              topk_groups, B.GROUP_SCORE[group_score], int(bool(renormalise)),
                              scale)
        self._rows, self._slots = torch.Size((T, E)), torch.Size((T, k))
        self._experts = torch.Size((E,))
        self._where = -1 if self.device.index is None else self.device.index

    def _need(self, t, name, shape, dtype):
        if not _plain(t, shape, dtype, self._where):
            _need(t, name, shape, dtype, self.device)

    def _check_bias(self, bias):
        if bias is not None:
            self._need(bias, "bias", self._experts, torch.float32)

    def forward(self, logits, bias=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(topk_idx [T, k] int32, topk_w [T, k] fp32)."""
        self._need(logits, "logits", self._rows, self.dtype)
        self._check_bias(bias)
        idx = torch.empty(self._slots, dtype=torch.int32, device=self.device)
        w = torch.empty(self._slots, dtype=torch.float32, device=self.device)
        _on(self.device, B.mm_moe_select_forward, self.shape, logits, bias, idx, w,
            _stream(stream, self.device, idx, w))
        return idx, w

    def backward(self, logits, topk_idx, dtopk_w, dlogits_aux=None,
                 dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The gradient of the forward's logits from that of its topk_w, its topk_idx given again.
        dlogits_aux [T, E] fp32: a further gradient of the logits (MoEBalanceLoss's), added.
        The gradient must not overlap the logits or dlogits_aux (MoEError)."""
        self._need(logits, "logits", self._rows, self.dtype)
        self._need(topk_idx, "topk_idx", self._slots, torch.int32)
        self._need(dtopk_w, "dtopk_w", self._slots, torch.float32)
        if dlogits_aux is not None:
            self._need(dlogits_aux, "dlogits_aux", self._rows, torch.float32)
        if dlogits is None:
            dlogits = torch.empty(self._rows, dtype=self.grad_dtype, device=self.device)
        else:
            self._need(dlogits, "dlogits", self._rows, self.grad_dtype)
        _on(self.device, B.mm_moe_select_backward, self.shape, logits, topk_idx, dtopk_w,
            dlogits_aux, dlogits, _stream(stream, self.device, dlogits))
        return dlogits
