"""MoEResidualNorm: the RMS norms behind a block and in front of the next one, with the block's gate
and the residual addition between them.

Like the handles of train.py it owns its small device buffers, checks tensor dtypes, shapes
and devices, and forwards every call to the C ABI.
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import torch

from . import binding as B
from .layer import _need
from .train import _device, _dtype, _need_rows, _on, _plain, _stream


class MoEResidualNorm:
    """T tokens of H channels between two blocks:

      u = post_weight f rstd_f   (an RMS norm behind the block; post=False: u = f)
      out = x + scale gate u     (gate: None, "channel" [H] or "token" [T])
      n = pre_weight out rstd_out   (an RMS norm in front of the next block; pre=False: none)

    Without f (and with pre) the call is the RMS norm of x.  dtype: of f, n and their gradients;
    res_dtype: of the residual stream x, out and its gradient (dtype, the default, or "fp32");
    param_dtype: of the weights and the gate (dtype, the default, or "fp32").  The forward keeps the
    reciprocal norms of every token (self.rstd_f, self.rstd_out, fp32) for its backward."""

    def __init__(self, T: int, H: int, dtype: str = "bf16", res_dtype: Optional[str] = None,
                 param_dtype: Optional[str] = None, post: bool = True, gate: Optional[str] = None,
                 pre: bool = True, scale: float = 1.0, eps: float = 1e-6,
                 device: Optional[torch.device] = None):
        res_dtype = dtype if res_dtype is None else res_dtype
        param_dtype = dtype if param_dtype is None else param_dtype
        if gate not in B.GATE:
            raise ValueError(f"gate must be one of {tuple(B.GATE)}, got {gate!r}")
        self.T, self.H, self.post, self.gate, self.pre = int(T), int(H), bool(post), gate, bool(pre)
        self.dtype, self.res_dtype = _dtype(dtype), _dtype(res_dtype)
        self.param_dtype = _dtype(param_dtype)
        self.device = _device(device)
        self.shape = B.ResNorm(self.T, self.H, B.DTYPE[dtype], B.DTYPE[res_dtype],
                               B.DTYPE[param_dtype], int(self.post), B.GATE[gate], int(self.pre),
                               scale, eps)
        size = B.mm_moe_resnorm_workspace_size(self.shape)
        self.rstd_f, self.rstd_out = (
            torch.empty(self.T, dtype=torch.float32, device=self.device) if has else None
            for has in (self.post, self.pre))
        self.workspace = torch.empty(size, dtype=torch.uint8, device=self.device)
        self._rows, self._cols = torch.Size((self.T, self.H)), torch.Size((self.H,))
        self._gates = torch.Size((self.H if gate == "channel" else self.T,))
        # whether a backward may have an f (False, True or both), once a forward has left what it reads
        self._with_f: Tuple[bool, ...] = ()
        self._where = -1 if self.device.index is None else self.device.index

    def _check_rows(self, t, name, dtype):
        if not _plain(t, self._rows, dtype, self._where):
            _need_rows(t, name, self._rows, dtype, self.device)

    def _check_param(self, t, name, has, shape):
        if not has:
            if t is not None:
                raise ValueError(f"{name}: this call has none")
        elif not _plain(t, shape, self.param_dtype, self._where):
            _need(t, name, shape, self.param_dtype, self.device)

    def _check_params(self, has_f, post_weight, gate, pre_weight):
        self._check_param(post_weight, "post_weight", self.post and has_f, self._cols)
        self._check_param(gate, "gate", self.gate is not None and has_f, self._gates)
        self._check_param(pre_weight, "pre_weight", self.pre, self._cols)

    def forward(self, x, f=None, post_weight=None, gate=None, pre_weight=None,
                out: Optional[torch.Tensor] = None, stream=None
                ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
        """(out, n); out is x itself without f, n None with pre=False.  `out` may be given, and may
        be x (in place); rows that overlap otherwise are refused (MoEError)."""
        self._check_rows(x, "x", self.res_dtype)
        has_f = f is not None
        if has_f:
            self._check_rows(f, "f", self.dtype)
        elif not self.pre:
            raise ValueError("f: needed without a norm in front of the next block")
        self._check_params(has_f, post_weight, gate, pre_weight)
        if not has_f:
            if out is not None and out is not x:
                raise ValueError("out: it is x itself without f")
            out = x
        elif out is None:
            out = torch.empty(self._rows, dtype=self.res_dtype, device=self.device)
        else:
            self._check_rows(out, "out", self.res_dtype)
        n = torch.empty(self._rows, dtype=self.dtype, device=self.device) if self.pre else None
        _on(self.device, B.mm_moe_resnorm_forward, self.shape, x, f, post_weight, gate, pre_weight,
            out, n, self.rstd_f, self.rstd_out,
            _stream(stream, self.device, out if has_f else None, n, self.rstd_f, self.rstd_out))
        # (without a norm behind the block a forward of the norm alone keeps what one with f would)
        self._with_f = (True,) if has_f else (False,) if self.post else (False, True)
        return out, n

    def load_stats(self, rstd_f=None, rstd_out=None) -> None:
        """Takes a forward's reciprocal norms (each where the shape has it) in place of a forward
        of this handle's own, for a backward on what that forward left."""
        for mine, t, name in ((self.rstd_f, rstd_f, "rstd_f"), (self.rstd_out, rstd_out, "rstd_out")):
            if mine is None:
                if t is not None:
                    raise ValueError(f"{name}: this norm has none")
            elif t is not None:
                _need(t, name, torch.Size((self.T,)), torch.float32, self.device)
        if self.pre and rstd_out is None:
            raise ValueError("rstd_out: needed with a norm in front of the next block")
        for mine, t in ((self.rstd_f, rstd_f), (self.rstd_out, rstd_out)):
            if t is not None:
                mine.copy_(t)
        self._with_f = (rstd_f is not None,) if self.post else (False, True)

    def backward(self, dout, dn=None, out=None, f=None, post_weight=None, gate=None,
                 pre_weight=None, stream=None
                 ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Dict[str, torch.Tensor]]:
        """(dx, df, gradients of post_weight, gate and pre_weight by name) of the last forward.

        dout: gradient of out, or None (with pre: out led nowhere but to n); dn: of n (with pre).
        The forward's out (x, where it had no f; with pre), f and parameters are given again."""
        has_f = f is not None
        if dout is not None:
            self._check_rows(dout, "dout", self.res_dtype)
        elif not self.pre:
            raise ValueError("dout: needed without a norm in front of the next block")
        if self.pre:
            self._check_rows(dn, "dn", self.dtype)
            self._check_rows(out, "out", self.res_dtype)
        elif dn is not None:
            raise ValueError("dn: this norm has no n")
        if has_f:
            self._check_rows(f, "f", self.dtype)
        self._check_params(has_f, post_weight, gate, pre_weight)
        if not self._with_f:
            raise RuntimeError("backward needs a forward first")
        if has_f not in self._with_f:
            raise ValueError("f: as the forward had it")
        dx = torch.empty(self._rows, dtype=self.res_dtype, device=self.device)
        df = torch.empty(self._rows, dtype=self.dtype, device=self.device) if has_f else None
        grads = {name: torch.empty_like(t) for name, t in
                 (("post_weight", post_weight), ("gate", gate), ("pre_weight", pre_weight))
                 if t is not None}
        _on(self.device, B.mm_moe_resnorm_backward, self.shape, dout, dn, out if self.pre else None,
            f, post_weight, gate, pre_weight, self.rstd_f, self.rstd_out, dx, df,
            grads.get("post_weight"), grads.get("gate"), grads.get("pre_weight"), self.workspace,
            _stream(stream, self.device, dx, df, *grads.values(), self.rstd_f, self.rstd_out,
                    self.workspace))
        return dx, df, grads
