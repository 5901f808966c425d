"""MoEAdamW: the optimiser's step over all parameters of a training step, with the clipping by
the gradient norm folded in.

Like the handles of train.py it owns its device buffers (the moments and the step counter),
checks tensor dtypes, shapes and devices, and forwards every call to the C ABI.
"""
from __future__ import annotations

import struct
from array import array
from typing import Optional, Sequence, Tuple, Union

import torch

from . import binding as B
from .train import _CODE, _device, _on, _stream


class MoEAdamW:
    """AdamW with decoupled weight decay over a fixed list of tensors.

    params: the tensors, in the order of every step (their sizes, dtypes and device are kept, not
    the tensors).  weight_decay: one number, or one for each tensor.  states: the moments' form,
    "fp32" or "8bit" (a byte an element and scales for blocks of 32, rounded at random from
    `seed`; include/mm_moe.h has the formats).

    The moments lie one tensor after the other in self.m and self.v (flat; 8-bit codes beside
    self.m_scale and self.v_scale), each tensor from a multiple of 32 elements on (self.first) and
    zero behind its end; with self.counter they are what a checkpoint keeps.  The step is counted
    on the device: a captured step counts on at every replay."""

    def __init__(self, params: Sequence[torch.Tensor], betas: Tuple[float, float] = (0.9, 0.999),
                 eps: float = 1e-8, weight_decay: Union[float, Sequence[float]] = 0.0,
                 states: str = "fp32", seed: int = 0, clip_eps: float = 1e-6,
                 device: Optional[torch.device] = None):
        if states not in B.STATES:
            raise ValueError(f"states must be one of {tuple(B.STATES)}, got {states!r}")
        for i, p in enumerate(params):
            if not isinstance(p, torch.Tensor):
                raise TypeError(f"params[{i}] must be a torch.Tensor")
            if p.dtype not in _CODE:
                raise ValueError(f"params[{i}]: expected bf16, fp16 or fp32, got {p.dtype}")
        if len(params) > B.MM_MOE_MAX_GRADS:
            raise ValueError(f"params: at most {B.MM_MOE_MAX_GRADS} tensors")
        b1, b2 = (float(b) for b in betas)
        if not (0.0 <= b1 < 1.0 and 0.0 <= b2 < 1.0):
            raise ValueError(f"betas must lie in [0, 1), got {betas}")
        if not 2.0 ** -126 <= eps < float("inf"):
            raise ValueError(f"eps must be at least 2^-126, got {eps}")
        decay = [float(weight_decay)] * len(params) if isinstance(weight_decay, (int, float)) \
            else [float(w) for w in weight_decay]
        if len(decay) != len(params):
            raise ValueError(f"weight_decay: expected {len(params)} numbers, got {len(decay)}")
        self.device = _device(params[0].device if device is None and len(params) else device)
        self.betas, self.eps, self.weight_decay, self.states = (b1, b2), eps, decay, states
        self.shapes = [p.shape for p in params]
        self.dtypes = [p.dtype for p in params]
        self._opt = B.AdamW(b1, b2, eps, float("inf"), clip_eps, B.STATES[states],
                            seed & 0xffffffff)
        # a word of each mm_moe_adamw_tensor that no step changes: weight_decay, reserved
        self._decay = [struct.unpack("<Q", struct.pack("<fi", w, 0))[0] for w in decay]
        self._numel = [s.numel() for s in self.shapes]
        self._where = -1 if self.device.index is None else self.device.index
        self.first, total = [], 0
        for n in self._numel:
            self.first.append(total)
            total += -(-n // 32) * 32
        dt = torch.float32 if states == "fp32" else torch.uint8
        d = self.device
        self.m = torch.zeros(total, dtype=dt, device=d)
        self.v = torch.zeros(total, dtype=dt, device=d)
        self.m_scale = self.v_scale = None
        if states == "8bit":
            self.m_scale = torch.zeros(total // 32, dtype=torch.uint8, device=d)
            self.v_scale = torch.zeros(total // 32, dtype=torch.uint8, device=d)
        self.counter = torch.zeros(4, dtype=torch.int64, device=d)
        self._put_step(0)

    def _wait(self):
        if self.device.type == "cuda":  # (a step may run on any stream)
            torch.cuda.synchronize(self.device)

    def _put_step(self, steps: int) -> None:
        b1, b2 = self.betas
        words = struct.unpack("<4q", struct.pack("<qddq", int(steps), b1 ** steps, b2 ** steps, 0))
        self.counter.copy_(torch.tensor(words, dtype=torch.int64))

    def set_step(self, steps: int) -> None:
        """Says that `steps` steps lie behind (a checkpoint's moments); waits for the device."""
        if steps < 0:
            raise ValueError(f"steps must be >= 0, got {steps}")
        self._wait()
        self._put_step(steps)

    def steps(self) -> int:
        """The steps behind; waits for the device."""
        self._wait()
        return int(self.counter[0])

    def _words(self, params, grads, masters):
        """The call's mm_moe_adamw_tensor array: six 64-bit words a tensor."""
        where, words, seen = self._where, [], set()
        for i, (p, g, n, shape, dt, decay) in enumerate(
                zip(params, grads, self._numel, self.shapes, self.dtypes, self._decay)):
            w = None if masters is None else masters[i]
            try:
                if p.dtype is not dt or p.shape != shape or p.get_device() != where \
                        or not p.is_contiguous():
                    raise ValueError(f"params[{i}]: expected a contiguous {dt} tensor of shape "
                                     f"{tuple(shape)} on {self.device}")
                gd = g.dtype
                if (gd is not dt and gd is not torch.float32) or g.shape != shape \
                        or g.get_device() != where or not g.is_contiguous():
                    raise ValueError(f"grads[{i}]: expected a contiguous tensor like params[{i}], "
                                     "of its dtype or fp32")
                if w is not None and (
                        dt is torch.float32 or w.dtype is not torch.float32 or w.shape != shape
                        or w.get_device() != where or not w.is_contiguous()):
                    raise ValueError(f"masters[{i}]: expected a contiguous fp32 tensor like the "
                                     f"16-bit params[{i}], or None")
                a, b = p.data_ptr(), 0 if w is None else w.data_ptr()
                words += (a, b, g.data_ptr(), n, _CODE[dt] | _CODE[gd] << 32, decay)
            except AttributeError:
                for name, t in (("params", p), ("grads", g), ("masters", w)):
                    if t is not None and not isinstance(t, torch.Tensor):
                        raise TypeError(f"{name}[{i}] must be a torch.Tensor") from None
                raise TypeError(f"params[{i}], grads[{i}]: a tensor is missing") from None
            if n:
                if a in seen or b in seen:
                    raise ValueError(f"params[{i}]: every tensor once, this one or its master "
                                     "is there already")
                seen.add(a)
                if b:
                    seen.add(b)
        return words

    def step(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
             lr: Union[float, torch.Tensor], masters: Optional[Sequence] = None,
             norm: Optional[torch.Tensor] = None, max_norm: Optional[float] = None,
             stream=None) -> None:
        """Steps the parameters, and their fp32 masters where given (a list with a tensor or
        None for each), in place.  lr: a number, or one fp32 on the device (which a captured step
        reads at every replay).  norm: one fp32 on the device, MoEGradClip.norm of the
        gradients: they are clipped to max_norm by it on the way (not in memory), and where it is
        not finite the step does nothing and does not count."""
        n = len(self.shapes)
        for name, ts in (("params", params), ("grads", grads), ("masters", masters)):
            if (ts is not None or name != "masters") and len(ts) != n:
                raise ValueError(f"{name}: expected {n} tensors, got {len(ts)}")
        words = array("Q", self._words(params, grads, masters))
        lr_dev = None
        if isinstance(lr, torch.Tensor):
            self._scalar(lr, "lr")
            lr_dev, lr = lr, 0.0
        if norm is not None:
            self._scalar(norm, "norm")
        elif max_norm is not None:
            raise ValueError("max_norm needs the gradients' norm (MoEGradClip.norm)")
        if max_norm is not None and not max_norm >= 0.0:
            raise ValueError(f"max_norm must be >= 0, got {max_norm}")
        self._opt.max_norm = float("inf") if max_norm is None else max_norm
        _on(self.device, B.mm_moe_adamw_step, self._opt, words.buffer_info()[0], n, self.m,
            self.m_scale, self.v, self.v_scale, self.counter, lr, lr_dev, norm,
            _stream(stream, self.device, self.m, self.m_scale, self.v, self.v_scale, self.counter))

    def _scalar(self, t, name):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not torch.float32 or t.numel() != 1 or t.get_device() != self._where:
            raise ValueError(f"{name}: expected one fp32 on {self.device}")

    def moments(self, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(m, v) of all tensors, flat: self.m and self.v themselves in fp32; of 8-bit states
        the values that they stand for, in bf16."""
        if self.states == "fp32":
            return self.m, self.v
        m, v = (torch.empty(self.m.shape, dtype=torch.bfloat16, device=self.device)
                for _ in range(2))
        _on(self.device, B.mm_moe_adamw_moments, self.m, self.m_scale, self.v, self.v_scale, m, v,
            _stream(stream, self.device, m, v, self.m, self.m_scale, self.v, self.v_scale))
        return m, v
