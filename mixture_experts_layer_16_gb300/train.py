"""The operators a training step needs around MoELayer: MoELayerNorm in front of it,
MoEBalanceLoss on the router's logits, MoEGradClip over the step's gradients.

Like MoELayer these are handles that own their small device buffers (torch allocations),
check tensor dtypes, shapes and devices, and forward every call to the C ABI.  No
arithmetic happens here.  `stream` is the stream a call runs on (a torch stream or a raw handle;
the current one by default).  The caller orders it after what made the call's tensors, and after
the current stream, from whose memory the handle's own and the returned ones come.
"""
from __future__ import annotations

from array import array
from typing import Optional, Sequence, Tuple

import torch

from . import binding as B
from .layer import _need

TORCH_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_CODE = {TORCH_DTYPE[n]: c for n, c in B.DTYPE.items()}
_TWO = torch.Size((2,))


def _device(device) -> torch.device:
    device = torch.device("cuda" if device is None else device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


def _dtype(name: str) -> torch.dtype:
    if name not in TORCH_DTYPE:
        raise ValueError(f"dtype must be one of {tuple(TORCH_DTYPE)}, got {name!r}")
    return TORCH_DTYPE[name]


def _stream(stream, device: torch.device, *mine: Optional[torch.Tensor]) -> int:
    """The stream of a call, the current one unless the caller names another.  `mine`: the tensors
    that the handle holds or made for this call, from the current stream's memory; on another
    stream they are marked as in use there, so that none of it is handed out again before that
    stream is done with it."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    raw = int(getattr(stream, "cuda_stream", stream))
    where = torch.cuda.ExternalStream(raw, device=device)
    for t in mine:
        if t is not None:
            t.record_stream(where)
    return raw


def _on(device: torch.device, fn, *args):
    """fn(*args) with `device` the current one (the library launches on the current device)."""
    if device.index is None or torch.cuda.current_device() == device.index:
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


def _plain(t, shape: torch.Size, dtype, where: int) -> bool:
    """A contiguous tensor of this shape and dtype on CUDA device `where` (-1: the CPU)."""
    try:
        return (t.dtype is dtype and t.shape == shape and t.get_device() == where
                and t.is_contiguous())
    except AttributeError:
        return False


def _need_rows(t, name: str, shape, dtype, device) -> None:
    """As _need, but the rows may lie apart (a slice of wider rows)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected device {device}, got {t.device}")
    T, H = shape
    ld, one = t.stride()
    if (H > 1 and one != 1) or (T > 1 and ld < H):
        raise ValueError(f"{name}: each row must be contiguous, rows at least {H} apart")


class MoELayerNorm:
    """Layer normalisation of T tokens of H channels: y = weight (x - mean) rstd + bias.

    dtype: of x, y and their gradients; param_dtype: of weight, bias and theirs (dtype
    itself, the default, or "fp32").  The forward keeps the mean and the reciprocal
    standard deviation of every token (self.mean, self.rstd, fp32) for its backward."""

    def __init__(self, T: int, H: int, dtype: str = "bf16", param_dtype: Optional[str] = None,
                 eps: float = 1e-5, bias: bool = True, device: Optional[torch.device] = None):
        param_dtype = dtype if param_dtype is None else param_dtype
        self.T, self.H, self.eps, self.bias = T, H, eps, bias
        self.dtype, self.param_dtype = _dtype(dtype), _dtype(param_dtype)
        self.device = _device(device)
        self.shape = B.NormShape(int(T), int(H), B.DTYPE[dtype], B.DTYPE[param_dtype], eps)
        n = B.mm_moe_norm_workspace_size(self.shape)
        self.mean = torch.empty(T, dtype=torch.float32, device=self.device)
        self.rstd = torch.empty(T, dtype=torch.float32, device=self.device)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)
        self._rows, self._cols = torch.Size((T, H)), torch.Size((H,))
        self._ran = False  # a forward has left what a backward reads
        self._where = -1 if self.device.index is None else self.device.index

    def _check_rows(self, t, name):
        if not _plain(t, self._rows, self.dtype, self._where):
            _need_rows(t, name, self._rows, self.dtype, self.device)

    def _check_param(self, t, name):
        if not _plain(t, self._cols, self.param_dtype, self._where):
            _need(t, name, self._cols, self.param_dtype, self.device)

    def _check_params(self, weight, bias, prefix=""):
        self._check_param(weight, prefix + "weight")
        if self.bias:
            self._check_param(bias, prefix + "bias")
        elif bias is not None:
            raise ValueError(f"{prefix}bias: this layer norm has none")

    def forward(self, x, weight, bias=None, y: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """y may be x itself (in place); rows that overlap otherwise are refused (MoEError)."""
        self._check_rows(x, "x")
        self._check_params(weight, bias)
        if y is None:
            y = torch.empty(self._rows, dtype=self.dtype, device=self.device)
        else:
            self._check_rows(y, "y")
        B.mm_moe_norm_forward(self.shape, x, weight, bias, y, self.mean, self.rstd,
                              _stream(stream, self.device, y, self.mean, self.rstd))
        self._ran = True
        return y

    def backward(self, dy, x, weight, dx_add=None, out=None, stream=None
                 ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
        """Gradients (dx, dweight, dbias) of the last forward, whose x and weight are given
        again (dbias None without a bias).  dx_add: a gradient that joins dx (the residual
        path's); dx may be written over it (out), but not over x or dy (MoEError)."""
        self._check_rows(dy, "dy")
        self._check_rows(x, "x")
        self._check_param(weight, "weight")
        if dx_add is not None:
            self._check_rows(dx_add, "dx_add")
        if out is None:
            out = (torch.empty(self._rows, dtype=self.dtype, device=self.device),
                   torch.empty_like(weight), torch.empty_like(weight) if self.bias else None)
        else:
            self._check_rows(out[0], "dx")
            self._check_params(out[1], out[2], "d")
        if not self._ran:
            raise RuntimeError("backward needs a forward first")
        dx, dweight, dbias = out
        B.mm_moe_norm_backward(self.shape, dy, x, weight, self.mean, self.rstd, dx_add, dx,
                               dweight, dbias, self.workspace,
                               _stream(stream, self.device, dx, dweight, dbias, self.mean,
                                       self.rstd, self.workspace))
        return dx, dweight, dbias


class MoEBalanceLoss:
    """The router's balance and z losses over T tokens in `sequences` sequences, with the
    per-expert counts, and their logit gradient.

    The forward takes the router's logits and topk_idx and returns (losses [2] fp32: the
    balance and the z loss; counts [sequences, E] int32).  seq_offsets [sequences + 1]
    int32 (ascending, on the device) splits the tokens; a token whose mask is 0 does not
    count.  self.seq_loss, self.tokens, self.lse hold each sequence's balance loss, its
    counting tokens and each token's log-sum-exp.  All of these are the handle's own
    tensors, which the next forward overwrites."""

    def __init__(self, T: int, E: int, k: int, sequences: int = 1, dtype: str = "fp32",
                 device: Optional[torch.device] = None):
        self.T, self.E, self.k, self.G = T, E, k, sequences
        self.dtype = _dtype(dtype)
        self.device = _device(device)
        self.shape = B.BalanceShape(int(T), int(E), int(k), int(sequences), B.DTYPE[dtype])
        n = B.mm_moe_balance_workspace_size(self.shape)
        f, i, d = torch.float32, torch.int32, self.device
        self.losses = torch.empty(2, dtype=f, device=d)
        self.seq_loss = torch.empty(sequences, dtype=f, device=d)
        self.counts = torch.empty((sequences, E), dtype=i, device=d)
        self.tokens = torch.empty(sequences, dtype=i, device=d)
        self.lse = torch.empty(T, dtype=f, device=d)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=d)
        self._rows, self._slots = torch.Size((T, E)), torch.Size((T, k))
        self._tokens, self._offsets = torch.Size((T,)), torch.Size((sequences + 1,))
        self._ran = False  # a forward has left what a backward reads
        self._where = -1 if d.index is None else d.index

    def _need(self, t, name, shape, dtype):
        if not _plain(t, shape, dtype, self._where):
            _need(t, name, shape, dtype, self.device)

    def _check(self, logits, seq_offsets, mask):
        self._need(logits, "logits", self._rows, self.dtype)
        if seq_offsets is not None:
            self._need(seq_offsets, "seq_offsets", self._offsets, torch.int32)
        elif self.G != 1:
            raise ValueError("seq_offsets: needed for more than one sequence")
        if mask is not None and not _plain(mask, self._tokens, torch.bool, self._where):
            self._need(mask, "mask", self._tokens, torch.uint8)

    def forward(self, logits, topk_idx, seq_offsets=None, mask=None, stream=None
                ) -> Tuple[torch.Tensor, torch.Tensor]:
        self._check(logits, seq_offsets, mask)
        self._need(topk_idx, "topk_idx", self._slots, torch.int32)
        B.mm_moe_balance_forward(self.shape, logits, topk_idx, seq_offsets, mask, self.losses,
                                 self.seq_loss, self.counts, self.tokens, self.lse,
                                 self.workspace,
                                 _stream(stream, self.device, self.losses, self.seq_loss,
                                         self.counts, self.tokens, self.lse, self.workspace))
        self._ran = True
        return self.losses, self.counts

    def backward(self, logits, dlosses, seq_offsets=None, mask=None,
                 dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The logit gradient of dlosses[0] balance + dlosses[1] z (dlosses [2] fp32 on the
        device) of the last forward, whose logits, seq_offsets and mask are given again.
        MoERouter.backward takes it as dlogits_aux.  It must not overlap the logits (MoEError)."""
        self._check(logits, seq_offsets, mask)
        self._need(dlosses, "dlosses", _TWO, torch.float32)
        if dlogits is None:
            dlogits = torch.empty_like(logits)
        else:
            self._need(dlogits, "dlogits", self._rows, self.dtype)
        if not self._ran:
            raise RuntimeError("backward needs a forward first")
        B.mm_moe_balance_backward(self.shape, logits, seq_offsets, mask, self.counts, self.tokens,
                                  dlosses, dlogits, self.workspace,
                                  _stream(stream, self.device, dlogits, self.counts, self.tokens,
                                          self.workspace))
        return dlogits


class MoEGradClip:
    """The global L2 norm of up to max_tensors gradients, and clipping by it: every
    gradient times min(1, max_norm / (norm + eps)).  What is clipped must not overlap another
    gradient or output: in place, each tensor once."""

    def __init__(self, max_tensors: int = 1024, eps: float = 1e-6,
                 device: Optional[torch.device] = None):
        self.max_tensors, self.eps = max_tensors, eps
        self.device = _device(device)
        n = B.mm_moe_grad_workspace_size(max_tensors)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=self.device)

    def _entries(self, grads: Sequence[torch.Tensor], out):
        """The call's mm_moe_grad array: four 64-bit words a tensor."""
        if len(grads) > self.max_tensors:
            raise ValueError(f"grads: {len(grads)} tensors, made for at most {self.max_tensors}")
        if out is not None and len(out) != len(grads):
            raise ValueError(f"out: expected {len(grads)} tensors, got {len(out)}")
        try:
            return array("Q", self._words(grads, out))
        except AttributeError:  # (looked for only now: short lists are bound by the host)
            for name, ts in (("grads", grads), ("out", out or ())):
                for i, t in enumerate(ts):
                    if not isinstance(t, torch.Tensor):
                        raise TypeError(f"{name}[{i}] must be a torch.Tensor") from None
            raise

    def _words(self, grads, out):
        where = -1 if self.device.index is None else self.device.index
        words = []
        for i, g in enumerate(grads):
            d = _CODE.get(g.dtype)
            if d is None or g.get_device() != where or not g.is_contiguous():
                raise ValueError(f"grads[{i}]: expected a contiguous bf16, fp16 or fp32 tensor "
                                 f"on {self.device}")
            p = g.data_ptr()
            if out is None:
                words += (p, p, g.numel(), d | d << 32)
                continue
            o = out[i]
            od = _CODE.get(o.dtype)
            if (od != d and od != B.MM_MOE_DT_F32) or o.get_device() != where \
                    or not o.is_contiguous() or o.shape != g.shape:
                raise ValueError(f"out[{i}]: expected a contiguous tensor like grads[{i}], of "
                                 "its dtype or fp32")
            words += (p, o.data_ptr(), g.numel(), d | od << 32)
        return words

    def norm(self, grads: Sequence[torch.Tensor], stream=None) -> torch.Tensor:
        """The norm as a 0-d fp32 tensor on the device (no synchronisation)."""
        norm = torch.empty((), dtype=torch.float32, device=self.device)
        B.mm_moe_grad_norm(self._entries(grads, None), norm, self.workspace,
                           _stream(stream, self.device, norm, self.workspace))
        return norm

    def clip(self, grads: Sequence[torch.Tensor], max_norm: float, out=None,
             stream=None) -> torch.Tensor:
        """Clips in place, or into `out` (tensors of the gradients' dtypes or fp32);
        returns the norm before clipping as a 0-d fp32 tensor on the device."""
        if not max_norm >= 0.0:
            raise ValueError(f"max_norm must be >= 0, got {max_norm}")
        norm = torch.empty((), dtype=torch.float32, device=self.device)
        B.mm_moe_grad_clip(self._entries(grads, out), max_norm, self.eps, norm, self.workspace,
                           _stream(stream, self.device, norm, self.workspace))
        return norm
