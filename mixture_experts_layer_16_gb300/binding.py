"""Thin ctypes binding of libmm_moe.so (include/mm_moe.h).

Argument marshalling only: every step of the layer runs in the CUDA library.
PyTorch is used for device memory and streams.  There is no fallback: if the
library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import array
import ctypes
import os
from typing import Optional, Tuple

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmm_moe.so")

MM_MOE_BF16, MM_MOE_MXFP8, MM_MOE_FP8_BWD, MM_MOE_FP8_BLOCK = 0, 1, 2, 3
PRECISION = {"bf16": MM_MOE_BF16, "mxfp8": MM_MOE_MXFP8, "fp8_bwd": MM_MOE_FP8_BWD,
             "fp8_block": MM_MOE_FP8_BLOCK}
STATUS = {0: "MM_MOE_OK", 1: "MM_MOE_EINVAL", 2: "MM_MOE_ENOTSUP", 3: "MM_MOE_EBADIDX",
          4: "MM_MOE_ETIMEOUT", 5: "MM_MOE_ECUDA"}
MM_MOE_OK, MM_MOE_EINVAL, MM_MOE_ENOTSUP, MM_MOE_EBADIDX, MM_MOE_ETIMEOUT, MM_MOE_ECUDA = range(6)

# every symbol include/mm_moe.h declares
EXPORTS = ("mm_moe_workspace_size", "mm_moe_forward", "mm_moe_backward", "mm_moe_get_routing",
           "mm_moe_read_status", "mm_moe_last_launch_count", "mm_moe_profile_start",
           "mm_moe_profile_stop", "mm_moe_kernel_name", "mm_moe_kernel_count",
           "mm_moe_route_noalloc", "mm_moe_mx_qdq", "mm_moe_router_forward",
           "mm_moe_router_backward", "mm_moe_fp8_block_qdq", "mm_moe_mx_quantize",
           "mm_moe_fp8_block_quantize", "mm_moe_router_backward_aux",
           "mm_moe_norm_workspace_size", "mm_moe_norm_forward", "mm_moe_norm_backward",
           "mm_moe_balance_workspace_size", "mm_moe_balance_forward", "mm_moe_balance_backward",
           "mm_moe_grad_workspace_size", "mm_moe_grad_norm", "mm_moe_grad_clip",
           "mm_moe_adamw_step", "mm_moe_adamw_moments", "mm_moe_select_forward",
           "mm_moe_select_backward", "mm_moe_router_select_forward",
           "mm_moe_router_select_backward", "mm_moe_resnorm_workspace_size",
           "mm_moe_resnorm_forward", "mm_moe_resnorm_backward")


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64),
                ("E", ctypes.c_int64), ("k", ctypes.c_int64), ("prec", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


# element types of the operators around the layer (mm_moe_dtype)
MM_MOE_DT_BF16, MM_MOE_DT_F16, MM_MOE_DT_F32 = 0, 1, 2
DTYPE = {"bf16": MM_MOE_DT_BF16, "fp16": MM_MOE_DT_F16, "fp32": MM_MOE_DT_F32}
MM_MOE_MAX_GRADS = 65536


class NormShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class BalanceShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int64), ("k", ctypes.c_int64),
                ("G", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class Grad(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


# moments of AdamW (mm_moe_states)
MM_MOE_STATES_F32, MM_MOE_STATES_8BIT = 0, 1
STATES = {"fp32": MM_MOE_STATES_F32, "8bit": MM_MOE_STATES_8BIT}


class AdamW(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("max_norm", ctypes.c_float), ("clip_eps", ctypes.c_float),
                ("states", ctypes.c_int32), ("seed", ctypes.c_uint32)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("weight_decay", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


# forms of the choice of experts (mm_moe_score, mm_moe_group_score)
SCORE = {"softmax": 0, "sigmoid": 1}
GROUP_SCORE = {"max": 0, "top2": 1}


class Select(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int64), ("k", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_score", ctypes.c_int32),
                ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float)]


# gates of the residual norm (mm_moe_gate)
GATE = {None: 0, "channel": 1, "token": 2}


class ResNorm(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("post", ctypes.c_int32), ("gate", ctypes.c_int32), ("pre", ctypes.c_int32),
                ("scale", ctypes.c_float), ("eps", ctypes.c_float)]


MM_MOE_RECOMPUTE = 1  # activation checkpointing (include/mm_moe.h)
MM_MOE_MULTICAST = 2  # A-multicast clusters of two SM pairs (include/mm_moe.h)


def _ranks() -> int:
    """Ranks of the job that this process belongs to."""
    import torch.distributed as dist
    if dist.is_available() and dist.is_initialized():
        return dist.get_world_size()
    return int(os.environ.get("WORLD_SIZE") or 1)


def make_shape(T, H, I, E, k, prec="bf16", recompute: bool = False,
               multicast: bool = False) -> Shape:
    """multicast: in a job of one GPU only (its loads are for code that runs alone)."""
    if multicast and _ranks() > 1:
        raise ValueError(f"multicast is for jobs of one GPU, this one has {_ranks()} ranks")
    return Shape(int(T), int(H), int(I), int(E), int(k), PRECISION.get(prec, prec),
                 (MM_MOE_RECOMPUTE if recompute else 0) | (MM_MOE_MULTICAST if multicast else 0))


_lib: Optional[ctypes.CDLL] = None
_vp = ctypes.c_void_p


def lib() -> ctypes.CDLL:
    """Load the library once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "mixture_experts_layer_16_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        sp = ctypes.POINTER(Shape)
        L.mm_moe_workspace_size.argtypes = [sp, ctypes.POINTER(ctypes.c_size_t),
                                            ctypes.POINTER(ctypes.c_size_t)]
        L.mm_moe_forward.argtypes = [sp] + [_vp] * 10
        L.mm_moe_backward.argtypes = [sp] + [_vp] * 13
        L.mm_moe_get_routing.argtypes = [sp, _vp, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                         ctypes.POINTER(_vp)]
        L.mm_moe_read_status.argtypes = [_vp, _vp]
        L.mm_moe_last_launch_count.argtypes = []
        L.mm_moe_profile_start.argtypes = []
        L.mm_moe_profile_stop.argtypes = [ctypes.POINTER(ctypes.c_float),
                                          ctypes.POINTER(ctypes.c_int), ctypes.c_int]
        L.mm_moe_kernel_name.argtypes = [ctypes.c_int]
        L.mm_moe_kernel_count.argtypes = []
        L.mm_moe_route_noalloc.argtypes = [sp] + [_vp] * 6
        L.mm_moe_mx_qdq.argtypes = [_vp, _vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, _vp]
        L.mm_moe_fp8_block_qdq.argtypes = [_vp, _vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                           _vp]
        L.mm_moe_mx_quantize.argtypes = [_vp, _vp, _vp, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_int, _vp]
        L.mm_moe_fp8_block_quantize.argtypes = [_vp, _vp, _vp, ctypes.c_int64, ctypes.c_int64,
                                                ctypes.c_int, _vp]
        L.mm_moe_router_forward.argtypes = [sp] + [_vp] * 6
        L.mm_moe_router_backward.argtypes = [sp] + [_vp] * 9
        L.mm_moe_router_backward_aux.argtypes = [sp] + [_vp] * 10
        i64, szp = ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)
        nsp, bsp = ctypes.POINTER(NormShape), ctypes.POINTER(BalanceShape)
        L.mm_moe_norm_workspace_size.argtypes = [nsp, szp]
        L.mm_moe_norm_forward.argtypes = [nsp, _vp, i64, _vp, _vp, _vp, i64, _vp, _vp, _vp]
        L.mm_moe_norm_backward.argtypes = [nsp, _vp, i64, _vp, i64, _vp, _vp, _vp, _vp, i64, _vp,
                                           i64, _vp, _vp, _vp, _vp]
        L.mm_moe_balance_workspace_size.argtypes = [bsp, szp]
        L.mm_moe_balance_forward.argtypes = [bsp] + [_vp] * 11
        L.mm_moe_balance_backward.argtypes = [bsp] + [_vp] * 9
        L.mm_moe_grad_workspace_size.argtypes = [i64, szp]
        L.mm_moe_grad_norm.argtypes = [_vp, i64, _vp, _vp, _vp]
        L.mm_moe_grad_clip.argtypes = [_vp, i64, ctypes.c_float, ctypes.c_float, _vp, _vp, _vp]
        L.mm_moe_adamw_step.argtypes = [ctypes.POINTER(AdamW), _vp, i64] + [_vp] * 5 + \
            [ctypes.c_double] + [_vp] * 3
        L.mm_moe_adamw_moments.argtypes = [_vp] * 4 + [i64] + [_vp] * 3
        qp = ctypes.POINTER(Select)
        L.mm_moe_select_forward.argtypes = [qp] + [_vp] * 5
        L.mm_moe_select_backward.argtypes = [qp] + [_vp] * 6
        L.mm_moe_router_select_forward.argtypes = [sp, qp] + [_vp] * 7
        L.mm_moe_router_select_backward.argtypes = [sp, qp] + [_vp] * 10
        rp = ctypes.POINTER(ResNorm)
        L.mm_moe_resnorm_workspace_size.argtypes = [rp, szp]
        L.mm_moe_resnorm_forward.argtypes = [rp, _vp, i64, _vp, i64] + [_vp] * 4 + \
            [i64, _vp, i64] + [_vp] * 3
        L.mm_moe_resnorm_backward.argtypes = [rp] + [_vp, i64] * 4 + [_vp] * 5 + \
            [_vp, i64] * 2 + [_vp] * 5
        for fn in EXPORTS:
            getattr(L, fn).restype = ctypes.c_int
        L.mm_moe_kernel_name.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    return int(getattr(stream, "cuda_stream", stream))


def _check(fn: str, st: int) -> None:
    if st != MM_MOE_OK:
        raise MoEError(fn, st)


def mm_moe_workspace_size(shape: Shape) -> Tuple[int, int]:
    sc, sv = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("mm_moe_workspace_size",
           lib().mm_moe_workspace_size(ctypes.byref(shape), ctypes.byref(sc), ctypes.byref(sv)))
    return sc.value, sv.value


def mm_moe_forward(shape: Shape, x, topk_idx, topk_w, W_gate, W_up, W_down, y, scratch, saved,
                   stream=None, check: bool = True) -> int:
    st = lib().mm_moe_forward(ctypes.byref(shape), _ptr(x), _ptr(topk_idx), _ptr(topk_w),
                              _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(y), _ptr(scratch),
                              _ptr(saved), _stream(stream))
    if check:
        _check("mm_moe_forward", st)
    return st


def mm_moe_backward(shape: Shape, dy, saved, W_gate, W_up, W_down, x, dx, dW_gate, dW_up,
                    dW_down, dtopk_w, scratch, stream=None, check: bool = True) -> int:
    st = lib().mm_moe_backward(ctypes.byref(shape), _ptr(dy), _ptr(saved), _ptr(W_gate),
                               _ptr(W_up), _ptr(W_down), _ptr(x), _ptr(dx), _ptr(dW_gate),
                               _ptr(dW_up), _ptr(dW_down), _ptr(dtopk_w), _ptr(scratch),
                               _stream(stream))
    if check:
        _check("mm_moe_backward", st)
    return st


def mm_moe_get_routing(shape: Shape, saved):
    """Views of `saved` (a uint8 device tensor): offsets [E+1], perm [T*k], inv [T*k], int32."""
    import torch
    o, p, i = _vp(), _vp(), _vp()
    _check("mm_moe_get_routing",
           lib().mm_moe_get_routing(ctypes.byref(shape), _ptr(saved), ctypes.byref(o),
                                    ctypes.byref(p), ctypes.byref(i)))
    base = saved.data_ptr()
    R = shape.T * shape.k

    def view(ptr, n):
        off = ptr.value - base
        return saved[off:off + 4 * n].view(torch.int32)
    return view(o, shape.E + 1), view(p, R), view(i, R)


def mm_moe_route_noalloc(shape: Shape, topk_idx, topk_w, offsets, perm, inv, stream=None,
                         check: bool = True) -> int:
    """Routing into caller-provided offsets/perm/inv with no scratch buffer (the
    library's own fixed device array is used; calls on different streams race)."""
    st = lib().mm_moe_route_noalloc(ctypes.byref(shape), _ptr(topk_idx), _ptr(topk_w),
                                    _ptr(offsets), _ptr(perm), _ptr(inv), _stream(stream))
    if check:
        _check("mm_moe_route_noalloc", st)
    return st


def mm_moe_mx_qdq(inp, out, axis: int, stream=None) -> None:
    """MXFP8 quantise-dequantise of a 2-D bf16 CUDA tensor into `out` (may be `inp`):
    32-element blocks along rows (axis=1) or down columns (axis=0)."""
    import torch
    if inp.dim() != 2 or inp.dtype != torch.bfloat16 or not inp.is_contiguous():
        raise ValueError("inp must be a contiguous 2-D bf16 tensor")
    if out.shape != inp.shape or out.dtype != inp.dtype or not out.is_contiguous():
        raise ValueError("out must match inp")
    _check("mm_moe_mx_qdq", lib().mm_moe_mx_qdq(_ptr(inp), _ptr(out), inp.shape[0],
                                                inp.shape[1], int(axis), _stream(stream)))


def mm_moe_mx_quantize(inp, codes, scales, axis: int, stream=None) -> None:
    """MXFP8 quantisation of a 2-D bf16 CUDA tensor [rows, cols] (multiples of 128)
    into e4m3 codes (uint8, same shape) and E8M0 scales (uint8, rows * cols / 32 bytes
    in the block-scaled tensor cores' atom arrangement): 32-element blocks along rows
    (axis=1) or down columns (axis=0)."""
    import torch
    if inp.dim() != 2 or inp.dtype != torch.bfloat16 or not inp.is_contiguous():
        raise ValueError("inp must be a contiguous 2-D bf16 tensor")
    if codes.shape != inp.shape or codes.dtype != torch.uint8 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous uint8 tensor of inp's shape")
    if scales.dtype != torch.uint8 or scales.numel() != inp.numel() // 32:
        raise ValueError("scales must hold rows * cols / 32 uint8")
    _check("mm_moe_mx_quantize", lib().mm_moe_mx_quantize(
        _ptr(inp), _ptr(codes), _ptr(scales), inp.shape[0], inp.shape[1], int(axis),
        _stream(stream)))


def mm_moe_fp8_block_quantize(inp, codes, scales, layout: int, stream=None) -> None:
    """Blockwise FP8 quantisation of a 2-D bf16 CUDA tensor [rows, cols] (multiples of
    128) into e4m3 codes (uint8, same shape) and E8M0 scales (uint8, in the block-scaled
    tensor cores' atom arrangement; rows * cols / 32 bytes, twice that for tiles):
    128-element blocks along rows (layout 0), down columns (1), or 128 x 128 tiles (2)."""
    import torch
    if inp.dim() != 2 or inp.dtype != torch.bfloat16 or not inp.is_contiguous():
        raise ValueError("inp must be a contiguous 2-D bf16 tensor")
    if codes.shape != inp.shape or codes.dtype != torch.uint8 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous uint8 tensor of inp's shape")
    n = inp.numel() // 32 * (2 if int(layout) == 2 else 1)
    if scales.dtype != torch.uint8 or scales.numel() != n:
        raise ValueError("scales must hold rows * cols / 32 uint8 (twice that for tiles)")
    _check("mm_moe_fp8_block_quantize", lib().mm_moe_fp8_block_quantize(
        _ptr(inp), _ptr(codes), _ptr(scales), inp.shape[0], inp.shape[1], int(layout),
        _stream(stream)))


def mm_moe_fp8_block_qdq(inp, out, layout: int, stream=None) -> None:
    """Blockwise FP8 quantise-dequantise of a 2-D bf16 CUDA tensor into `out` (may be
    `inp`): 128-element blocks along rows (layout 0), down columns (1), or 128 x 128
    tiles (2)."""
    import torch
    if inp.dim() != 2 or inp.dtype != torch.bfloat16 or not inp.is_contiguous():
        raise ValueError("inp must be a contiguous 2-D bf16 tensor")
    if out.shape != inp.shape or out.dtype != inp.dtype or not out.is_contiguous():
        raise ValueError("out must match inp")
    _check("mm_moe_fp8_block_qdq", lib().mm_moe_fp8_block_qdq(
        _ptr(inp), _ptr(out), inp.shape[0], inp.shape[1], int(layout), _stream(stream)))


def mm_moe_router_forward(shape: Shape, x, W_router, logits, topk_idx, topk_w, stream=None,
                          check: bool = True) -> int:
    st = lib().mm_moe_router_forward(ctypes.byref(shape), _ptr(x), _ptr(W_router), _ptr(logits),
                                     _ptr(topk_idx), _ptr(topk_w), _stream(stream))
    if check:
        _check("mm_moe_router_forward", st)
    return st


def mm_moe_router_backward(shape: Shape, x, W_router, topk_idx, topk_w, dtopk_w, dlogits, dx,
                           dW_router, stream=None, check: bool = True) -> int:
    st = lib().mm_moe_router_backward(ctypes.byref(shape), _ptr(x), _ptr(W_router),
                                      _ptr(topk_idx), _ptr(topk_w), _ptr(dtopk_w),
                                      _ptr(dlogits), _ptr(dx), _ptr(dW_router), _stream(stream))
    if check:
        _check("mm_moe_router_backward", st)
    return st


def mm_moe_router_backward_aux(shape: Shape, x, W_router, topk_idx, topk_w, dtopk_w, dlogits_aux,
                               dlogits, dx, dW_router, stream=None) -> None:
    _check("mm_moe_router_backward_aux", lib().mm_moe_router_backward_aux(
        ctypes.byref(shape), _ptr(x), _ptr(W_router), _ptr(topk_idx), _ptr(topk_w),
        _ptr(dtopk_w), _ptr(dlogits_aux), _ptr(dlogits), _ptr(dx), _ptr(dW_router),
        _stream(stream)))


def _size(fn: str, arg) -> int:
    n = ctypes.c_size_t(0)
    _check(fn, getattr(lib(), fn)(arg, ctypes.byref(n)))
    return n.value


def mm_moe_norm_workspace_size(shape: NormShape) -> int:
    return _size("mm_moe_norm_workspace_size", ctypes.byref(shape))


def mm_moe_norm_forward(shape: NormShape, x, weight, bias, y, mean, rstd, stream=None) -> None:
    """x and y [T, H] with rows stride(0) elements apart."""
    st = lib().mm_moe_norm_forward(
        shape, x.data_ptr(), x.stride(0), weight.data_ptr(), 0 if bias is None else bias.data_ptr(),
        y.data_ptr(), y.stride(0), mean.data_ptr(), rstd.data_ptr(),
        stream if type(stream) is int else _stream(stream))
    if st:
        _check("mm_moe_norm_forward", st)


def mm_moe_norm_backward(shape: NormShape, dy, x, weight, mean, rstd, dx_add, dx, dweight, dbias,
                         workspace, stream=None) -> None:
    st = lib().mm_moe_norm_backward(
        shape, dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0), weight.data_ptr(),
        mean.data_ptr(), rstd.data_ptr(), 0 if dx_add is None else dx_add.data_ptr(),
        0 if dx_add is None else dx_add.stride(0), dx.data_ptr(), dx.stride(0),
        dweight.data_ptr(), 0 if dbias is None else dbias.data_ptr(), workspace.data_ptr(),
        stream if type(stream) is int else _stream(stream))
    if st:
        _check("mm_moe_norm_backward", st)


def mm_moe_balance_workspace_size(shape: BalanceShape) -> int:
    return _size("mm_moe_balance_workspace_size", ctypes.byref(shape))


def mm_moe_balance_forward(shape: BalanceShape, logits, topk_idx, seq_offsets, mask, losses,
                           seq_loss, counts, tokens, lse, workspace, stream=None) -> None:
    st = lib().mm_moe_balance_forward(
        shape, logits.data_ptr(), topk_idx.data_ptr(),
        0 if seq_offsets is None else seq_offsets.data_ptr(),
        0 if mask is None else mask.data_ptr(), losses.data_ptr(), seq_loss.data_ptr(),
        counts.data_ptr(), tokens.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
        stream if type(stream) is int else _stream(stream))
    if st:
        _check("mm_moe_balance_forward", st)


def mm_moe_balance_backward(shape: BalanceShape, logits, seq_offsets, mask, counts, tokens,
                            dlosses, dlogits, workspace, stream=None) -> None:
    st = lib().mm_moe_balance_backward(
        shape, logits.data_ptr(), 0 if seq_offsets is None else seq_offsets.data_ptr(),
        0 if mask is None else mask.data_ptr(), counts.data_ptr(), tokens.data_ptr(),
        dlosses.data_ptr(), dlogits.data_ptr(), workspace.data_ptr(),
        stream if type(stream) is int else _stream(stream))
    if st:
        _check("mm_moe_balance_backward", st)


def mm_moe_grad_workspace_size(n_tensors: int) -> int:
    return _size("mm_moe_grad_workspace_size", int(n_tensors))


def grad_array(entries):
    """[(grad pointer, out pointer, numel, dtype, out dtype)] as a packed mm_moe_grad array."""
    words = []
    for g, o, n, d, od in entries:
        words += (g, o, n, d | od << 32)
    return array.array("Q", words)


def mm_moe_grad_norm(grads, norm, workspace, stream=None) -> None:
    """grads: a packed mm_moe_grad array (grad_array); the out fields are ignored."""
    p, n = grads.buffer_info()
    _check("mm_moe_grad_norm", lib().mm_moe_grad_norm(p, n // 4, _ptr(norm), _ptr(workspace),
                                                      _stream(stream)))


def mm_moe_grad_clip(grads, max_norm: float, eps: float, norm, workspace, stream=None) -> None:
    """grads: a packed mm_moe_grad array (grad_array)."""
    p, n = grads.buffer_info()
    _check("mm_moe_grad_clip", lib().mm_moe_grad_clip(p, n // 4, max_norm, eps, _ptr(norm),
                                                      _ptr(workspace), _stream(stream)))


def mm_moe_adamw_step(opt: AdamW, tensors, n: int, m, m_scale, v, v_scale, counter, lr: float,
                      lr_dev=None, norm=None, stream=None) -> None:
    """tensors: the address of n packed mm_moe_adamw_tensor."""
    _check("mm_moe_adamw_step", lib().mm_moe_adamw_step(
        opt, tensors, n, _ptr(m), _ptr(m_scale), _ptr(v), _ptr(v_scale), _ptr(counter), lr,
        _ptr(lr_dev), _ptr(norm), _stream(stream)))


def mm_moe_adamw_moments(m, m_scale, v, v_scale, m_out, v_out, stream=None) -> None:
    _check("mm_moe_adamw_moments", lib().mm_moe_adamw_moments(
        _ptr(m), _ptr(m_scale), _ptr(v), _ptr(v_scale), m.numel(), _ptr(m_out), _ptr(v_out),
        _stream(stream)))


def mm_moe_select_forward(select: Select, logits, bias, topk_idx, topk_w, stream=None) -> None:
    st = lib().mm_moe_select_forward(select, logits.data_ptr(), _ptr(bias), topk_idx.data_ptr(),
                                     topk_w.data_ptr(),
                                     stream if type(stream) is int else _stream(stream))
    if st:
        _check("mm_moe_select_forward", st)


def mm_moe_select_backward(select: Select, logits, topk_idx, dtopk_w, dlogits_aux, dlogits,
                           stream=None) -> None:
    st = lib().mm_moe_select_backward(select, logits.data_ptr(), topk_idx.data_ptr(),
                                      dtopk_w.data_ptr(), _ptr(dlogits_aux), dlogits.data_ptr(),
                                      stream if type(stream) is int else _stream(stream))
    if st:
        _check("mm_moe_select_backward", st)


def mm_moe_router_select_forward(shape: Shape, select: Select, x, W_router, bias, logits, topk_idx,
                                 topk_w, stream=None) -> None:
    _check("mm_moe_router_select_forward", lib().mm_moe_router_select_forward(
        ctypes.byref(shape), select, _ptr(x), _ptr(W_router), _ptr(bias), _ptr(logits),
        _ptr(topk_idx), _ptr(topk_w), _stream(stream)))


def mm_moe_router_select_backward(shape: Shape, select: Select, x, W_router, logits, topk_idx,
                                  dtopk_w, dlogits_aux, dlogits, dx, dW_router,
                                  stream=None) -> None:
    _check("mm_moe_router_select_backward", lib().mm_moe_router_select_backward(
        ctypes.byref(shape), select, _ptr(x), _ptr(W_router), _ptr(logits), _ptr(topk_idx),
        _ptr(dtopk_w), _ptr(dlogits_aux), _ptr(dlogits), _ptr(dx), _ptr(dW_router),
        _stream(stream)))


def mm_moe_resnorm_workspace_size(shape: ResNorm) -> int:
    return _size("mm_moe_resnorm_workspace_size", ctypes.byref(shape))


def _rows(t) -> Tuple[int, int]:
    return (0, 0) if t is None else (t.data_ptr(), t.stride(0))


def mm_moe_resnorm_forward(shape: ResNorm, x, f, post_weight, gate, pre_weight, out, n, rstd_f,
                           rstd_out, stream=None) -> None:
    """x, f, out and n [T, H] with rows stride(0) elements apart."""
    # (written out: short calls are bound by the host)
    st = lib().mm_moe_resnorm_forward(
        shape, x.data_ptr(), x.stride(0), 0 if f is None else f.data_ptr(),
        0 if f is None else f.stride(0), 0 if post_weight is None else post_weight.data_ptr(),
        0 if gate is None else gate.data_ptr(), 0 if pre_weight is None else pre_weight.data_ptr(),
        out.data_ptr(), out.stride(0), 0 if n is None else n.data_ptr(),
        0 if n is None else n.stride(0), 0 if rstd_f is None else rstd_f.data_ptr(),
        0 if rstd_out is None else rstd_out.data_ptr(),
        stream if type(stream) is int else _stream(stream))
    if st:
        _check("mm_moe_resnorm_forward", st)


def mm_moe_resnorm_backward(shape: ResNorm, dout, dn, out, f, post_weight, gate, pre_weight, rstd_f,
                            rstd_out, dx, df, dpost_weight, dgate, dpre_weight, workspace,
                            stream=None) -> None:
    st = lib().mm_moe_resnorm_backward(
        shape, *_rows(dout), *_rows(dn), *_rows(out), *_rows(f), _ptr(post_weight), _ptr(gate),
        _ptr(pre_weight), _ptr(rstd_f), _ptr(rstd_out), *_rows(dx), *_rows(df), _ptr(dpost_weight),
        _ptr(dgate), _ptr(dpre_weight), _ptr(workspace),
        stream if type(stream) is int else _stream(stream))
    if st:
        _check("mm_moe_resnorm_backward", st)


def mm_moe_read_status(scratch, stream=None) -> int:
    return int(lib().mm_moe_read_status(_ptr(scratch), _stream(stream)))


def mm_moe_last_launch_count() -> int:
    return int(lib().mm_moe_last_launch_count())


def mm_moe_kernel_count() -> int:
    return int(lib().mm_moe_kernel_count())


def mm_moe_kernel_name(i: int) -> str:
    n = lib().mm_moe_kernel_name(int(i))
    return n.decode() if n else ""


def mm_moe_profile_start() -> None:
    _check("mm_moe_profile_start", lib().mm_moe_profile_start())


def mm_moe_profile_stop():
    """{kernel name: (total ms, launches)} of the calls since mm_moe_profile_start."""
    n = mm_moe_kernel_count()
    ms = (ctypes.c_float * n)()
    cnt = (ctypes.c_int * n)()
    _check("mm_moe_profile_stop", lib().mm_moe_profile_stop(ms, cnt, n))
    return {mm_moe_kernel_name(i): (float(ms[i]), int(cnt[i])) for i in range(n)}


class Workspace:
    """The two caller-owned device buffers of one layer shape, allocated with torch."""

    def __init__(self, shape: Shape, device="cuda"):
        import torch
        self.shape = shape
        sc, sv = mm_moe_workspace_size(shape)
        self.scratch = torch.empty(max(sc, 256), dtype=torch.uint8, device=device)
        self.saved = torch.empty(max(sv, 256), dtype=torch.uint8, device=device)
