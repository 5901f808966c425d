"""Refusals of the residual norm, before anything touches a device (no GPU needed)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEError, MoEResidualNorm
from mixture_experts_layer_16_gb300 import binding as B
from mixture_experts_layer_16_gb300 import build

EI = B.MM_MOE_EINVAL
P = [(1 << 24) * (i + 1) for i in range(20)]     # aligned addresses that are never read
GOOD = dict(T=16, H=64, dtype=0, res_dtype=2, param_dtype=0, post=1, gate=1, pre=1, scale=1.0,
            eps=1e-6)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def fwd():
    return [P[0], 64, P[1], 64, P[2], P[3], P[4], P[5], 64, P[6], 64, P[7], P[8], None]


def bwd():
    return [P[0], 64, P[1], 64, P[2], 64, P[3], 64, P[4], P[5], P[6], P[7], P[8], P[9], 64, P[10], 64,
            P[11], P[12], P[13], P[14], None]


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(T=1 << 31), dict(H=0), dict(H=(1 << 20) + 1), dict(dtype=3), dict(res_dtype=1),
    dict(dtype=2, res_dtype=0), dict(param_dtype=1), dict(post=2), dict(gate=3), dict(gate=-1),
    dict(pre=-1), dict(scale=float("inf")), dict(scale=float("nan")), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf"))])
def test_shapes(lib, bad):
    n = ctypes.c_size_t(0)
    assert lib.mm_moe_resnorm_workspace_size(ctypes.byref(B.ResNorm(*GOOD.values())),
                                             ctypes.byref(n)) == 0 and n.value > 0
    s = ctypes.byref(B.ResNorm(*{**GOOD, **bad}.values()))
    assert lib.mm_moe_resnorm_workspace_size(s, ctypes.byref(n)) == EI
    assert lib.mm_moe_resnorm_forward(s, *fwd()) == EI
    assert lib.mm_moe_resnorm_backward(s, *bwd()) == EI


def test_pointers(lib):
    s = ctypes.byref(B.ResNorm(*GOOD.values()))
    assert lib.mm_moe_resnorm_workspace_size(s, None) == EI
    for i, v in ((0, None), (0, P[0] + 2), (1, 63), (2, P[1] + 1), (3, 63), (4, None), (5, None),
                 (5, P[3] + 1), (6, None), (7, None), (8, 63), (9, None), (10, 63), (11, None),
                 (12, P[8] + 2), (7, P[0] + 256), (7, P[1]), (9, P[1]), (9, P[0]), (9, P[5] + 64)):
        a = fwd()
        a[i] = v
        assert lib.mm_moe_resnorm_forward(s, *a) == EI, (i, v)
    for i, v in ((0, P[0] + 2), (1, 63), (2, None), (3, 63), (4, None), (6, P[3] + 1), (8, None),
                 (9, None), (10, None), (11, None), (12, None), (13, None), (14, 63), (15, None),
                 (16, 63), (17, None), (18, None), (19, None), (20, None), (20, P[14] + 8),
                 (13, P[0]), (13, P[2]), (15, P[3]), (15, P[1]), (15, P[9])):
        a = bwd()
        a[i] = v
        assert lib.mm_moe_resnorm_backward(s, *a) == EI, (i, v)
    plain = ctypes.byref(B.ResNorm(*{**GOOD, "pre": 0}.values()))
    a = fwd()
    a[2] = None                                    # neither a block's output nor a norm
    assert lib.mm_moe_resnorm_forward(plain, *a) == EI
    a = bwd()
    a[0] = None
    assert lib.mm_moe_resnorm_backward(plain, *a) == EI
    a = bwd()
    a[6] = None
    assert lib.mm_moe_resnorm_backward(plain, *a) == EI


def test_handle(lib):
    T, H = 4, 8
    h = MoEResidualNorm(T, H, "bf16", "fp32", "fp32", gate="token", device="cpu")
    x, f = torch.zeros(T, H), torch.zeros(T, H, dtype=torch.bfloat16)
    w, g = torch.ones(H), torch.ones(T)
    good = dict(x=x, f=f, post_weight=w, gate=g, pre_weight=w)
    for kw, exc in ((dict(x=None), TypeError), (dict(x=x.bfloat16()), ValueError),
                    (dict(f=f.float()), ValueError), (dict(f=f[:3]), ValueError),
                    (dict(x=x.t().contiguous().t()), ValueError), (dict(post_weight=None), TypeError),
                    (dict(post_weight=w.bfloat16()), ValueError), (dict(gate=w), ValueError),
                    (dict(gate=None), TypeError), (dict(pre_weight=w[:7]), ValueError),
                    (dict(out=f), ValueError), (dict(f=None), ValueError)):
        with pytest.raises(exc):
            h.forward(**{**good, **kw})
    back = dict(dout=x, dn=f, out=x, f=f, post_weight=w, gate=g, pre_weight=w)
    for kw, exc in ((dict(dout=f), ValueError), (dict(dn=x), ValueError), (dict(dn=None), TypeError),
                    (dict(out=None), TypeError), (dict(gate=w), ValueError),
                    (dict(pre_weight=None), TypeError), (dict(), RuntimeError)):
        with pytest.raises(exc):
            h.backward(**{**back, **kw})
    for kw in (dict(dtype="fp8"), dict(res_dtype="fp16"), dict(param_dtype="fp16"), dict(gate="head")):
        with pytest.raises((ValueError, MoEError)):
            MoEResidualNorm(**{**dict(T=T, H=H, dtype="bf16", device="cpu"), **kw})
    with pytest.raises(MoEError):
        MoEResidualNorm(T, 0, device="cpu")
    p = MoEResidualNorm(T, H, "fp32", post=False, pre=False, device="cpu")
    for a in ((x,), (x, x, w)):
        with pytest.raises(ValueError):
            p.forward(*a)
    with pytest.raises(ValueError):
        p.load_stats(g)
