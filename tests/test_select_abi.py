"""Refusals of the choice of experts, before anything touches a device (no GPU needed)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_16_gb300 import MoERouter, MoESelect
from mixture_experts_layer_16_gb300 import binding as B
from mixture_experts_layer_16_gb300 import build

EI = B.MM_MOE_EINVAL
P = [(1 << 30) * (i + 1) for i in range(16)]     # aligned addresses that are never read
GOOD = dict(T=16, E=64, k=4, dtype=2, grad_dtype=2, score=1, groups=8, topk_groups=2, group_score=1,
            renormalise=1, scale=1.0)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(T=1 << 31), dict(E=0), dict(E=1025, groups=1, topk_groups=1), dict(k=0), dict(k=17),
    dict(k=33, topk_groups=8), dict(dtype=3), dict(grad_dtype=1), dict(dtype=0, grad_dtype=2),
    dict(score=2), dict(score=-1), dict(groups=0), dict(groups=5), dict(groups=64, topk_groups=64),
    dict(topk_groups=0), dict(topk_groups=9), dict(group_score=2), dict(renormalise=2),
    dict(scale=float("inf")), dict(scale=float("nan"))])
def test_shapes(lib, bad):
    s = ctypes.byref(B.Select(*{**GOOD, **bad}.values()))
    assert lib.mm_moe_select_forward(s, *P[:4], None) == EI
    assert lib.mm_moe_select_backward(s, *P[:5], None) == EI


def test_pointers(lib):
    s = ctypes.byref(B.Select(*GOOD.values()))
    fwd = P[:4] + [None]
    for i, v in ((0, None), (0, P[0] + 2), (1, P[1] + 1), (2, None), (2, P[2] + 2), (3, None)):
        a = list(fwd)
        a[i] = v
        assert lib.mm_moe_select_forward(s, *a) == EI, (i, v)
    bwd = P[:5] + [None]
    for i, v in ((0, None), (1, None), (1, P[1] + 1), (2, None), (3, P[3] + 2), (4, None),
                 (4, P[4] + 2), (4, P[0]), (4, P[0] + 16 * 64 * 4 - 4), (4, P[3] + 64)):
        a = list(bwd)
        a[i] = v
        assert lib.mm_moe_select_backward(s, *a) == EI, (i, v)
    assert lib.mm_moe_select_forward(None, *fwd) == EI


def test_router(lib):
    shape = ctypes.byref(B.make_shape(16, 128, 64, 64, 4))
    good = {**GOOD, "grad_dtype": 0}
    for bad in (dict(T=17), dict(E=128), dict(k=5), dict(dtype=0), dict(grad_dtype=2)):
        q = ctypes.byref(B.Select(*{**good, **bad}.values()))
        assert lib.mm_moe_router_select_forward(shape, q, *P[:6], None) == EI, bad
        assert lib.mm_moe_router_select_backward(shape, q, *P[:9], None) == EI, bad
    q = ctypes.byref(B.Select(*good.values()))
    for i, v in ((0, None), (1, P[1] + 8), (2, P[2] + 2), (3, None), (4, None), (5, P[5] + 1)):
        a = P[:6] + [None]
        a[i] = v
        assert lib.mm_moe_router_select_forward(shape, q, *a) == EI, (i, v)
    for i, v in ((0, None), (1, None), (2, P[2] + 4), (3, None), (4, None), (5, P[5] + 2), (6, None),
                 (7, P[7] + 8), (8, None)):
        a = P[:9] + [None]
        a[i] = v
        assert lib.mm_moe_router_select_backward(shape, q, *a) == EI, (i, v)


def test_handle(lib):
    for kw in (dict(score="relu"), dict(group_score="sum"), dict(groups=5), dict(groups=0),
               dict(groups=64, topk_groups=64), dict(topk_groups=2), dict(k=65), dict(k=0), dict(T=0),
               dict(E=2000), dict(dtype="fp8"), dict(grad_dtype="fp16"), dict(scale=float("nan")),
               dict(groups=16, topk_groups=1, k=5), dict(k=33)):
        with pytest.raises(ValueError):
            MoESelect(**{**dict(T=16, E=64, k=4, device="cpu"), **kw})
    h = MoESelect(16, 64, 4, "sigmoid", 8, 2, "top2", device="cpu")
    l, b = torch.zeros(16, 64), torch.zeros(64)
    idx, g = torch.zeros(16, 4, dtype=torch.int32), torch.zeros(16, 4)
    for args in ((l.bfloat16(), b), (l[:15], b), (l.t().contiguous().t(), b), (l, b[:63]),
                 (l, b.double()), (l, b.bfloat16())):
        with pytest.raises(ValueError):
            h.forward(*args)
    with pytest.raises(TypeError):
        h.forward(None)
    for kw in (dict(logits=l.half()), dict(topk_idx=idx.long()), dict(topk_idx=idx[:, :3]),
               dict(dtopk_w=g.bfloat16()), dict(dlogits_aux=l.bfloat16()), dict(dlogits_aux=l[:3]),
               dict(dlogits=l.bfloat16()), dict(dlogits=l[:, :63])):
        with pytest.raises(ValueError):
            h.backward(**{**dict(logits=l, topk_idx=idx, dtopk_w=g), **kw})
    with pytest.raises(TypeError):
        MoERouter(16, 128, 64, 4, device="cpu", select=dict(top=3))


def test_router_backward_needs_a_forward():
    T, H, E, k = 16, 128, 64, 4
    r = MoERouter(T, H, E, k, device="cpu", select={})
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(RuntimeError):
        r.backward(torch.zeros(T, H, **bf), torch.zeros(E, H, **bf),
                   torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k), torch.zeros(T, k),
                   torch.zeros(T, H, **bf))
