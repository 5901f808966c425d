"""Refusals of the training-step operators, before anything touches a device (no GPU
needed): the C ABI's status for bad shapes, types, pointers and counts, and the
exceptions of the Python handles' argument checks."""
import ctypes

import pytest
import torch

from mixture_experts_layer_16_gb300 import binding as B
from mixture_experts_layer_16_gb300 import build
from mixture_experts_layer_16_gb300 import train

EI = B.MM_MOE_EINVAL
P = [4096 * (i + 1) for i in range(16)]     # aligned addresses that are never read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def size(fn, *a):
    return fn(*a, ctypes.byref(ctypes.c_size_t(0)))


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(T=1 << 31), dict(H=0), dict(H=(1 << 20) + 1), dict(dtype=3), dict(dtype=-1),
    dict(param_dtype=B.MM_MOE_DT_F16), dict(eps=-1.0), dict(eps=float("nan"))])
def test_norm_shapes(lib, bad):
    a = dict(T=4, H=8, dtype=B.MM_MOE_DT_BF16, param_dtype=B.MM_MOE_DT_BF16, eps=1e-5)
    ok = B.NormShape(*a.values())
    assert size(lib.mm_moe_norm_workspace_size, ctypes.byref(ok)) == 0
    s = B.NormShape(*{**a, **bad}.values())
    assert size(lib.mm_moe_norm_workspace_size, ctypes.byref(s)) == EI
    assert lib.mm_moe_norm_forward(ctypes.byref(s), P[0], 8, P[1], P[2], P[3], 8, P[4], P[5],
                                   None) == EI


def test_norm_pointers(lib):
    s = ctypes.byref(B.NormShape(4, 8, 0, 0, 1e-5))
    assert lib.mm_moe_norm_workspace_size(s, None) == EI
    fwd = [P[0], 8, P[1], P[2], P[3], 8, P[4], P[5], None]
    for i, v in ((0, None), (0, P[0] + 1), (1, 7), (2, None), (2, P[1] + 1), (3, P[2] + 1),
                 (4, None), (5, 4), (6, None), (7, P[5] + 2)):
        a = list(fwd)
        a[i] = v
        assert lib.mm_moe_norm_forward(s, *a) == EI, (i, v)
    bwd = [P[0], 8, P[1], 8, P[2], P[3], P[4], P[5], 8, P[6], 8, P[7], P[8], P[9], None]
    for i, v in ((0, None), (1, 7), (2, None), (3, 0), (4, None), (5, None), (6, P[4] + 2),
                 (7, P[5] + 1), (8, 7), (9, None), (10, 2), (11, None), (12, P[8] + 1),
                 (13, None), (13, P[9] + 8)):
        a = list(bwd)
        a[i] = v
        assert lib.mm_moe_norm_backward(s, *a) == EI, (i, v)


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(T=(1 << 31) - 65536), dict(E=0), dict(E=1025), dict(k=0), dict(k=9),
    dict(G=0), dict(G=(1 << 24) + 1), dict(dtype=3)])
def test_balance_shapes(lib, bad):
    a = dict(T=16, E=8, k=2, G=1, dtype=B.MM_MOE_DT_F32)
    assert size(lib.mm_moe_balance_workspace_size, ctypes.byref(B.BalanceShape(*a.values()))) == 0
    s = B.BalanceShape(*{**a, **bad}.values())
    assert size(lib.mm_moe_balance_workspace_size, ctypes.byref(s)) == EI
    assert lib.mm_moe_balance_forward(ctypes.byref(s), *P[:10], None) == EI


def test_balance_pointers(lib):
    s = ctypes.byref(B.BalanceShape(16, 8, 2, 3, B.MM_MOE_DT_F32))
    fwd = P[:10] + [None]
    for i, v in ((0, None), (0, P[0] + 2), (1, None), (2, None), (2, P[2] + 1), (4, None),
                 (5, None), (6, P[6] + 2), (7, None), (8, None), (9, None), (9, P[9] + 4)):
        a = list(fwd)
        a[i] = v
        assert lib.mm_moe_balance_forward(s, *a) == EI, (i, v)
    bwd = P[:8] + [None]
    for i, v in ((0, None), (1, None), (3, None), (4, None), (5, None), (6, None), (6, P[6] + 2),
                 (7, None)):
        a = list(bwd)
        a[i] = v
        assert lib.mm_moe_balance_backward(s, *a) == EI, (i, v)


def test_grad_arguments(lib):
    def call(entries, n=None, max_norm=1.0, eps=1e-6, norm=P[10], ws=P[11], clip=True):
        flat = B.grad_array(entries)
        n = len(entries) if n is None else n
        p = flat.buffer_info()[0] if entries else None
        if clip:
            return lib.mm_moe_grad_clip(p, n, max_norm, eps, norm, ws, None)
        return lib.mm_moe_grad_norm(p, n, norm, ws, None)

    good = (P[0], P[1], 10, 0, 0)
    for e in ((None or 0, P[1], 10, 0, 0),          # no gradient
              (P[0], 0, 10, 0, 0),                  # no output
              (P[0] + 1, P[1], 10, 0, 0),           # not on an element
              (P[0], P[1] + 2, 10, 0, 2),
              (P[0], P[1], 10, 3, 3), (P[0], P[1], 10, 0, 1), (P[0], P[1], 10, 2, 0),
              (P[0], P[0], 10, 0, 2),               # in place into a wider type
              (P[0], P[1], (1 << 43) + 1, 0, 0),
              (P[0], P[1], (1 << 64) - 1, 0, 0)):   # -1 elements
        assert call([good, e]) == EI, e
    assert call([(P[0], 0, 1 << 43, 0, 0), good], clip=False) == EI      # too many together
    assert call([good], n=-1) == EI and call([good], n=B.MM_MOE_MAX_GRADS + 1) == EI
    assert call([], n=1) == EI
    assert call([good], max_norm=-1.0) == EI and call([good], max_norm=float("nan")) == EI
    assert call([good], eps=-1.0) == EI
    assert call([good], norm=None) == EI and call([good], ws=None) == EI
    assert call([good], ws=P[11] + 8, clip=False) == EI
    n = ctypes.c_size_t(0)
    assert lib.mm_moe_grad_workspace_size(-1, ctypes.byref(n)) == EI
    assert lib.mm_moe_grad_workspace_size(0, ctypes.byref(n)) == 0 and n.value > 0


def test_router_aux_arguments(lib):
    s = ctypes.byref(B.make_shape(64, 128, 64, 16, 4))
    a = P[:9] + [None]
    for i, v in ((0, None), (4, None), (5, P[5] + 2), (6, P[6] + 4), (7, None), (8, None)):
        b = list(a)
        b[i] = v
        assert lib.mm_moe_router_backward_aux(s, *b) == EI, (i, v)


# ------------------------------------------------------------ the handles, on the CPU
def test_norm_handle_checks(lib):
    n = train.MoELayerNorm(4, 8, "bf16", "fp32", device="cpu")
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.ones(8)
    for args, exc in (((None, w, w), TypeError), ((x[:3], w, w), ValueError),
                      ((x.float(), w, w), ValueError), ((x.t().contiguous().t(), w, w), ValueError),
                      ((x[:1].expand(4, 8), w, w), ValueError),
                      ((x, w.bfloat16(), w), ValueError), ((x, w[:7], w), ValueError),
                      ((x, w, None), TypeError)):
        with pytest.raises(exc):
            n.forward(*args)
    with pytest.raises(ValueError):
        n.backward(x, x, w, dx_add=x.float())
    with pytest.raises(ValueError):
        n.backward(x, x, w, out=(x, w, w[:3]))
    with pytest.raises(ValueError):
        train.MoELayerNorm(4, 8, "fp8", device="cpu")
    with pytest.raises(B.MoEError):
        train.MoELayerNorm(0, 8, device="cpu")
    with pytest.raises(ValueError):
        train.MoELayerNorm(4, 8, "fp32", bias=False, device="cpu").forward(x.float(), w, w)


def test_balance_handle_checks(lib):
    b = train.MoEBalanceLoss(16, 8, 2, 3, device="cpu")
    lg, idx = torch.zeros(16, 8), torch.zeros(16, 2, dtype=torch.int32)
    off, mask = torch.zeros(4, dtype=torch.int32), torch.ones(16, dtype=torch.bool)
    for args in ((lg.half(), idx, off, mask), (lg[:15], idx, off, mask),
                 (lg, idx.long(), off, mask), (lg, idx, off[:3], mask), (lg, idx, None, mask),
                 (lg, idx, off.long(), mask), (lg, idx, off, mask.float()),
                 (lg, idx, off, mask[:3])):
        with pytest.raises(ValueError):
            b.forward(*args)
    with pytest.raises(ValueError):
        b.backward(lg, torch.zeros(1), off, mask)
    with pytest.raises(B.MoEError):
        train.MoEBalanceLoss(16, 8, 9, device="cpu")


def test_clip_handle_checks(lib):
    c = train.MoEGradClip(2, device="cpu")
    g = torch.ones(4, 6)
    with pytest.raises(ValueError):
        c.clip([g, g, g], 1.0)
    for bad in (g.double(), g.t(), g[:, :3]):
        with pytest.raises(ValueError):
            c.norm([bad])
    for out in ([g], [g, g.half()], [g, torch.ones(24)], [g, g.t()]):
        with pytest.raises(ValueError):
            c.clip([g, g], 1.0, out=out)
    with pytest.raises(ValueError):
        c.clip([g], -1.0)
    with pytest.raises(ValueError):
        c.clip([g], float("nan"))
