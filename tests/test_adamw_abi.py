"""Refusals of the AdamW step, before anything touches a device (no GPU needed): the C ABI's
status and the handle's checks; and the oracle's 8-bit formats."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import oracle.adamw as oa
from mixture_experts_layer_16_gb300 import binding as B
from mixture_experts_layer_16_gb300 import MoEAdamW, build

EI = B.MM_MOE_EINVAL
P = [4096 * (i + 1) for i in range(16)]     # aligned addresses that are never read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


GOOD = dict(param=P[0], master=P[1], grad=P[2], numel=10, dtype=0, grad_dtype=0, weight_decay=0.1)


def call(lib, tensors=(GOOD,), n=None, opt=(), m=P[3], ms=None, v=P[4], vs=None, counter=P[5],
         lr=1e-3, lr_dev=None, norm=None):
    o = B.AdamW(*{**dict(beta1=0.9, beta2=0.99, eps=1e-8, max_norm=1.0, clip_eps=1e-6, states=0,
                         seed=0), **dict(opt)}.values())
    arr = (B.AdamWTensor * max(1, len(tensors)))(*[B.AdamWTensor(**t) for t in tensors])
    return lib.mm_moe_adamw_step(ctypes.byref(o), ctypes.addressof(arr),
                                 len(tensors) if n is None else n, m, ms, v, vs, counter, lr,
                                 lr_dev, norm, None)


def test_layout():
    """The handle packs six 64-bit words a tensor."""
    assert ctypes.sizeof(B.AdamWTensor) == 48 and ctypes.sizeof(B.AdamW) == 40
    t = B.AdamWTensor(1, 2, 3, 4, 1, 2, 0.25, 0)
    want = struct.pack("<3Q", 1, 2, 3) + struct.pack("<qQ", 4, 1 | 2 << 32) + struct.pack("<fi", .25, 0)
    assert bytes(t) == want


@pytest.mark.parametrize("bad", [
    dict(beta1=-0.1), dict(beta1=1.0), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0),
    dict(eps=1e-60), dict(eps=1e-39), dict(eps=-1e-8), dict(eps=float("inf")), dict(max_norm=-1.0),
    dict(max_norm=float("nan")), dict(clip_eps=-1.0), dict(states=2), dict(states=-1)])
def test_options(lib, bad):
    assert call(lib, opt=bad.items()) == EI


@pytest.mark.parametrize("bad", [
    dict(param=0), dict(param=P[0] + 1), dict(grad=0), dict(grad=P[2] + 1), dict(master=P[1] + 2),
    dict(numel=-1), dict(numel=(1 << 41) + 1), dict(dtype=3), dict(dtype=-1), dict(grad_dtype=1),
    dict(dtype=2, grad_dtype=2), dict(dtype=2, grad_dtype=0, master=0),
    dict(weight_decay=float("nan")), dict(weight_decay=float("inf"))])
def test_tensors(lib, bad):
    assert call(lib, (GOOD, {**GOOD, **bad})) == EI


def test_buffers(lib):
    for bad in (dict(m=None), dict(m=P[3] + 16), dict(v=None), dict(v=P[4] + 4),
                dict(counter=None), dict(counter=P[5] + 8), dict(norm=P[6] + 2),
                dict(lr_dev=P[6] + 1), dict(lr=float("nan")), dict(lr=float("inf")),
                dict(n=-1), dict(n=B.MM_MOE_MAX_GRADS + 1)):
        assert call(lib, **bad) == EI, bad
    assert call(lib, opt=(("states", 1),), vs=P[7]) == EI          # no scales
    assert call(lib, opt=(("states", 1),), ms=P[7]) == EI
    assert call(lib, ({**GOOD, "numel": 1 << 41}, GOOD)) == EI      # too many together
    mom = [P[0], P[1], P[2], P[3], 64, P[4], P[5], None]
    for i, v in ((0, None), (0, P[0] + 8), (1, None), (2, None), (3, None), (4, 63), (4, -32),
                 (5, None), (6, P[5] + 2)):
        a = list(mom)
        a[i] = v
        assert lib.mm_moe_adamw_moments(*a) == EI, (i, v)
    assert lib.mm_moe_adamw_moments(None, None, None, None, 0, None, None, None) == 0


def test_handle(lib):
    p = [torch.zeros(4, 6, dtype=torch.bfloat16), torch.zeros(5)]
    g = [torch.zeros(4, 6, dtype=torch.bfloat16), torch.zeros(5)]
    o = MoEAdamW(p, weight_decay=(0.1, 0.0), device="cpu")
    assert o.first == [0, 32] and o.m.numel() == 64 and o.steps() == 0
    o.set_step(3)
    assert o.steps() == 3
    words = [int(w) for w in o.counter]
    assert struct.unpack("<2d", struct.pack("<2q", *words[1:3])) == (0.9 ** 3, 0.999 ** 3)
    w = [p[0].float(), None]
    for kw, exc in ((dict(params=p[:1]), ValueError), (dict(grads=g[:1]), ValueError),
                    (dict(masters=w[:1]), ValueError), (dict(params=[p[0], None]), TypeError),
                    (dict(params=[p[0], p[1].half()]), ValueError),
                    (dict(params=[p[0].t().contiguous().t(), p[1]]), ValueError),
                    (dict(params=[p[0].reshape(6, 4), p[1]]), ValueError),
                    (dict(grads=[g[0].half(), g[1]]), ValueError),
                    (dict(grads=[g[0], g[1].bfloat16()]), ValueError),
                    (dict(grads=[g[0], None]), TypeError),
                    (dict(grads=[g[0][:, :5], g[1]]), ValueError),
                    (dict(masters=[p[0], None]), ValueError),
                    (dict(masters=[None, p[1].clone()]), ValueError),
                    (dict(masters=["x", None]), TypeError),
                    (dict(norm=1.0), TypeError), (dict(norm=torch.zeros(2)), ValueError),
                    (dict(norm=torch.zeros((), dtype=torch.float64)), ValueError),
                    (dict(max_norm=1.0), ValueError),
                    (dict(norm=torch.zeros(()), max_norm=-1.0), ValueError),
                    (dict(lr=torch.zeros(2)), ValueError)):
        with pytest.raises(exc):
            o.step(**{**dict(params=p, grads=g, lr=1e-3, masters=w), **kw})
    two = MoEAdamW([p[1], p[1]], device="cpu")
    with pytest.raises(ValueError):                   # the same tensor twice
        two.step([p[1], p[1]], [g[1], g[1]], 1e-3)
    for kw in (dict(states="int8"), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=0.0), dict(eps=1e-39),
               dict(weight_decay=[0.1])):
        with pytest.raises(ValueError):
            MoEAdamW(p, device="cpu", **kw)
    with pytest.raises(ValueError):
        MoEAdamW([torch.zeros(3, dtype=torch.float64)], device="cpu")
    with pytest.raises(TypeError):
        MoEAdamW([3], device="cpu")
    with pytest.raises(ValueError):
        o.set_step(-1)


@pytest.mark.parametrize("kind,codes", [(oa.M8, 127), (oa.V8, 256)])
def test_oracle_formats(kind, codes):
    """Every code's value is on the grid, in order; what lies on the grid stays there under
    any random bits; the largest value of a block fits its scale and not half of it."""
    n = -(-codes // 32) * 32
    c = np.minimum(np.arange(n), codes - 1)
    val = oa.decode(c, np.full(n // 32, 127), kind)[:codes]
    assert np.array_equal(val, oa.grid(kind))
    for r in (0, 65535):
        assert np.array_equal(oa.held(val, 0, kind, np.full(codes, r)), val)
    for a in (1e-30, 0.3, kind[0], np.nextafter(kind[0], np.inf), 2 * kind[0], 1e25):
        e = oa.scale_exponent(a, kind)
        assert a <= kind[0] * 2.0 ** e and a > kind[0] * 2.0 ** (e - 1)


def test_random_bits_are_even():
    """Means and shares of 2^20 elements' bits, within six standard deviations."""
    m, v = oa.random16(3, 17, 2, np.arange(1 << 20))
    for x in (m, v):
        assert abs(x.mean() / 65535 - 0.5) < 6 * 0.2887 / 1024
        share = np.bincount(x >> 12, minlength=16) / len(x)
        assert np.abs(share - 1 / 16).max() < 6 * np.sqrt(1 / 16 * 15 / 16) / 1024
    assert abs(np.corrcoef(m, v)[0, 1]) < 6 / 1024
    assert abs(np.corrcoef(m[1:], m[:-1])[0, 1]) < 6 / 1024
    n = oa.random16(3, 18, 2, np.arange(1 << 20))[0]
    assert abs(np.corrcoef(m, n)[0, 1]) < 6 / 1024


def test_overlap(lib):
    """What is written lies apart from all the rest, in part too; two gradients may be the same."""
    a, b = dict(GOOD), dict(GOOD, param=P[6], master=P[7], grad=P[8])
    for bad in (dict(param=P[0]), dict(param=P[0] + 18), dict(param=P[1] + 38), dict(master=P[1] - 36),
                dict(master=P[0] + 16), dict(grad=P[0] + 18), dict(grad=P[1] - 18),
                dict(param=P[2] + 18), dict(master=P[8] + 16), dict(param=P[7] - 18)):
        assert call(lib, (a, {**b, **bad})) == EI, bad
        many = [dict(GOOD, numel=0)] * 40                 # (more than a short list)
        assert call(lib, (a, *many, {**b, **bad})) == EI, bad
    assert call(lib, lr=1e300) == EI
