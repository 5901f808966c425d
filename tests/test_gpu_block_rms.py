"""Two MoEBlocks between RMS norms, with a router of sigmoid scores in groups: against the composed
fp64 oracles, and a step of them with the gradient norm and AdamW.

As for the block with a layer norm: the layer's outputs and gradients hold to 1e-2 of their maximum,
what adds such terms to 2e-2 and through a second block to 4e-2; tensors that the GPU rounds to bf16
or decides on are taken from it."""
import numpy as np
import pytest
import torch

import oracle
import oracle.adamw as oa
import oracle.resnorm as orn
import oracle.router as orr
import oracle.selection as osel
import oracle.train as ot
from examples import train_block
from mixture_experts_layer_16_gb300 import MoEAdamW, MoEBlock, MoEGradClip
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
SELECT = dict(score="sigmoid", groups=4, topk_groups=2, group_score="top2", scale=1.5)


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def rel(a, b):
    return G.rel_err(G.f32(a), b)


def build(T, H, I, E, k, post, gate):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    a = MoEBlock(T, H, I, E, k, sequences=2, select=SELECT, norm="rms", post_norm=post, gate=gate,
                 next_norm=True, scale=0.5)
    b = MoEBlock(T, H, I, E, k, sequences=2, select=SELECT, norm="rms", post_norm=post, gate=gate,
                 first=False, scale=0.5)
    params = [MoEBlock.init_params(H, I, E, seed=3 + i, std=0.08, rms=True) for i in range(2)]
    for p, gone in zip(params, ((), ("norm_weight", "next_weight"))):
        for n in (*gone, *(() if post else ("post_weight",)), *(() if gate else ("gate",))):
            del p[n]
        for n in ("norm_weight", "post_weight", "gate", "next_weight"):
            if n in p:
                p[n] = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).bfloat16()
    x = (2 * torch.randn((T, H), generator=gen, device="cuda")).bfloat16()
    dout = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    off = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    mask = torch.rand(T, generator=gen, device="cuda") < 0.9
    bias = 0.05 * torch.randn(E, generator=gen, device="cuda")
    return a, b, params, x, dout, off, mask, bias


def inner(blk, w, n, off, mask, bias, k, lg):
    """The block's layer and losses from the GPU's n and logits: what the oracle says of them."""
    kept = blk._kept
    idx = kept[2].cpu().numpy()
    ri, tw = osel.forward(lg, G.f32(bias), k, **SELECT)
    assert np.array_equal(idx, ri)
    assert rel(kept[3], tw) <= 1e-5
    f = oracle.forward(n, idx, tw, w["W_gate"], w["W_up"], w["W_down"])
    return idx, tw, f


@pytest.mark.parametrize("T,H,I,E,k,post,gate", [(384, 256, 128, 16, 4, True, True),
                                                 (300, 128, 64, 8, 2, False, False),
                                                 (257, 128, 64, 16, 3, True, False)])
def test_two_blocks(T, H, I, E, k, post, gate):
    a, b, params, x, dout, off, mask, bias = build(T, H, I, E, k, post, gate)
    dl = torch.tensor([3.0, 0.5], device="cuda")
    h, _, _, n2 = a.forward(x, params[0], off, mask, bias=bias)
    out, losses, counts = b.forward(h, params[1], off, mask, bias=bias, n=n2)
    dh, g1, dn2 = b.backward(dout, params[1], dl)
    dx, g0 = a.backward(dh, params[0], dl, dnext=dn2)
    torch.cuda.synchronize()
    offn, m = off.cpu().numpy(), mask.cpu().numpy()
    w = [{n: G.f32(t) for n, t in p.items()} for p in params]
    x64, h64, n264 = G.f32(x), G.f32(h), G.f32(n2)
    eps = 1e-6

    def join(i, res, f, w_pre):
        return orn.forward(res, f, w[i].get("post_weight"), w[i].get("gate"), w_pre,
                           "channel" if gate else None, 0.5, eps)

    # forward, block by block
    r1 = orn.forward(x64, None, None, None, w[0]["norm_weight"], None, 1.0, eps)
    n1 = G.f32(a._kept[1])
    assert rel(a._kept[1], r1["n"]) <= 2.0 ** -8
    lg1, lg2 = G.f32(a.router.logits), G.f32(b.router.logits)
    for lg, n, i in ((lg1, n1, 0), (lg2, n264, 1)):
        assert G.rel_err(lg, orr.logits(n, w[i]["W_router"])) <= 1e-4
    i1, t1, f1 = inner(a, w[0], n1, off, mask, bias, k, lg1)
    j1 = join(0, x64, f1["y"], w[0]["next_weight"])
    assert rel(h, j1["out"]) <= 1e-2 and rel(n2, j1["n"]) <= 2e-2
    i2, t2, f2 = inner(b, w[1], n264, off, mask, bias, k, lg2)
    j2 = join(1, h64, f2["y"], None)
    assert rel(out, j2["out"]) <= 1e-2
    bf = ot.balance_forward(lg2, i2, 2, offn, m)
    assert np.array_equal(counts.cpu().numpy(), bf["counts"])
    assert np.allclose(G.f32(losses), bf["losses"], rtol=1e-4)

    # backward, the second block first
    def back(i, do, dnext, out64, f, n, idx, tw, lg, rstd_out):
        fg = G.f32((a, b)[i]._kept[6])                 # (the layer's output as it was stored)
        rf = (fg ** 2).mean(axis=1)
        g = orn.backward(do, dnext, out64, fg, w[i].get("post_weight"), w[i].get("gate"),
                         w[i].get("next_weight"), "channel" if gate else None, 0.5,
                         (rf + eps) ** -0.5, rstd_out)
        lb = oracle.backward(g["df"], n, idx, tw, w[i]["W_gate"], w[i]["W_up"], w[i]["W_down"], fwd=f)
        ds = osel.backward(lg, idx, lb["dtopk_w"], "sigmoid", True, 1.5) + \
            ot.balance_backward(lg, idx, [3.0, 0.5], 2, offn, m)
        return g, lb, ds.T @ n, lb["dx"] + ds @ w[i]["W_router"]
    g, lb, dWr, dn = back(1, G.f32(dout), None, None, f2, n264, i2, t2, lg2, None)
    assert rel(dh, g["dx"]) <= 1e-2 and rel(dn2, dn) <= 2e-2
    assert rel(g1["W_router"], dWr) <= 2e-2
    for n in ("W_gate", "W_up", "W_down"):
        assert rel(g1[n], lb["d" + n]) <= 1e-2, n
    for n in ("post_weight", "gate"):
        assert (n in g1) == (n in w[1])
        if n in g1:
            assert rel(g1[n], g[n]) <= 1e-2, n
    g, lb, dWr, dn = back(0, G.f32(dh), G.f32(dn2), h64, f1, n1, i1, t1, lg1,
                          G.f32(a.join.rstd_out))
    for n in ("post_weight", "gate", "pre_weight"):
        name = "next_weight" if n == "pre_weight" else n
        if name in g0:
            assert rel(g0[name], g[n]) <= 1e-2, n
    for n in ("W_gate", "W_up", "W_down"):
        assert rel(g0[n], lb["d" + n]) <= 1e-2, n
    assert rel(g0["W_router"], dWr) <= 2e-2
    first = orn.backward(g["dx"], dn, x64, None, None, None, w[0]["norm_weight"], None, 1.0, None,
                         r1["rstd_out"])
    assert rel(dx, first["dx"]) <= 2e-2
    assert rel(g0["norm_weight"], first["pre_weight"]) <= 2e-2
    assert set(g0) == set(params[0]) and set(g1) == set(params[1])


@pytest.mark.parametrize("states", ["fp32", "8bit"])
def test_a_step_of_both(states):
    """Forward, backward, gradient norm and AdamW over both blocks' parameters: the masters move as
    the oracle's step from the same gradients says, and the next forward reads their roundings."""
    T, H, I, E, k = 256, 128, 64, 16, 4
    a, b, params, x, dout, off, mask, bias = build(T, H, I, E, k, True, True)
    dl = torch.tensor([0.1, 0.01], device="cuda")
    flat = [p[n] for p in params for n in p]
    masters = [t.float() for t in flat]
    opt = MoEAdamW(flat, (0.9, 0.99), weight_decay=0.1, states=states, seed=1)
    clip = MoEGradClip(len(flat))
    for t in (1, 2):
        h, _, _, n2 = a.forward(x, params[0], off, mask, bias=bias)
        out, _, _ = b.forward(h, params[1], off, mask, bias=bias, n=n2)
        dh, g1, dn2 = b.backward(dout, params[1], dl)
        _, g0 = a.backward(dh, params[0], dl, dnext=dn2)
        grads = [g[n] for g, p in zip((g0, g1), params) for n in p]
        norm = clip.norm(grads)
        before = [G.f32(m) for m in masters]
        m0, v0 = (G.f32(s) for s in opt.moments())
        opt.step(flat, grads, 1e-3, masters, norm, 0.5)
        torch.cuda.synchronize()
        n64 = ot.grad_norm([G.f32(g) for g in grads])
        assert abs(float(norm) / n64 - 1) < 1e-6 and float(norm) > 0.5
        coef = 0.5 / (n64 + 1e-6)
        for i, (m, p) in enumerate(zip(masters, flat)):
            s = slice(opt.first[i], opt.first[i] + p.numel())
            want, _, _ = oa.step(before[i].ravel(), G.f32(grads[i]).ravel(), m0[s], v0[s], t, 1e-3, 0.1,
                                 (0.9, 0.99), 1e-8, coef)
            # a step of at most 1e-3 sqrt(1 / 0.1) or so, right to 1e-5 of it; fp32 masters of size 1
            assert np.abs(G.f32(m).ravel() - want).max() <= 4e-8 + 2.0 ** -24 * np.abs(want).max()
            assert torch.equal(p, m.to(torch.bfloat16))
    assert opt.steps() == 2


@pytest.mark.parametrize("states", ["fp32", "8bit"])
def test_example(states):
    """It runs, and what it reports is finite."""
    h = train_block.train_rms(T=512, H=128, I=64, E=16, k=2, steps=3, states=states,
                              log=lambda *a: None)
    assert len(h) == 3 and np.isfinite(h).all()


def test_refusals():
    a, b, params, x, dout, off, mask, bias = build(257, 128, 64, 8, 2, True, False)
    n = torch.zeros_like(x)
    with pytest.raises(ValueError):
        a.forward(x, params[0], off, mask, n=n)
    with pytest.raises(ValueError):
        b.forward(x, params[1], off, mask)
    with pytest.raises(RuntimeError):
        b.backward(dout, params[1], torch.zeros(2, device="cuda"))
    for kw in (dict(gate=True), dict(next_norm=True), dict(first=False), dict(scale=0.5)):
        with pytest.raises(ValueError):
            MoEBlock(64, 128, 64, 8, 2, **kw)
    with pytest.raises(ValueError):
        MoEBlock(64, 128, 64, 8, 2, norm="batch")
