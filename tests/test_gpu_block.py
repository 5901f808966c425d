"""MoEBlock against the composed fp64 oracles, the router's backward with auxiliary logit
gradients, and the example's training steps.

The layer's outputs and gradients hold to 1e-2 of their maximum (its own bound); what adds
two such terms (dn, then dx) to 2e-2.  The block's inner tensors that the GPU rounds to bf16
(n) or decides on (topk_idx) are taken from it, the routing having its own tests."""
import numpy as np
import pytest
import torch

import oracle
import oracle.router as orr
import oracle.train as ot
from examples import train_block
from mixture_experts_layer_16_gb300 import MoEBlock, MoERouter
from mixture_experts_layer_16_gb300.inputs import custom_inputs, router_weights
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def rel(a, b):
    return G.rel_err(G.f32(a), b)


@pytest.mark.parametrize("T,H,I,E,k,recompute", [(384, 256, 128, 16, 4, False),
                                                 (300, 128, 64, 8, 2, True)])
def test_block_against_the_oracles(T, H, I, E, k, recompute):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)
    p = MoEBlock.init_params(H, I, E, seed=3, std=0.08)
    p["norm_weight"] = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).bfloat16()
    p["norm_bias"] = (0.2 * torch.randn(H, generator=gen, device="cuda")).bfloat16()
    x = (2 * torch.randn((T, H), generator=gen, device="cuda") + 0.5).bfloat16()
    dout = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32, device="cuda")
    mask = torch.rand(T, generator=gen, device="cuda") < 0.9
    dl = torch.tensor([3.0, 0.5], device="cuda")
    blk = MoEBlock(T, H, I, E, k, sequences=3, recompute=recompute)
    out, losses, counts = blk.forward(x, p, off, mask)
    dx, g = blk.backward(dout, p, dl)
    torch.cuda.synchronize()

    x64, do = G.f32(x), G.f32(dout)
    w = {n: G.f32(t) for n, t in p.items()}
    _, n, idx, tw, _, _ = blk._kept
    nf = ot.norm_forward(x64, w["norm_weight"], w["norm_bias"], 1e-5)
    assert rel(n, nf["y"]) <= 2.0 ** -8
    n64, idx = G.f32(n), idx.cpu().numpy()
    lg = orr.logits(n64, w["W_router"])
    tw64 = orr.topk_softmax(np.take_along_axis(lg, idx.astype(np.int64), axis=1))
    assert rel(tw, tw64) <= 1e-5
    f = oracle.forward(n64, idx, tw64, w["W_gate"], w["W_up"], w["W_down"])
    assert rel(out, x64 + f["y"]) <= 1e-2
    offn, m = off.cpu().numpy(), mask.cpu().numpy()
    bf = ot.balance_forward(lg, idx, 3, offn, m)
    assert np.array_equal(counts.cpu().numpy(), bf["counts"])
    assert np.allclose(G.f32(losses), bf["losses"], rtol=1e-4)
    b = oracle.backward(do, n64, idx, tw64, w["W_gate"], w["W_up"], w["W_down"], fwd=f)
    rb = orr.backward(n64, w["W_router"], idx, tw64, b["dtopk_w"])
    ds = rb["dlogits"] + ot.balance_backward(lg, idx, [3.0, 0.5], 3, offn, m)
    dn = b["dx"] + ds @ w["W_router"]
    nb = ot.norm_backward(dn, x64, w["norm_weight"], 1e-5, do)
    assert rel(g["W_router"], ds.T @ n64) <= 1e-2
    for name in ("W_gate", "W_up", "W_down"):
        assert rel(g[name], b["d" + name]) <= 1e-2
    assert rel(dx, nb["dx"]) <= 2e-2
    assert rel(g["norm_weight"], nb["dweight"]) <= 2e-2
    assert rel(g["norm_bias"], nb["dbias"]) <= 2e-2


def test_router_backward_aux():
    """An auxiliary logit gradient of zeros changes no bit; a real one is the oracle's sum."""
    T, H, E, k = 500, 256, 32, 4
    d = custom_inputs(T, H, 64, 8, 2, seed=12)
    rw = router_weights(E, H, seed=12)
    gk = np.random.default_rng(1).standard_normal((T, k)).astype(np.float32)
    r = MoERouter(T, H, E, k)
    x, Wr = G.bf16_dev(d["x_bits"]), G.bf16_dev(rw["W_router_bits"])
    idx, w = r.forward(x, Wr)
    g = torch.from_numpy(gk).cuda()

    def back(aux):
        dx = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
        dW = r.backward(x, Wr, idx, w, g, dx, dlogits_aux=aux)
        return dx, dW, r.dlogits.clone()
    plain = back(None)
    zero = back(torch.zeros((T, E), device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(plain, zero))
    aux = torch.randn((T, E), device="cuda")
    dx, dW, dlog = back(aux)
    ro = orr.forward(d["x"], rw["W_router"], k)
    assert np.array_equal(ro["topk_idx"], idx.cpu().numpy())
    ds = orr.backward(d["x"], rw["W_router"], ro["topk_idx"], ro["topk_w"], gk)["dlogits"] + \
        G.f32(aux)
    assert rel(dlog, ds) <= 2.0 ** -8
    assert rel(dW, ds.T @ d["x"]) <= 1e-2
    assert rel(dx, ds @ rw["W_router"]) <= 1e-2
    with pytest.raises(ValueError):
        back(aux.bfloat16())


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_example_trains(prec):
    h = train_block.train(T=1024, H=256, I=128, E=8, k=2, prec=prec, steps=12, sequences=4,
                          log=lambda *_: None)
    mse = [s[0] for s in h]
    assert all(np.isfinite(v) for s in h for v in s)
    assert mse[-1] < 0.9 * mse[0] and all(b <= a * 1.05 for a, b in zip(mse, mse[1:]))
    assert all(s[1] >= 0.9 for s in h)


def test_block_needs_a_forward():
    b = MoEBlock(64, 128, 64, 8, 2)
    with pytest.raises(RuntimeError):
        b.backward(torch.zeros((64, 128), dtype=torch.bfloat16, device="cuda"),
                   MoEBlock.init_params(128, 64, 8), torch.zeros(2, device="cuda"))
