"""The choice of experts, the residual norm and AdamW beside other work: memory that they took from the
current stream's pool on another stream, and calls of several host threads."""
import threading

import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEAdamW, MoEResidualNorm, MoERouter, MoESelect
from tests import gpu_util as G
from tests.test_gpu_train_streams import check

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def test_select_on_another_stream():
    T, E, k = 4096, 128, 4
    l, b = torch.randn((T, E), device="cuda"), torch.zeros(E, device="cuda")
    h = MoESelect(T, E, k, "sigmoid")
    idx, _ = h.forward(l, b)
    g = torch.randn((T, k), device="cuda")
    check(lambda s: list(h.forward(l, b, stream=s)))
    check(lambda s: [h.backward(l, idx, g, stream=s)])


def test_router_on_another_stream():
    T, H, E, k = 4096, 256, 128, 4
    x, W = torch.randn((T, H), device="cuda").to(BF), torch.randn((E, H), device="cuda").to(BF)
    g, dx = torch.randn((T, k), device="cuda"), torch.randn((T, H), device="cuda").to(BF)

    def fwd(s):
        r = MoERouter(T, H, E, k, select=dict(score="sigmoid"))
        return [*r.forward(x, W, stream=s), r.logits]
    check(fwd)
    kept = MoERouter(T, H, E, k, select=dict(score="sigmoid"))
    idx, w = kept.forward(x, W)

    def bwd(s):
        return [kept.backward(x, W, idx, w, g, dx, stream=s)]
    check(bwd)


def test_residual_norm_on_another_stream():
    T, H = 4096, 2048
    x, f, dout, dn = (torch.randn((T, H), device="cuda").to(BF) for _ in range(4))
    p = dict(post_weight=torch.randn(H, device="cuda").to(BF), gate=torch.randn(H, device="cuda").to(BF),
             pre_weight=torch.randn(H, device="cuda").to(BF))

    def fwd(s):
        h = MoEResidualNorm(T, H, gate="channel")
        return [*h.forward(x, f, stream=s, **p), h.rstd_f, h.rstd_out]

    def bwd(s):
        h = MoEResidualNorm(T, H, gate="channel")
        out, n = h.forward(x, f, stream=s, **p)
        dx, df, grads = h.backward(dout, dn, out, f, stream=s, **p)
        return [out, n, dx, df, *grads.values(), h.rstd_f, h.rstd_out, h.workspace]
    check(fwd)
    check(bwd)


@pytest.mark.parametrize("states", ["fp32", "8bit"])
def test_adamw_on_another_stream(states):
    p, g = [torch.randn(1 << 20, device="cuda")], [torch.randn(1 << 20, device="cuda")]

    def step(s):
        o = MoEAdamW(p, states=states)
        o.step(p, g, 1e-3, stream=s)
        return [t for t in (o.m, o.v, o.m_scale, o.v_scale) if t is not None]

    def moments(s):
        o = MoEAdamW(p, states="8bit")
        return list(o.moments(stream=s))
    check(step)
    check(moments)


def test_host_threads():
    """Each with its own handles, buffers and stream, at sizes with different shared-memory limits."""
    def job(i, out):
        s = torch.cuda.Stream()
        gen = torch.Generator(device="cuda")
        gen.manual_seed(i)
        with torch.cuda.stream(s):
            T, H, E = 200 + 300 * i, 256 << (i % 4), 64 << (i % 3)
            x, f, dout, dn = (torch.randn((T, H), generator=gen, device="cuda").to(BF) for _ in range(4))
            w = torch.ones(H, dtype=BF, device="cuda")
            h = MoEResidualNorm(T, H)
            sel = MoESelect(T, E, 4, "sigmoid", 4, 2, "top2")
            l = torch.randn((T, E), generator=gen, device="cuda")
            b = torch.zeros(E, device="cuda")
            opt = MoEAdamW([x], states="8bit")
            first = None
            for _ in range(20):
                o, n = h.forward(x, f, post_weight=w, pre_weight=w)
                dx, df, g = h.backward(dout, dn, o, f, post_weight=w, pre_weight=w)
                idx, tw = sel.forward(l, b)
                res = [o, n, dx, df, g["post_weight"], g["pre_weight"], idx, tw]
                opt.step([x.clone()], [dout], 1e-3)
                if first is None:
                    first = res
                s.synchronize()
                if not all(torch.equal(a, c) for a, c in zip(first, res)):
                    out.append((i, "differs"))
                    return
        out.append((i, "ok"))
    out = []
    ts = [threading.Thread(target=job, args=(i, out)) for i in range(6)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert sorted(out) == [(i, "ok") for i in range(6)]


def test_one_graph_of_all():
    """A captured run of the operators as a step makes it, replayed: the same as without a graph."""
    T, H, E, k = 300, 512, 64, 4
    x, f, dout, dn = (torch.randn((T, H), device="cuda").to(BF) for _ in range(4))
    w = torch.ones(H, dtype=BF, device="cuda")
    l, b = torch.randn((T, E), device="cuda"), torch.zeros(E, device="cuda")
    dw = torch.randn((T, k), device="cuda")
    h, sel = MoEResidualNorm(T, H, scale=0.5), MoESelect(T, E, k, "sigmoid", 8, 4, "top2")
    master = [torch.randn(H, device="cuda"), torch.randn(H, device="cuda")]
    params = [m.to(BF) for m in master]
    opt = MoEAdamW(params, states="8bit")

    def go(s=None):
        o, n = h.forward(x, f, post_weight=w, pre_weight=w, stream=s)
        idx, tw = sel.forward(l, b, stream=s)
        dl = sel.backward(l, idx, dw, stream=s)
        dx, df, g = h.backward(dout, dn, o, f, post_weight=w, pre_weight=w, stream=s)
        opt.step(params, [g["post_weight"], g["pre_weight"]], 1e-3, master, stream=s)
        return [o, n, idx, tw, dl, dx, df, *g.values()]
    kept = [t.clone() for t in (*master, *params, opt.m, opt.v, opt.m_scale, opt.v_scale, opt.counter)]
    mine = (*master, *params, opt.m, opt.v, opt.m_scale, opt.v_scale, opt.counter)
    want = [t.clone() for t in (*go(), *go())]
    after = [t.clone() for t in mine]
    for t, v in zip(mine, kept):
        t.copy_(v)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = go(s)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, v) for a, v in zip(got, want))
    assert all(torch.equal(a, v) for a, v in zip(mine, after)) and opt.steps() == 2
