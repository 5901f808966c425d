"""MoEAdamW on the GPU against the fp64 oracle.

Bounds (e = 2^-24, u: half an ulp of the stored type).  g = coef grad takes a division, a sum and a
product: 4 e of |g| (the coefficient's input norm is exact).  m = b1 m + a1 g with betas
rounded to fp32: 3 roundings of each term, so at most 8 e (|b1 m| + |a1 g|); v: g twice and a product
more, 14 e (b2 v + a2 g^2).  The update u = m c1 / (sqrt(v) c2 + eps): the root halves v's error, the
approximate root and division are within 2^-22 = 4 e each, corrections and products one each: with
terms of both signs in m, 8 e (|b1 m| + |a1 g|) c1 / (sqrt(v) c2 + eps) + 24 e |u|.  p takes one
rounding: e |p| + lr (that + 2 e (|u| + decay |p|)), and its own type's half ulp where it is stored.
"""
import math

import numpy as np
import pytest
import torch

import oracle.adamw as oa
from mixture_experts_layer_16_gb300 import MoEAdamW, MoEGradClip
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {n: torch.finfo(t).eps / 2 for n, t in DT.items()}
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
E = 2.0 ** -24
BETAS, EPS = (0.9, 0.99), 1e-8
SIZES = (5000, 1, 0, 7, 31, 32, 33, 2047, 2048, 2049, 40003)


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def f64(t):
    return t.double().cpu().numpy()


def make(sizes, dtype, grad, master, seed=0, odd=False):
    """params, grads, masters; odd: each on an address that no vector begins on."""
    r = np.random.default_rng(seed)

    def dev(a, dt):
        t = torch.from_numpy(a.astype(np.float32)).to("cuda", DT[dt])
        if odd:
            wide = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            wide[1:] = t
            t = wide[1:]
        return t
    w = [0.05 * r.standard_normal(n) for n in sizes]
    g = [np.exp(r.normal(-6, 1.5, n)) * r.choice([-1, 1], n) for n in sizes]
    masters = [dev(a, "fp32") for a in w] if master else None
    return [dev(a, dtype) for a in w], [dev(a, grad) for a in g], masters


def check(name, got, want, bound):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:3],
                           float(np.nanmax(np.abs(got - want) / bound)))


def slices(o):
    return [slice(a, a + n) for a, n in zip(o.first, (s.numel() for s in o.shapes))]


def check_step(o, before, after, grads, t, lr, coef, dtype, m, v):
    """One step of one tensor: before = (p, m, v) in fp64, after = (wide p, param)."""
    p0, m0, v0, decay = before
    g = f64(grads)
    p, m1, v1 = oa.step(p0, g, m0, v0, t, lr, decay, BETAS, EPS, coef)
    g = np.abs(g * coef)
    am = BETAS[0] * np.abs(m0) + (1 - BETAS[0]) * g
    if m is not None:
        check("m", m, m1, 8 * E * am + 1e-44)
        check("v", v, v1, 14 * E * v1 + 1e-44)
    c1, c2 = 1 / (1 - BETAS[0] ** t), 1 / math.sqrt(1 - BETAS[1] ** t)
    den = np.sqrt(v1) * c2 + EPS
    u = np.abs(m1 * c1 / den)
    bound = E * np.abs(p) + lr * (8 * E * am * c1 / den + 26 * E * u + 2 * E * decay * np.abs(p0))
    wide, param = after
    if wide is not None:
        check("master", f64(wide), p, bound + 1e-44)
    check("param", f64(param), p, bound * (1 + U[dtype]) + U[dtype] * np.abs(p) + SUB[dtype] + 1e-44)


@pytest.mark.parametrize("dtype,grad,master", [
    ("bf16", "bf16", True), ("bf16", "fp32", False), ("fp16", "fp16", True), ("fp16", "fp32", True),
    ("fp32", "fp32", False), ("bf16", "bf16", False)])
@pytest.mark.parametrize("odd", [False, True])
def test_fp32_states(dtype, grad, master, odd):
    params, grads, masters = make(SIZES, dtype, grad, master, odd=odd)
    decay = [0.1 * (i % 3) for i in range(len(SIZES))]
    o = MoEAdamW(params, BETAS, EPS, decay)
    for t in range(1, 4):
        lr = 1e-3 * t
        norm = MoEGradClip(16).norm(grads)
        max_norm = 0.5 * float(norm) if t == 2 else 1e9
        coef = min(1.0, max_norm / (float(norm) + 1e-6)) if t == 2 else 1.0
        wide = params if masters is None else masters
        before = [(f64(w), f64(o.m[s]), f64(o.v[s]), d)
                  for w, s, d in zip(wide, slices(o), decay)]
        # (numbers that reach the kernel in fp32)
        coef = float(np.float32(max_norm) / (float(norm) + 1e-6)) if t == 2 else 1.0
        o.step(params, grads, lr, masters, norm if t != 3 else None, max_norm if t != 3 else None)
        lr = float(np.float32(lr))
        for i, s in enumerate(slices(o)):
            check_step(o, before[i], (None if masters is None else masters[i], params[i]),
                       grads[i], t, lr, coef, dtype, f64(o.m[s]), f64(o.v[s]))
    assert o.steps() == 3
    behind = torch.ones(o.m.numel(), dtype=torch.bool, device="cuda")
    for s in slices(o):
        behind[s] = False
    assert not o.m[behind].any() and not o.v[behind].any()


def check_held(got, scales, values, err, kind, rand16):
    """Codes between those of the values less and plus their error, under the same random bits;
    a block's scale is that of its largest value, within its error."""
    values = np.pad(values, (0, -len(values) % 32))
    err = np.pad(err, (0, -len(err) % 32))
    for b in range(len(values) // 32):
        w = slice(32 * b, 32 * b + 32)
        a = np.abs(values[w])
        e = int(scales[b]) - 127
        assert oa.scale_exponent((a - err[w]).clip(0).max(), kind) <= e <= \
            oa.scale_exponent((a + err[w]).max(), kind), b
        lo = oa.held((a - err[w]).clip(0), e, kind, rand16[w])
        hi = oa.held(np.minimum(a + err[w], kind[0] * 2.0 ** e), e, kind, rand16[w])
        mag = np.abs(got[w])
        assert ((lo <= mag) & (mag <= hi)).all(), (b, np.argwhere((lo > mag) | (mag > hi))[:3])
        assert (np.sign(got[w]) * np.sign(values[w]) >= 0).all()


@pytest.mark.parametrize("dtype,grad,master,odd", [
    ("bf16", "bf16", True, False), ("fp16", "fp32", False, True), ("fp32", "fp32", False, False)])
def test_8bit_states(dtype, grad, master, odd):
    sizes = (5000, 1, 0, 33, 64, 2049)
    seed = 11
    params, grads, masters = make(sizes, dtype, grad, master, seed=3, odd=odd)
    o = MoEAdamW(params, BETAS, EPS, 0.05, states="8bit", seed=seed)
    for t in range(1, 4):
        m0 = oa.decode(o.m.cpu().numpy(), o.m_scale.cpu().numpy(), oa.M8)
        v0 = oa.decode(o.v.cpu().numpy(), o.v_scale.cpu().numpy(), oa.V8)
        wide = params if masters is None else masters
        before = [f64(w) for w in wide]
        o.step(params, grads, 1e-3, masters)
        m1, v1 = (f64(x) for x in o.moments())
        assert np.array_equal(m1, oa.decode(o.m.cpu().numpy(), o.m_scale.cpu().numpy(), oa.M8))
        assert np.array_equal(v1, oa.decode(o.v.cpu().numpy(), o.v_scale.cpu().numpy(), oa.V8))
        for i, s in enumerate(slices(o)):
            if sizes[i] == 0:
                continue
            check_step(o, (before[i], m0[s], v0[s], 0.05),
                       (None if masters is None else masters[i], params[i]), grads[i], t,
                       float(np.float32(1e-3)), 1.0, dtype, None, None)
            _, m, v = oa.step(before[i], f64(grads[i]), m0[s], v0[s], t, 1e-3, 0, BETAS, EPS)
            em = 8 * E * (BETAS[0] * np.abs(m0[s]) + (1 - BETAS[0]) * np.abs(f64(grads[i])))
            blocks = slice(s.start, s.start + -(-sizes[i] // 32) * 32)
            q = slice(blocks.start // 32, blocks.stop // 32)
            rm, rv = oa.random16(seed, t, i, np.arange(blocks.stop - blocks.start))
            # (2^-17 of a step: the random bits' own grid, and the product's rounding below it)
            check_held(m1[blocks], o.m_scale[q].cpu().numpy(), m, em, oa.M8, rm)
            check_held(v1[blocks], o.v_scale[q].cpu().numpy(), v, 14 * E * v, oa.V8, rv)
            assert (v1[s][v > 0] > 0).all()


def test_8bit_averages_keep_their_expectation():
    """A constant gradient in one half and alternating ones in the other: the mean over many elements
    of each kept average is the average itself.  The relative error of one element's v after t steps
    has a variance of at most t (f (1 - f) d^2) with a step d <= 1/8 of it and f <= 1: below t / 256;
    a mean over n elements lies within 6 sqrt(t / 256 / n) of its expectation."""
    n, t = 1 << 20, 50
    g = torch.full((n,), 1e-3, device="cuda")
    g[n // 2:] = 3e-3
    p = [torch.zeros(n, device="cuda")]
    o = MoEAdamW(p, (0.9, 0.999), 1e-8, states="8bit", seed=5)
    for i in range(t):
        o.step(p, [g if i % 2 else 2 * g], 0.0)
    m, v = (x.double() for x in o.moments())
    em, ev = 0.0, 0.0
    for i in range(t):
        x = 1.0 if i % 2 else 2.0
        em, ev = 0.9 * em + 0.1 * x, 0.999 * ev + 0.001 * x * x
    tol = 6 * math.sqrt(t / 256 / (n / 2))
    for part, x in ((slice(0, n // 2), 1e-3), (slice(n // 2, n), 3e-3)):
        assert abs(float(m[part].mean()) / (em * x) - 1) < tol
        assert abs(float(v[part].mean()) / (ev * x * x) - 1) < tol


def test_8bit_extremes():
    """Blocks of zeros, of the largest and of the smallest gradients."""
    g = torch.zeros(7 * 32, device="cuda")
    g[32:64] = 1e18
    g[64:96] = 1e-18          # v = 1e-38: among the subnormals
    g[96] = 1e15
    g[97:128] = 1e-15         # far below the block's largest
    g[128:160] = 1e-30        # v = 0 in fp32
    g[160] = float("inf")
    g[192] = float("nan")
    p = [torch.ones(7 * 32, device="cuda")]
    o = MoEAdamW(p, (0.9, 0.99), 1e-8, states="8bit")
    o.step(p, [g], 0.125)
    m, v = o.moments()
    q = p[0]
    assert torch.equal(q[:32], torch.ones(32, device="cuda")) and not m[:32].any()
    assert not v[:32].any()
    assert torch.isfinite(m[:160]).all() and torch.isfinite(v[:160]).all()
    assert (v[32:128] > 0).all() and not v[128:160].any()
    # the first step moves every element by lr sign(g), as far as eps lets it
    want = 1 - 0.125 * (g / (g.abs() + 1e-8))[:160]
    assert float((q[:160] - want).abs().max()) < 1e-5
    # the infinity's and the NaN's blocks are NaN from here on, their other elements have moved still
    assert torch.isnan(m[160:]).all() and torch.isnan(v[160:]).all()
    assert torch.isfinite(q[161:192]).all() and torch.isfinite(q[193:]).all()


@pytest.mark.parametrize("states", ["fp32", "8bit"])
def test_many_tensors(states):
    """More tensors than a launch takes: as in parts of one launch each, and counted once."""
    r = np.random.default_rng(2)
    sizes = [int(n) for n in r.integers(0, 400, 600)]
    params, grads, _ = make(sizes, "fp32", "fp32", False, seed=4)
    o = MoEAdamW(params, BETAS, EPS, 0.01, states=states)
    ref = [(f64(p), np.zeros(p.numel()), np.zeros(p.numel())) for p in params]
    for t in (1, 2):
        if t == 1 or states == "fp32":
            ref = [oa.step(p, f64(g), m, v, t, 1e-2, 0.01, BETAS, EPS)
                   for (p, m, v), g in zip(ref, grads)]
        o.step(params, grads, 1e-2)
        if t == 1 or states == "fp32":
            for p, (want, _, _) in zip(params, ref):
                # (a relative 1e-4 of the step of at most lr a step, against 1e-2 for a wrong count)
                assert np.abs(f64(p) - want).max(initial=0) < 1e-6 * t + 2e-7
    assert o.steps() == 2


def test_no_tensors_and_empty_ones():
    o = MoEAdamW([], device="cuda")
    o.step([], [], 1e-3)
    assert o.steps() == 1
    e = [torch.empty(0, device="cuda"), torch.empty((3, 0), device="cuda")]
    o = MoEAdamW(e, states="8bit")
    o.step(e, e, 1e-3)
    assert o.steps() == 1 and o.moments()[0].numel() == 0


@pytest.mark.parametrize("states", ["fp32", "8bit"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan"), -float("inf")])
def test_a_norm_that_is_not_finite_skips_the_step(states, bad):
    params, grads, masters = make((3000, 70), "bf16", "bf16", True)
    o = MoEAdamW(params, states=states)
    o.step(params, grads, 1e-3, masters)
    kept = [t.clone() for t in (*params, *masters, o.m, o.v, o.counter)]
    grads[0][5] = float("nan")
    o.step(params, grads, 1e-3, masters, torch.tensor(bad, device="cuda"), 1.0)
    for a, b in zip(kept, (*params, *masters, o.m, o.v, o.counter)):
        assert torch.equal(a, b)
    grads[0][5] = 0.0
    o.step(params, grads, 1e-3, masters, MoEGradClip(4).norm(grads), 1.0)
    assert o.steps() == 2 and not torch.equal(kept[0], params[0])


def test_not_finite_without_a_norm():
    params, grads, _ = make((100,), "fp32", "fp32", False)
    grads[0][40] = float("nan")
    o = MoEAdamW(params)
    o.step(params, grads, 1e-3)
    bad = torch.isnan(params[0])
    assert int(bad.sum()) == 1 and bool(bad[40])


@pytest.mark.parametrize("states", ["fp32", "8bit"])
def test_captured(states):
    """A captured step counts on, and reads the learning rate and the norm anew at every replay."""
    def fresh():
        params, grads, masters = make((40000, 33), "bf16", "bf16", True)
        return params, grads, masters, MoEAdamW(params, BETAS, EPS, 0.1, states, seed=3), \
            MoEGradClip(2)
    params, grads, masters, o, c = fresh()
    lr = torch.tensor(0.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o.step(params, grads, lr, masters, c.norm(grads), 1.0)
    for t in range(4):
        lr.fill_(1e-3 * (t + 1))
        graph.replay()
    torch.cuda.synchronize()
    p2, g2, m2, o2, c2 = fresh()
    for t in range(4):
        lr.fill_(1e-3 * (t + 1))
        o2.step(p2, g2, lr, m2, c2.norm(g2), 1.0)
    assert o.steps() == o2.steps() == 4
    for a, b in zip((*params, *masters, o.m, o.v, o.counter), (*p2, *m2, o2.m, o2.v, o2.counter)):
        assert torch.equal(a, b)


def test_a_number_and_a_tensor_as_the_learning_rate_agree():
    a, g, _ = make((3000,), "fp32", "fp32", False)
    b = [t.clone() for t in a]
    MoEAdamW(a).step(a, g, 1e-3)
    MoEAdamW(b).step(b, g, torch.tensor([1e-3], device="cuda"))
    assert torch.equal(a[0], b[0])


@pytest.mark.parametrize("states", ["fp32", "8bit"])
def test_resumed(states):
    """A handle that takes over another's moments and count goes on as that one does."""
    params, grads, masters = make((5000, 40), "bf16", "bf16", True)
    a = MoEAdamW(params, BETAS, states=states, seed=9)
    for _ in range(3):
        a.step(params, grads, 1e-3, masters)
    p2, m2 = [t.clone() for t in params], [t.clone() for t in masters]
    b = MoEAdamW(p2, BETAS, states=states, seed=9)
    for name in ("m", "v", "m_scale", "v_scale"):
        if getattr(a, name) is not None:
            getattr(b, name).copy_(getattr(a, name))
    b.set_step(a.steps())
    a.step(params, grads, 1e-3, masters)
    b.step(p2, grads, 1e-3, m2)
    for x, y in zip((*params, *masters, a.m, a.v), (*p2, *m2, b.m, b.v)):
        assert torch.equal(x, y)


def test_past_32_bit_offsets():
    """A tensor of more than 2^31 elements and one behind it (their moments begin past 2^31)."""
    n = (1 << 31) + 40961
    p = [torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
         torch.zeros(100, dtype=torch.bfloat16, device="cuda")]
    g = [torch.full_like(t, 1e-3) for t in p]
    g[0][n - 20000:] = -1e-3
    o = MoEAdamW(p, BETAS, states="8bit")
    o.step(p, g, 0.25)
    # the first step moves every element by lr g / (|g| + eps), rounded to bf16
    for a, want in ((p[0][:50000], -0.25), (p[0][(1 << 31) - 50000:1 << 31], -0.25),
                    (p[0][n - 20000:], 0.25), (p[1], -0.25)):
        assert float((a.float() - want).abs().max()) <= 0.25 * (2 ** -8 + 2e-5)
    assert bool(o.v[n - 20000:n].any()) and not o.m[n:-(-n // 32) * 32].any()


def test_on_another_stream():
    params, grads, masters = make((300000,), "bf16", "bf16", True)
    p2, m2 = [t.clone() for t in params], [t.clone() for t in masters]
    a, b = MoEAdamW(params), MoEAdamW(p2)
    a.step(params, grads, 1e-3, masters)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.step(p2, grads, 1e-3, m2, stream=s)
    s.synchronize()
    assert torch.equal(params[0], p2[0]) and torch.equal(a.m, b.m)


def test_side_by_side():
    """Parts of one buffer next to each other, the same gradient for both: as tensors of their own."""
    p, g, w = make((1001, 1001), "bf16", "bf16", True, 9)
    out = []
    for shared in (False, True):
        if shared:
            flat = torch.cat(p)
            ps = [flat[:1001], flat[1001:]]
        else:
            ps = [t.clone() for t in p]
        ws = [t.clone() for t in w]
        o = MoEAdamW(ps, BETAS, EPS, 0.1)
        o.step(ps, [g[0], g[0] if shared else g[0].clone()], 1e-3, ws)
        out.append([t.clone() for t in (*ps, *ws, o.m, o.v)])
    assert all(torch.equal(a, b) for a, b in zip(*out))
