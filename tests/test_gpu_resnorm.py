"""MoEResidualNorm on the GPU against the fp64 oracle.

Bounds (u: half an ulp of the stored type, e = 2^-24).  A sum over H channels is a chain of at most
H / 256 + 32 fp32 additions, so it is within gam = (H / 256 + 40) e of its terms' sizes, products and
coefficients' roundings included; the reciprocal root is within 2 ulp (4 e).  Forward:
  rstd : (gam + 6 e) rstd
  out  : u |out| + eo,  eo = e |x| + (gam + 12 e) |c f rstd_f|
  n    : u |n| + |w| ro eo + |n| (gam + 8 e + ro <eo^2>^(1/2))
Backward, from the kept reciprocal norms, with A = <|oh v|>, B = sum |c fh| (|dout| + ro |v|) +
ro A sum |c fh oh| and eD = 2 e |dout| + 2 gam ro (|v| + |oh| A):
  dx : u |dx| + eD
  df : u |df| + rf (|c g| eD + 4 e |c g D| + |fh| (2 gam |g| B / H))         (without the norm: |c g| eD + ...)
  dgate_t : u |.| + 2 gam B
  sums over the tokens (at most T / 64 + 128 additions in a chain, gamT of that many e):
  K : sum |g fh| eD + gamT sum |g fh D|,  dw_pre : (gamT + 4 e) sum |dn oh|
all with a factor 2 for what multiplies them.  fp16 adds half its smallest subnormal step.
"""
import numpy as np
import pytest
import torch

import oracle.resnorm as orn
from mixture_experts_layer_16_gb300 import MoEError, MoEResidualNorm
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {n: torch.finfo(t).eps / 2 for n, t in DT.items()}
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
E = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def data(T, H, dtype, res, param, post, gate, pre, seed=0, pad=0, shift=0):
    """The operands, rows H + pad apart, their storage beginning `shift` elements past a vector."""
    r = np.random.default_rng(seed + 7 * T + H)

    def dev(a, dt):
        return torch.from_numpy(a.astype(np.float32)).to("cuda", DT[dt])

    def rows(a, dt):
        if pad == 0 and shift == 0:
            return dev(a, dt)
        wide = torch.full((T * (H + pad) + shift,), 777.0, dtype=DT[dt], device="cuda")
        v = wide[shift:].view(T, H + pad)[:, :H]
        v.copy_(dev(a, dt))
        return v
    sc = np.exp(r.normal(0, 0.7, H))
    return dict(
        x=rows(r.standard_normal((T, H)) * sc, res), f=rows(0.6 * r.standard_normal((T, H)), dtype),
        dout=rows(r.standard_normal((T, H)), res), dn=rows(r.standard_normal((T, H)), dtype),
        post_weight=dev(1 + 0.3 * r.standard_normal(H), param) if post else None,
        pre_weight=dev(1 + 0.3 * r.standard_normal(H), param) if pre else None,
        gate=None if gate is None else dev(
            0.5 + 0.3 * r.standard_normal(H if gate == "channel" else T), param))


def check(name, got, want, bound):
    bad = ~(np.abs(f64(got) - want) <= bound)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:3],
                           float((np.abs(f64(got) - want) / bound).max()))


def check_forward(h, d, types, out, n, has_f=True):
    dtype, res, _ = types
    w1, w2, g = f64(d["post_weight"]), f64(d["pre_weight"]), f64(d["gate"])
    x, f = f64(d["x"]), f64(d["f"]) if has_f else None
    H = h.H
    gam = (H / 256 + 40) * E
    scale, eps = h.shape.scale, h.shape.eps
    want = orn.forward(x, f, w1 if has_f else None, g if has_f else None, w2, h.gate, scale, eps)
    eo = np.zeros_like(x)
    if has_f:
        eo = E * np.abs(x) + (gam + 12 * E) * np.abs(want["out"] - x) + 1e-44
        check("out", out, want["out"], U[res] * np.abs(want["out"]) + SUB[res] + 2 * eo)
        if w1 is not None:
            check("rstd_f", h.rstd_f, want["rstd_f"], 2 * (gam + 6 * E) * want["rstd_f"])
    if w2 is None:
        assert n is None
        return
    ro = want["rstd_out"]
    rms = np.sqrt((eo ** 2).mean(axis=1))
    check("rstd_out", h.rstd_out, ro, 2 * ro * (gam + 6 * E + ro * rms))
    check("n", n, want["n"], U[dtype] * np.abs(want["n"]) + SUB[dtype] + 2 * (
        np.abs(w2) * ro[:, None] * eo + np.abs(want["n"]) * (gam + 8 * E + (ro * rms)[:, None]))
        + 1e-44)


def check_backward(h, d, types, out, got, has_f=True, has_dout=True):
    dtype, res, param = types
    dx, df, grads = got
    w1, w2 = f64(d["post_weight"]), f64(d["pre_weight"])
    f = f64(d["f"]) if has_f else None
    gate = f64(d["gate"]) if has_f else None
    dout = f64(d["dout"]) if has_dout else None
    dn, o = (f64(d["dn"]), f64(out)) if w2 is not None else (None, None)
    T, H = h.T, h.H
    rf, ro = f64(h.rstd_f), f64(h.rstd_out)
    kind, scale = (h.gate if has_f else None), h.shape.scale
    want = orn.backward(dout, dn, o, f, w1 if has_f else None, gate, w2, kind, scale, rf, ro)
    gam, gamT = (H / 256 + 40) * E, (T / 64 + 128) * E
    z = np.zeros((T, H))
    ad = np.abs(dout) if has_dout else z
    oh, v = (np.abs(o * ro[:, None]), np.abs(dn * w2)) if w2 is not None else (z, z)
    ro = ro[:, None] if w2 is not None else np.zeros((T, 1))
    A = (oh * v).mean(axis=1)[:, None]
    eD = 2 * E * ad + 2 * gam * ro * (v + oh * A) + 1e-44
    D = np.abs(want["dx"])
    check("dx", dx, want["dx"], U[res] * D + SUB[res] + 2 * eD)
    if w2 is not None:
        check("dpre", grads["pre_weight"], want["pre_weight"], U[param] * np.abs(want["pre_weight"])
              + SUB[param] + 2 * (gamT + 4 * E) * (np.abs(dn) * oh).sum(axis=0) + 1e-44)
    if not has_f:
        assert df is None and set(grads) == ({"pre_weight"} if w2 is not None else set())
        return
    c = scale * np.ones((1, H)) * (w1 if w1 is not None else 1)
    if kind == "channel":
        c = c * gate
    gt = np.abs(gate)[:, None] if kind == "token" else np.ones((T, 1))
    c = np.abs(c)
    rf1 = rf[:, None] if w1 is not None else np.ones((T, 1))
    fh = np.abs(f) * rf1
    B = (c * fh * (ad + ro * v)).sum(axis=1)[:, None] + ro * A * (c * fh * oh).sum(axis=1)[:, None]
    e = c * gt * eD + 8 * E * c * gt * D
    if w1 is not None:
        e = rf1 * (e + fh * (2 * gam * gt * B / H))
    check("df", df, want["df"], U[dtype] * np.abs(want["df"]) + SUB[dtype] + 2 * e + 1e-44)
    eK = (gt * fh * eD).sum(axis=0) + gamT * (gt * fh * D).sum(axis=0)
    if w1 is not None:
        k = abs(scale) * (np.abs(gate) if kind == "channel" else 1)
        check("dpost", grads["post_weight"], want["post_weight"], U[param] *
              np.abs(want["post_weight"]) + SUB[param] + 2 * k * eK + 1e-44)
    if kind == "channel":
        k = abs(scale) * (np.abs(w1) if w1 is not None else 1)
        check("dgate", grads["gate"], want["gate"], U[param] * np.abs(want["gate"]) + SUB[param] +
              2 * k * eK + 1e-44)
    if kind == "token":
        check("dgate", grads["gate"], want["gate"], U[param] * np.abs(want["gate"]) + SUB[param] +
              4 * gam * B[:, 0] + 1e-44)


FORMS = [(True, "channel", True), (True, None, True), (False, "token", True), (True, "token", False),
         (False, "channel", False), (False, None, True), (False, None, False), (True, "token", True)]
TYPES = [("bf16", "bf16", "bf16"), ("bf16", "fp32", "fp32"), ("fp16", "fp16", "fp32"),
         ("fp32", "fp32", "fp32"), ("fp16", "fp32", "fp16")]


def go(T, H, types, form, scale=0.7, has_dout=True, **kw):
    post, gate, pre = form
    d = data(T, H, *types, *form, **kw)
    h = MoEResidualNorm(T, H, *types, post=post, gate=gate, pre=pre, scale=scale, eps=EPS)
    p = dict(post_weight=d["post_weight"], gate=d["gate"], pre_weight=d["pre_weight"])
    out, n = h.forward(d["x"], d["f"], **p)
    got = h.backward(d["dout"] if has_dout else None, d["dn"] if pre else None, out, d["f"], **p)
    torch.cuda.synchronize()
    check_forward(h, d, types, out, n)
    check_backward(h, d, types, out, got, has_dout=has_dout)
    return h, d, p, out, n, got


@pytest.mark.parametrize("T,H", [
    (1, 1), (1, 2), (2, 7), (1, 2048), (3, 8), (5, 64), (64, 128), (33, 129), (7, 1000), (129, 1111),
    (700, 256), (1201, 264), (700, 24), (300, 2048), (157, 4096), (40, 4104), (12, 8192), (9, 8191),
    (3, 16384), (5, 20001), (400, 4097), (2, 70000)])
@pytest.mark.parametrize("types", TYPES)
def test_forms(T, H, types):
    for i, form in enumerate(FORMS):
        if (i + T + H) % 2 and H > 300:
            continue
        go(T, H, types, form, has_dout=not form[2] or i % 3 != 0)


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (1, 0), (0, 1), (24, 8), (5, 3)])
def test_rows_apart(types, pad, shift):
    for H in (256, 200, 1000):
        go(70, H, types, FORMS[0], pad=pad, shift=shift)
        go(3, H, types, FORMS[7], pad=pad, shift=shift)
    go(4, 8200, types, FORMS[0], pad=pad, shift=shift)


@pytest.mark.parametrize("T,H", [(1, 2048), (300, 264), (77, 129), (5, 9000)])
@pytest.mark.parametrize("types", TYPES)
def test_the_norm_alone(T, H, types):
    """Without a block's output: the RMS norm of x and its backward, joined with the residual's."""
    d = data(T, H, *types, True, "channel", True)
    h = MoEResidualNorm(T, H, *types, post=True, gate="channel", eps=EPS)
    out, n = h.forward(d["x"], pre_weight=d["pre_weight"])
    assert out is d["x"]
    check_forward(h, d, types, out, n, has_f=False)
    for dout in (d["dout"], None):
        got = h.backward(dout, d["dn"], d["x"], pre_weight=d["pre_weight"])
        check_backward(h, d, types, out, got, has_f=False, has_dout=dout is not None)


@pytest.mark.parametrize("H", [256, 129, 9000])
def test_in_place(H):
    types = TYPES[1]
    d = data(50, H, *types, *FORMS[0])
    h = MoEResidualNorm(50, H, *types, post=True, gate="channel")
    p = dict(post_weight=d["post_weight"], gate=d["gate"], pre_weight=d["pre_weight"])
    out, n = h.forward(d["x"], d["f"], **p)
    x = d["x"].clone()
    o2, n2 = h.forward(x, d["f"], out=x, **p)
    assert o2 is x and torch.equal(x, out) and torch.equal(n, n2)


def test_overlaps():
    T, H = 20, 64
    types = TYPES[0]
    d = data(T, H, *types, *FORMS[1])
    h = MoEResidualNorm(T, H)
    p = dict(post_weight=d["post_weight"], pre_weight=d["pre_weight"])
    buf = torch.zeros((T + 1) * H, dtype=torch.bfloat16, device="cuda")
    a, b = buf[:T * H].view(T, H), buf[H:].view(T, H)
    with pytest.raises(MoEError):
        h.forward(a, d["f"], out=b, **p)
    with pytest.raises(MoEError):
        h.forward(d["x"], a, out=a, **p)
    wide = torch.zeros((T, 2 * H), dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = d["x"]
    want, n = h.forward(d["x"], d["f"], **p)
    out, n2 = h.forward(wide[:, :H], d["f"], out=wide[:, H:], **p)   # in one another's gaps
    assert torch.equal(out, want) and torch.equal(n, n2) and torch.equal(wide[:, :H], d["x"])
    with pytest.raises(MoEError):
        h.forward(wide[:, :H], d["f"], out=wide[:, H - 8:2 * H - 8], **p)


@pytest.mark.parametrize("types", TYPES)
def test_extreme_rows(types):
    """Rows of zeros, of tiny and of large values, and one with an infinity and a NaN: each in
    its own row."""
    T, H = 12, 512
    d = data(T, H, *types, True, None, True)
    h = MoEResidualNorm(T, H, *types, eps=EPS)
    p = dict(post_weight=d["post_weight"], pre_weight=d["pre_weight"])
    want = h.forward(d["x"], d["f"], **p)
    d["f"][1] = 0
    d["x"][2] = 0
    d["f"][2] = 0
    d["f"][3] *= 1e-3
    d["x"][4] *= 200
    d["f"][5, 7] = float("nan")
    d["x"][6, 9] = float("inf")
    out, n = h.forward(d["x"], d["f"], **p)
    good = [0, 7, 8, 9, 10, 11]
    assert torch.equal(out[good], want[0][good]) and torch.equal(n[good], want[1][good])
    assert not out[2].any() and not n[2].any()
    assert torch.isnan(out[5]).all() and torch.isnan(n[5]).all()
    assert torch.isinf(out[6, 9])
    g = h.backward(d["dout"], d["dn"], out, d["f"], **p)
    finite = [0, 1, 2, 3, 4, 7, 8, 9, 10, 11]
    assert torch.isfinite(g[0][finite]).all()
    # a row of zeros has a reciprocal norm of eps^(-1/2) = 1000, two of them a gradient of 10^6 times
    # dn: above fp16's 65504, where infinity is what the value rounds to
    want = orn.backward(f64(d["dout"])[finite], f64(d["dn"])[finite], f64(out)[finite],
                        f64(d["f"])[finite], f64(d["post_weight"]), None, f64(d["pre_weight"]),
                        None, 1.0, f64(h.rstd_f)[finite], f64(h.rstd_out)[finite])["df"]
    fits = np.abs(want) < 0.99 * torch.finfo(DT[types[0]]).max
    assert np.isfinite(f64(g[1])[finite][fits]).all() and fits[0].all() and fits[3:].all()


def test_gradient_against_differences():
    """The oracle's gradients against central differences of its forward (fp64)."""
    r = np.random.default_rng(3)
    T, H = 3, 10
    for post, kind, pre in FORMS:
        v = dict(x=r.standard_normal((T, H)), f=r.standard_normal((T, H)),
                 w_post=1 + 0.3 * r.standard_normal(H) if post else None,
                 gate=None if kind is None else r.standard_normal(H if kind == "channel" else T),
                 w_pre=1 + 0.3 * r.standard_normal(H) if pre else None)
        go_, gn = r.standard_normal((T, H)), r.standard_normal((T, H))

        def loss(**kw):
            a = orn.forward(**{**v, **kw}, kind=kind, scale=0.7, eps=1e-3)
            return (a["out"] * go_).sum() + ((a["n"] * gn).sum() if pre else 0)
        a = orn.forward(**v, kind=kind, scale=0.7, eps=1e-3)
        g = orn.backward(go_, gn if pre else None, a["out"], v["f"], v["w_post"], v["gate"], v["w_pre"],
                         kind, 0.7, a.get("rstd_f"), a.get("rstd_out"))
        names = dict(x="dx", f="df", w_post="post_weight", gate="gate", w_pre="pre_weight")
        for k, name in names.items():
            if v[k] is None:
                continue
            for i in np.ndindex(v[k].shape):
                h = np.zeros_like(v[k])
                h[i] = 1e-6
                num = (loss(**{k: v[k] + h}) - loss(**{k: v[k] - h})) / 2e-6
                assert abs(num - g[name][i]) < 1e-6 * max(1, abs(num)), (name, i)


def test_repeats_and_captured():
    T, H = 700, 2048
    types = TYPES[0]
    h, d, p, out, n, got = go(T, H, types, FORMS[0])

    def run(s=None):
        o, n_ = h.forward(d["x"], d["f"], stream=s, **p)
        dx, df, gr = h.backward(d["dout"], d["dn"], o, d["f"], stream=s, **p)
        return [o, n_, dx, df, *(gr[k] for k in sorted(gr))]
    want = [out, n, got[0], got[1], *(got[2][k] for k in sorted(got[2]))]
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        res = run(s)
    for t in (*res, h.rstd_f, h.rstd_out, h.workspace):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(res, want))


def test_past_32_bit_offsets():
    T, H = (1 << 20) + 300, 2048
    types = TYPES[0]
    d = data(400, H, *types, *FORMS[0])
    big = {k: torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
           for k in ("x", "f", "dout", "dn")}
    for k, t in big.items():
        t[-400:] = d[k]
    p = dict(post_weight=d["post_weight"], gate=d["gate"], pre_weight=d["pre_weight"])
    h = MoEResidualNorm(T, H, post=True, gate="channel", scale=0.7)
    out, n = h.forward(big["x"], big["f"], **p)
    dx, df, grads = h.backward(big["dout"], big["dn"], out, big["f"], **p)
    s = MoEResidualNorm(400, H, post=True, gate="channel", scale=0.7)
    s.rstd_f, s.rstd_out = h.rstd_f[-400:], h.rstd_out[-400:]
    check_forward(s, d, types, out[-400:], n[-400:])
    s.T = T            # (rows of zeros add nothing, but their additions are in the chains)
    z = dict(d)
    s.T = 400
    check_backward(s, z, types, out[-400:], (dx[-400:], df[-400:], grads))
    assert not out[:-400].any() and not df[1000:2000].any()


def test_load_stats_and_refusals():
    T, H = 30, 64
    d = data(T, H, *TYPES[0], *FORMS[0])
    p = dict(post_weight=d["post_weight"], gate=d["gate"], pre_weight=d["pre_weight"])
    a = MoEResidualNorm(T, H, gate="channel")
    out, _ = a.forward(d["x"], d["f"], **p)
    b = MoEResidualNorm(T, H, gate="channel")
    with pytest.raises(RuntimeError):
        b.backward(d["dout"], d["dn"], out, d["f"], **p)
    b.load_stats(a.rstd_f, a.rstd_out)
    x, y = (h.backward(d["dout"], d["dn"], out, d["f"], **p) for h in (a, b))
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    a.forward(d["x"], pre_weight=d["pre_weight"])
    with pytest.raises(ValueError):      # that forward had no f
        a.backward(d["dout"], d["dn"], out, d["f"], **p)


@pytest.mark.parametrize("T,H", [(1500, 1024), (1101, 2048), (1000, 2304), (700, 4104), (471, 8192),
                                 (461, 7003), (330, 5000)])
@pytest.mark.parametrize("types", TYPES)
def test_many_rows(T, H, types):
    """Three rows and more to every group of threads, groups without a last row among them."""
    for form in (FORMS[0], FORMS[3], FORMS[7]):
        go(T, H, types, form)
