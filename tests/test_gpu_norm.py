"""MoELayerNorm on the GPU against the fp64 oracle.

Bounds (u: half an ulp of the stored type, e = 2^-24 of fp32).  A sum over H channels is a
chain of at most H / 256 + 32 fp32 additions (a thread's share, then a tree), so its
relative error is at most gam = (H / 256 + 32) e of the sum of magnitudes: the mean is off by at
most gam A, A = mean |x|, which moves xh by at most gam rstd A; the centred squares, rstd
and the products add a few more roundings.  With a factor 8 for those:
  y   : u |y| + 8 gam (|w| (|xh| + rstd A) + |b|)
  dx  : u |dx| + 16 gam rstd (|g| + <|g|> + (|xh| + rstd A) (<|g xh|> + rstd A <|g|>)) + e |add|
  dw  : u |dw| + (8 gam + gamT) sum_t |dy| (|xh| + rstd A),  db likewise with sum_t |dy|
where gamT = (T / 64 + 128) e covers the sums over the tokens.  fp16 adds half its smallest
subnormal step.
"""
import numpy as np
import pytest
import torch

import oracle.train as ot
from mixture_experts_layer_16_gb300 import MoELayerNorm
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {n: torch.finfo(t).eps / 2 for n, t in DT.items()}
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
E32 = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def data(T, H, dtype, param, seed=0, offset=1.0, pad=0):
    """x, dy, add [T, H] (rows H + pad apart), weight, bias."""
    r = np.random.default_rng(seed + 7 * T + H)

    def dev(a, dt):
        return torch.from_numpy(a.astype(np.float32)).to("cuda", DT[dt])

    def rows(a):
        if pad == 0:
            return dev(a, dtype)
        wide = torch.full((T, H + pad), 777.0, dtype=DT[dtype], device="cuda")
        wide[:, :H] = dev(a, dtype)
        return wide[:, :H]

    sc = np.exp(r.normal(0, 0.7, H))
    return dict(x=rows(r.standard_normal((T, H)) * sc + offset * r.standard_normal(H)),
                dy=rows(r.standard_normal((T, H))), add=rows(r.standard_normal((T, H))),
                w=dev(1 + 0.3 * r.standard_normal(H), param), b=dev(r.standard_normal(H), param))


def f64(t):
    return t.double().cpu().numpy()


def check(name, got, want, bound):
    bad = np.abs(got - want) > bound
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:3],
                           float((np.abs(got - want) / bound).max()))


def check_all(d, dtype, param, norm, y, grads, bias=True, add=True):
    x, dy, w, b = (f64(d[n]) for n in ("x", "dy", "w", "b"))
    T, H = x.shape
    gam, gamT = (H / 256 + 32) * E32, (T / 64 + 128) * E32
    f = ot.norm_forward(x, w, b if bias else None, EPS)
    g64 = ot.norm_backward(dy, x, w, EPS, f64(d["add"]) if add else None)
    A = np.abs(x).mean(1)[:, None]
    r = f["rstd"][:, None]
    axh = np.abs(f["xh"]) + r * A
    check("mean", f64(norm.mean), f["mean"], gam * A[:, 0] + 1e-38)
    # var's error: 2 gam of itself, plus the mean's error squared
    dvar = 4 * gam / f["rstd"] ** 2 + (gam * A[:, 0]) ** 2
    check("rstd", f64(norm.rstd), f["rstd"],
          f["rstd"] * (4 * E32 + 1 - 1 / np.sqrt(1 + f["rstd"] ** 2 * dvar)) * 2)
    check("y", f64(y), f["y"], U[dtype] * np.abs(f["y"]) + SUB[dtype] +
          8 * gam * (np.abs(w) * axh + (np.abs(b) if bias else 0)) + 1e-38)
    if grads is None:
        return
    dx, dw, db = grads
    g = np.abs(dy * w)
    gm, gx = g.mean(1)[:, None], (g * np.abs(f["xh"])).mean(1)[:, None]
    bound = U[dtype] * np.abs(g64["dx"]) + SUB[dtype] + \
        16 * gam * r * (g + gm + axh * (gx + r * A * gm)) + 1e-38
    if add:
        bound = bound + E32 * np.abs(f64(d["add"]))
    check("dx", f64(dx), g64["dx"], bound)
    ady = np.abs(dy)
    check("dweight", f64(dw), g64["dweight"], U[param] * np.abs(g64["dweight"]) + SUB[param] +
          (8 * gam + gamT) * (ady * axh).sum(0) + 1e-38)
    if bias:
        check("dbias", f64(db), g64["dbias"], U[param] * np.abs(g64["dbias"]) + SUB[param] +
              (8 * gam + gamT) * ady.sum(0) + 1e-38)
    else:
        assert db is None


def go(T, H, dtype="bf16", param="bf16", bias=True, add=True, **kw):
    d = data(T, H, dtype, param, **kw)
    n = MoELayerNorm(T, H, dtype, param, eps=EPS, bias=bias)
    y = n.forward(d["x"], d["w"], d["b"] if bias else None)
    grads = n.backward(d["dy"], d["x"], d["w"], dx_add=d["add"] if add else None)
    torch.cuda.synchronize()
    check_all(d, dtype, param, n, y, grads, bias, add)
    return d, n, y, grads


@pytest.mark.parametrize("T,H", [
    (1, 1), (1, 2), (2, 7), (1, 2048), (3, 8), (5, 64), (64, 128), (33, 129), (7, 1000), (129, 1111),
    (700, 256), (1201, 264), (300, 2048), (157, 4096), (40, 4104), (12, 8192), (9, 8191),
    (3, 16384), (5, 20001), (2, 70000)])
@pytest.mark.parametrize("dtype,param", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_norm(T, H, dtype, param):
    go(T, H, dtype, param, bias=(T + H) % 2 == 0, add=T % 2 == 1)


@pytest.mark.parametrize("dtype,param", [("bf16", "fp32"), ("fp16", "fp16")])
@pytest.mark.parametrize("T,H,pad", [(65, 256, 8), (65, 256, 3), (33, 1000, 24), (9, 333, 1),
                                     (1, 512, 5), (20, 4096, 64)])
def test_norm_rows_apart(dtype, param, T, H, pad):
    go(T, H, dtype, param, pad=pad)


@pytest.mark.parametrize("T", [4096, 5003])
def test_norm_many_rows(T):
    go(T, 512)
    go(T, 100, "fp32", "fp32", bias=False)


@pytest.mark.parametrize("H", [24, 520, 640, 768, 1016, 1272, 1536, 1792, 2056, 2560, 3333, 4100,
                               5120, 6144, 7168, 8176, 8191, 8192, 9000, 16384])
@pytest.mark.parametrize("dtype,param", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_norm_widths(H, dtype, param):
    """More rows than CTAs: every number of units a thread, and both sides of its limits."""
    go(331, H, dtype, param, bias=H % 3 != 0, add=H % 16 == 0)


@pytest.mark.parametrize("T,H,dtype,param", [
    *[(1300, H, "bf16", "bf16") for H in (129, 207, 250, 333, 511, 767, 1001, 1201, 1500, 1780,
                                          2047, 2049, 3333, 4095, 7001, 8191)],
    (1300, 1001, "fp16", "fp16"), (1300, 511, "fp16", "fp32"), (1300, 6001, "bf16", "fp32"),
    *[(7400, H, "fp32", "fp32") for H in (66, 67, 129, 255, 511, 1023, 1111, 1153, 1537)],
    (1300, 511, "fp32", "fp32"), (1300, 8191, "fp32", "fp32"), (1300, 8190, "fp32", "fp32")])
def test_norm_many_rows_on_no_boundary(T, H, dtype, param):
    """Forward: every number of units a thread, parts of a warp and several warps a row."""
    d = data(T, H, dtype, param, pad=0 if H % 2 else 8)
    n = MoELayerNorm(T, H, dtype, param, eps=EPS, bias=H % 3 != 0)
    y = n.forward(d["x"], d["w"], d["b"] if n.bias else None)
    check_all(d, dtype, param, n, y, None, n.bias)


@pytest.mark.parametrize("T", [152, 153, 304, 305, 608, 609, 1216, 1217])
@pytest.mark.parametrize("H,dtype", [(256, "bf16"), (1000, "bf16"), (2048, "fp16"), (1001, "bf16"),
                                     (128, "fp32"), (515, "fp32"), (1024, "fp32")])
def test_norm_one_row_a_group(T, H, dtype):
    """Few rows, up to one for every group of threads of the grid, and one more."""
    d = data(T, H, dtype, dtype)
    n = MoELayerNorm(T, H, dtype, eps=EPS)
    check_all(d, dtype, dtype, n, n.forward(d["x"], d["w"], d["b"]), None)


@pytest.mark.parametrize("T", [20, 152, 153, 304, 305])
@pytest.mark.parametrize("H,dtype", [(520, "bf16"), (1000, "bf16"), (1001, "fp16"), (8192, "bf16"),
                                     (515, "fp32"), (4096, "fp32")])
def test_norm_backward_few_rows(T, H, dtype):
    """One row a CTA (whole rows of partial sums), some groups of a CTA, and one more."""
    go(T, H, dtype, dtype, bias=T % 2 == 0, add=T % 3 == 0)


@pytest.mark.parametrize("T,H,dtype,param", [
    (700, 136, "bf16", "bf16"), (700, 207, "fp16", "fp32"), (700, 250, "bf16", "bf16"),
    (700, 300, "bf16", "fp32"), (700, 333, "bf16", "bf16"), (700, 511, "fp16", "fp16"),
    (700, 600, "bf16", "bf16"), (400, 4095, "bf16", "bf16"), (330, 8190, "bf16", "bf16"),
    (330, 8191, "fp16", "fp32"), (330, 10007, "bf16", "bf16"), (330, 12274, "bf16", "bf16"),
    (330, 12275, "bf16", "bf16"), (330, 12288, "fp16", "fp16"), (1300, 12288, "bf16", "bf16"),
    (1300, 9001, "bf16", "fp32"), (1220, 16383, "bf16", "bf16"), (330, 12296, "bf16", "bf16")])
def test_norm_three_units_and_wide_rows(T, H, dtype, param):
    go(T, H, dtype, param, bias=H % 3 != 0, add=H % 2 == 0)


@pytest.mark.parametrize("H", [256, 1001])
def test_norm_offsets_past_32_bits(H):
    """Rows a million elements apart: the last ones begin past 2^32 elements.  Bit by bit as
    with dense rows."""
    T, ld = 4200, (1 << 20) + (8 if H % 8 == 0 else H % 8 + 8)   # (rows are cut alike)
    d = data(T, H, "bf16", "bf16")
    n = MoELayerNorm(T, H, eps=EPS)
    y = n.forward(d["x"], d["w"], d["b"])
    dx, dw, db = n.backward(d["dy"], d["x"], d["w"], dx_add=d["add"])
    x2, dy2, y2 = (torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)[:, :H]
                   for _ in range(3))
    x2.copy_(d["x"])
    dy2.copy_(d["dy"])
    assert torch.equal(n.forward(x2, d["w"], d["b"], y=y2), y)
    out = (y2, torch.empty_like(dw), torch.empty_like(db))
    got = n.backward(dy2, x2, d["w"], dx_add=d["add"] if H % 8 == 0 else None, out=out)
    if H % 8:
        dx, dw, db = n.backward(d["dy"], d["x"], d["w"])
    for a, b in zip(got, (dx, dw, db)):
        assert torch.equal(a, b)


def test_norm_operands_cut_differently():
    """Rows of x lie apart, y and dx are dense with an odd width: no common cut."""
    T, H = 300, 333
    d = data(T, H, "bf16", "bf16", pad=3)
    n = MoELayerNorm(T, H, eps=EPS)
    y = n.forward(d["x"], d["w"], d["b"])
    check_all(d, "bf16", "bf16", n, y, n.backward(d["dy"], d["x"], d["w"], dx_add=d["add"]))


def test_norm_unaligned_pointers():
    # a row that starts on its element only (2 bytes past a 16-byte boundary)
    T, H = 19, 256
    d = data(T, H, "bf16", "bf16")
    sh = {k: torch.empty(T * H + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, H).copy_(d[k])
          for k in ("x", "dy", "add")}
    n = MoELayerNorm(T, H, eps=EPS)
    y = n.forward(sh["x"], d["w"], d["b"])
    grads = n.backward(sh["dy"], sh["x"], d["w"], dx_add=sh["add"])
    check_all(d, "bf16", "bf16", n, y, grads)
    # parameters off their 16-byte boundary, rows on theirs
    ow, ob = (torch.empty(H + 1, dtype=torch.bfloat16, device="cuda")[1:].copy_(d[k]) for k in "wb")
    out = (torch.empty_like(d["x"]), torch.empty(H + 1, dtype=torch.bfloat16, device="cuda")[1:],
           torch.empty(H + 1, dtype=torch.bfloat16, device="cuda")[1:])
    y2 = n.forward(d["x"], ow, ob)
    check_all(d, "bf16", "bf16", n, y2, n.backward(d["dy"], d["x"], ow, dx_add=d["add"], out=out))


@pytest.mark.parametrize("offset", [0.0, 300.0])
def test_norm_large_mean_and_constant_rows(offset):
    """A mean far above the spread, and rows of one value (variance 0: rstd = eps^-1/2)."""
    T, H = 20, 1024
    d = data(T, H, "fp32", "fp32", offset=offset)
    d["x"][3] = 5.0
    d["x"][4] = 0.0
    n = MoELayerNorm(T, H, "fp32", eps=EPS)
    y = n.forward(d["x"], d["w"], d["b"])
    check_all(d, "fp32", "fp32", n, y, n.backward(d["dy"], d["x"], d["w"], dx_add=d["add"]))
    assert torch.equal(y[4], d["b"])


def test_norm_in_place_and_out():
    T, H = 50, 768
    d, n, y, grads = go(T, H)
    x2 = d["x"].clone()
    n.forward(x2, d["w"], d["b"], y=x2)
    assert torch.equal(x2, y)
    n.forward(d["x"], d["w"], d["b"])
    add2 = d["add"].clone()
    out = (add2, torch.empty_like(d["w"]), torch.empty_like(d["b"]))
    n.backward(d["dy"], d["x"], d["w"], dx_add=add2, out=out)
    for a, b in zip(out, grads):
        assert torch.equal(a, b)


def test_norm_nan_and_inf_stay_in_their_row():
    T, H = 40, 640
    d = data(T, H, "bf16", "bf16")
    clean = MoELayerNorm(T, H, eps=EPS)
    y0 = clean.forward(d["x"], d["w"], d["b"])
    x = d["x"].clone()
    x[7, 3], x[21, 600] = float("nan"), float("inf")
    n = MoELayerNorm(T, H, eps=EPS)
    y = n.forward(x, d["w"], d["b"])
    keep = [t for t in range(T) if t not in (7, 21)]
    assert torch.equal(y[keep], y0[keep]) and y[7].isnan().all() and y[21].isnan().any()
    dx, dw, db = n.backward(d["dy"], x, d["w"])
    clean.forward(d["x"], d["w"], d["b"])
    dx0, _, db0 = clean.backward(d["dy"], d["x"], d["w"])
    assert torch.equal(dx[keep], dx0[keep]) and torch.equal(db, db0) and dw.isnan().all()


def test_norm_gradient_against_differences():
    """<gradient, v> against the central difference of the oracle's loss, in fp32."""
    T, H = 31, 200
    d = data(T, H, "fp32", "fp32")
    n = MoELayerNorm(T, H, "fp32", eps=EPS)
    n.forward(d["x"], d["w"], d["b"])
    grads = n.backward(d["dy"], d["x"], d["w"])
    x, w, b, dy = (f64(d[k]) for k in ("x", "w", "b", "dy"))
    r = np.random.default_rng(1)
    h = 1e-5
    for i, (val, g) in enumerate(zip((x, w, b), grads)):
        v = r.standard_normal(val.shape)

        def L(z):
            a = [x, w, b]
            a[i] = z
            return float((ot.norm_forward(*a, EPS)["y"] * dy).sum())
        num = (L(val + h * v) - L(val - h * v)) / (2 * h)
        # fp32 gradients: 1e-5 of the terms' magnitudes; the difference itself is good to h^2
        assert abs(num - (f64(g) * v).sum()) <= 1e-5 * np.abs(f64(g) * v).sum() + 1e-6


def test_norm_repeats_bit_for_bit_and_on_another_stream():
    d, n, y, grads = go(3000, 384)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, out = torch.empty_like(y), tuple(torch.empty_like(g) for g in grads)
    n.forward(d["x"], d["w"], d["b"], y=y2, stream=s)
    n.backward(d["dy"], d["x"], d["w"], dx_add=d["add"], out=out, stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(out, grads))


def test_norm_in_a_cuda_graph():
    d, n, y, grads = go(257, 512)
    y2, out = torch.empty_like(y), tuple(torch.empty_like(g) for g in grads)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n.forward(d["x"], d["w"], d["b"], y=y2)
        n.backward(d["dy"], d["x"], d["w"], dx_add=d["add"], out=out)
    for _ in range(2):
        for t in (y2, *out):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(out, grads))


def test_norm_rows_past_32_bits():
    """Rows so far apart that their offsets pass 2^31 elements (one buffer of 5 GB)."""
    T, H, ld = 5, 256, (1 << 29) + 8
    d = data(T, H, "bf16", "bf16")
    big = torch.empty((T - 1) * ld + H, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((T, H), (ld, 1))
    x.copy_(d["x"])
    n = MoELayerNorm(T, H, eps=EPS)
    y = n.forward(x, d["w"], d["b"])
    check_all(d, "bf16", "bf16", n, y, n.backward(d["dy"], x, d["w"], dx_add=d["add"]))
