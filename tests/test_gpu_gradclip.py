"""MoEGradClip on the GPU against the fp64 oracle.

Bounds: a thread sums at most 64 squares in fp32 (the rest in fp64), so the sum of squares
is off by at most 64 e of itself, e = 2^-24, and the norm by half that plus its rounding:
40 e.  A clipped element: its type's half ulp, plus 48 e for the norm's share, the
division and the product."""
import numpy as np
import pytest
import torch

import oracle.train as ot
from mixture_experts_layer_16_gb300 import MoEGradClip
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
BF, FH, F32 = torch.bfloat16, torch.float16, torch.float32
U = {t: torch.finfo(t).eps / 2 for t in (BF, FH, F32)}
SUB = {BF: 2.0 ** -134, FH: 2.0 ** -25, F32: 2.0 ** -149}
E32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def make(sizes, dtypes, scale=1.0, seed=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + len(sizes))
    return [(scale * torch.randn(n, generator=gen, device="cuda")).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


def f64(t):
    return t.double().cpu().numpy().reshape(-1)


def check(grads, max_norm, out="same", clip=None):
    src = [f64(g) for g in grads]
    n64, want = ot.grad_clip(src, max_norm)
    clip = MoEGradClip(max(len(grads), 1)) if clip is None else clip
    norm = clip.norm(grads)
    work = [g.clone() for g in grads]
    if out == "inplace":
        dst = work
        n2 = clip.clip(work, max_norm)
    else:
        dst = [torch.full(g.shape, 7.0, dtype=F32 if out == "fp32" else g.dtype, device="cuda")
               for g in grads]
        n2 = clip.clip(work, max_norm, out=dst)
        assert all(torch.equal(a, b) for a, b in zip(work, grads))
    torch.cuda.synchronize()
    assert norm.shape == () and torch.equal(norm, n2)
    if n64 > torch.finfo(F32).max:             # no fp32 number: infinite, coef 0
        assert torch.isinf(norm) and not any(d.any() for d in dst)
        return n64, norm, dst
    assert abs(float(norm) - n64) <= 40 * E32 * n64
    for d, w in zip(dst, want):
        err = np.abs(f64(d) - w)
        assert np.all(err <= (U[d.dtype] + 48 * E32) * np.abs(w) + SUB[d.dtype])
    return n64, norm, dst


SIZES = [1, 2, 7, 8, 9, 255, 4096, 16383, 16384, 16385, 40000, 0, 3, 100003]


@pytest.mark.parametrize("dtypes", [(BF,), (FH,), (F32,), (BF, F32, FH)])
@pytest.mark.parametrize("out", ["inplace", "same", "fp32"])
def test_clip_types_and_outputs(dtypes, out):
    g = make(SIZES, dtypes)
    check(g, 0.5, out)
    check(g, 1e6, out)           # under the bound


@pytest.mark.parametrize("sizes", [[], [0], [0, 0, 5], [1], [16384 * 3 + 1]])
def test_clip_few(sizes):
    check(make(sizes, (F32,)), 0.1, "inplace")


def test_clip_under_the_bound_keeps_every_bit():
    g = make(SIZES, (BF, F32, FH))
    w = [t.clone() for t in g]
    MoEGradClip().clip(w, 1e9)
    o = [torch.empty_like(t) for t in g]
    MoEGradClip().clip(g, float("inf"), out=o)
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(g, w, o))


def test_clip_more_tensors_than_one_launch_takes():
    r = np.random.default_rng(0)
    sizes = [int(n) for n in r.integers(0, 700, 1000)] + [200000]
    for out in ("inplace", "fp32"):
        check(make(sizes, (BF, F32)), 1.0, out)


def test_clip_views_off_the_boundary():
    """Slices of one flat buffer (any element offset), clipped into slices that share
    their offsets and into ones that do not."""
    for dt, odt in ((BF, BF), (BF, F32), (F32, F32), (FH, FH)):
        flat = torch.randn(60000, device="cuda").to(dt)
        cuts = [0, 1, 18, 20000, 20003, 37001, 60000]
        g = [flat[a:b] for a, b in zip(cuts[:-1], cuts[1:])]
        for shift in (0, 1, 3):
            o = torch.zeros(60000 + shift, dtype=odt, device="cuda")
            dst = [o[a + shift:b + shift] for a, b in zip(cuts[:-1], cuts[1:])]
            c = MoEGradClip(16)
            norm = c.clip(g, 2.0, out=dst)
            n64, want = ot.grad_clip([f64(t) for t in g], 2.0)
            assert abs(float(norm) - n64) <= 40 * E32 * n64
            for d, w in zip(dst, want):
                assert np.all(np.abs(f64(d) - w) <=
                              (U[odt] + 48 * E32) * np.abs(w) + SUB[odt])
            assert not o[:shift].any()


@pytest.mark.parametrize("scale", [1e30, 3e37, 1e-25, 1e-37])
def test_clip_squares_out_of_fp32_range(scale):
    for dt in (F32, BF):
        g = make([5000, 70, 16384], (dt,), scale)
        g[1][:] = 0
        check(g, scale * 10, "same")
    mixed = make([3000], (F32,), scale) + make([3000], (F32,), 1.0)
    check(mixed, 0.25, "same")


def test_clip_zero_gradients():
    g = [torch.zeros(50000, dtype=BF, device="cuda"), torch.zeros(3, device="cuda")]
    n, norm, dst = check(g, 1.0, "inplace")
    assert float(norm) == 0.0 and not any(d.any() for d in dst)


def test_clip_max_norm_zero():
    _, _, dst = check(make([100, 20000], (BF, F32)), 0.0, "inplace")
    assert not any(d.any() for d in dst)


def test_clip_non_finite_norms():
    for bad, first in ((float("inf"), 0), (float("nan"), 1)):
        g = make([50, 20000], (F32, BF))
        g[1][777] = bad
        norm = MoEGradClip(4).clip(g, 1.0)
        if first == 0:
            assert torch.isinf(norm) and not g[0].any() and g[1][777].isnan()
            assert int(g[1].isnan().sum()) == 1
        else:
            assert norm.isnan() and all(t.isnan().all() for t in g)


def test_clip_repeats_streams_and_graph():
    g = make([5, 300000, 77], (BF, F32))
    c = MoEGradClip(8)
    o1 = [torch.empty_like(t) for t in g]
    n1 = c.clip(g, 1.0, out=o1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2 = [torch.empty_like(t) for t in g]
    with torch.cuda.stream(s):
        n2 = c.clip(g, 1.0, out=o2)
    s.synchronize()
    assert torch.equal(n1, n2) and all(torch.equal(a, b) for a, b in zip(o1, o2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n3 = c.clip(g, 1.0, out=o2)
    for _ in range(2):
        for t in o2:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n1, n3) and all(torch.equal(a, b) for a, b in zip(o1, o2))


def test_clip_tensor_past_32_bits():
    n = (1 << 31) + 4099
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[-1], g[5], g[1 << 31] = 3.0, 4.0, 12.0
    norm = MoEGradClip(1).clip([g], 6.5)
    assert float(norm) == 13.0
    assert abs(float(g[-1]) - 1.5) <= 0.01 and abs(float(g[1 << 31]) - 6.0) <= 0.04
    assert int((g != 0).sum()) == 3


def test_gradclip_single_low_bits():
    """Subnormal fp32 values of one low bit each: their squares vanish in fp32."""
    for bit in (0, 7, 15, 16, 22):
        g = torch.full((1000,), 1 << bit, dtype=torch.int32, device="cuda").view(torch.float32)
        want = 2.0 ** (bit - 149) * 1000 ** 0.5
        got = float(MoEGradClip(1).norm([g]))
        assert abs(got - want) <= 2.0 ** -149 + 2.0 ** -23 * want, (bit, got, want)


@pytest.mark.parametrize("total", [4096 * 608, 4096 * 608 + 1])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_gradclip_around_the_short_chunks(total, dtype, out):
    """Few tensors, in short chunks up to one for every CTA and in long ones above."""
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    sizes = [1, 4095, 4096, 4097, 16385]
    sizes.append(total - sum(sizes))
    gen = torch.Generator("cuda").manual_seed(total)
    g = [torch.randn(n, device="cuda", generator=gen).to(dt[dtype]) for n in sizes]
    o = [torch.empty(n, dtype=dt[out], device="cuda") for n in sizes]
    norm = float(MoEGradClip(8).clip(g, 1.0, out=o))
    want = float(sum((t.double() ** 2).sum() for t in g)) ** 0.5
    assert abs(norm - want) <= 2.0 ** -20 * want     # fp32 sums of 64, fp64 beyond
    coef = 1.0 / (want + 1e-6)
    u = torch.finfo(dt[out]).eps / 2
    for a, b in zip(o, g):
        ref = b.double() * coef
        assert ((a.double() - ref).abs() <= (u + 2.0 ** -19) * ref.abs() + 2.0 ** -25).all()
