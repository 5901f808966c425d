"""MoESelect on the GPU against the fp64 oracle.

The indices are equal: the oracle ranks by the keys in 64 bits.  Bounds of the weights, e = 2^-24:
expf is within 2 ulp (4 e), the sigmoid with a sum and an approximate division (2 ulp) within 10 e of
itself; the softmax's exponent l - m is exact to e |l - m| (logits up to 40 in size here: 80 e), its
sum of E terms within (E / 32 + 8) e; a sum of k weights and two more operations (k + 4) e: together
below (128 + E / 32 + k) e of each weight, and as much again for the gradient's differences, relative
to the sum of its terms' sizes.  Gradients are rounded to their type (u: half an ulp).
"""
import itertools

import numpy as np
import pytest
import torch

import oracle.selection as os_
from mixture_experts_layer_16_gb300 import MoEBalanceLoss, MoERouter, MoESelect
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {n: torch.finfo(t).eps / 2 for n, t in DT.items()}
SUB = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
E24 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def f64(t):
    return t.double().cpu().numpy()


def logits_of(T, E, dtype, seed=0, size=1.5):
    r = np.random.default_rng(1000 * seed + 7 * T + E)
    l = size * r.standard_normal((T, E)) - 0.5 * np.log1p(np.arange(E))[r.permutation(E)]
    return torch.from_numpy(l.astype(np.float32)).cuda().to(DT[dtype])


def bias_of(E, score, seed=0):
    r = np.random.default_rng(seed + E)
    size = 0.1 if score == "sigmoid" else 0.5 / E
    return torch.from_numpy((size * r.standard_normal(E)).astype(np.float32)).cuda()


def wtol(E, k):
    return (128 + E / 32 + k) * E24


def check_forward(h, l, bias, opt):
    idx, w = h.forward(l, bias)
    ri, rw = os_.forward(f64(l), None if bias is None else f64(bias), h.k, **opt)
    got = idx.cpu().numpy()
    assert np.array_equal(got, ri), np.argwhere(got != ri)[:5]
    bad = ~(np.abs(f64(w) - rw) <= wtol(h.E, h.k) * np.abs(rw) + 1e-37)
    assert not bad.any(), (np.argwhere(bad)[:5], f64(w)[bad][:5], rw[bad][:5])
    return idx, w


def options(score, groups, topk_groups, group_score, renormalise, scale):
    return dict(score=score, groups=groups, topk_groups=topk_groups, group_score=group_score,
                renormalise=renormalise, scale=scale)


@pytest.mark.parametrize("T,E,k,groups,keep", [
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (5, 7, 3, 1, 1), (64, 8, 2, 1, 1), (33, 60, 4, 1, 1),
    (100, 128, 8, 1, 1), (17, 128, 8, 8, 2), (65, 160, 6, 8, 3), (70, 256, 8, 8, 4),
    (70, 256, 9, 8, 4), (41, 384, 8, 1, 1), (9, 512, 32, 4, 2), (7, 1024, 32, 32, 5),
    (6, 1023, 31, 3, 1), (5, 1020, 16, 17, 3), (50, 24, 2, 12, 1), (50, 8, 3, 8, 5), (20, 96, 8, 3, 2),
    (30, 31, 31, 31, 31), (12, 1000, 10, 20, 20)])
@pytest.mark.parametrize("score,dtype", [("softmax", "fp32"), ("sigmoid", "fp32"),
                                         ("softmax", "bf16"), ("sigmoid", "fp16")])
def test_forward(T, E, k, groups, keep, score, dtype):
    for n, (gsc, renorm, with_bias) in enumerate((("max", True, False), ("top2", False, True),
                                                  ("top2", True, False), ("max", False, True))):
        opt = options(score, groups, keep, gsc, renorm, 2.5 if renorm else 1.0)
        h = MoESelect(T, E, k, dtype=dtype, **opt)
        check_forward(h, logits_of(T, E, dtype, n), bias_of(E, score, n) if with_bias else None,
                      opt)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,keep,gsc", [(1, 1, "max"), (8, 3, "max"), (8, 3, "top2")])
def test_ties(score, with_bias, groups, keep, gsc):
    """Few different logits: equal keys go to the lower index."""
    T, E, k = 200, 128, 8
    opt = options(score, groups, keep, gsc, True, 1.0)
    r = np.random.default_rng(5)
    bias = torch.from_numpy(r.integers(0, 2, E).astype(np.float32) / 64).cuda() if with_bias \
        else None
    for values in (1, 2, 3, 10):
        l = torch.from_numpy(r.integers(0, values, (T, E)).astype(np.float32)).cuda()
        for dtype in ("fp32", "bf16"):
            h = MoESelect(T, E, k, dtype=dtype, **opt)
            if groups > 1 and gsc == "top2":
                check_groups(h, l.to(DT[dtype]), bias, opt)
            else:
                check_forward(h, l.to(DT[dtype]), bias, opt)


def check_groups(h, l, bias, opt):
    """Sums of two scores may be equal without their terms being so: (s1 + b) + s2 = s1 + (s2 + b).
    As numbers they tie, in 64 bits each way of adding them up has its own roundings: an exponential
    and a quotient (2^-52 each at most), two sums, of numbers below 2: less than 2^-50 apart.  So the
    kept groups are any whose scores lie within 2^-50 of the best ones', and the experts are those that
    the definition takes from these groups."""
    idx = h.forward(l, bias)[0].cpu().numpy()
    L, b = f64(l), None if bias is None else f64(bias)
    G, n = opt["groups"], opt["topk_groups"]
    for t in range(h.T):
        g = os_.group_scores(L[t], b, opt["score"], G, opt["group_score"])
        least = np.sort(g)[-n]
        sure = [i for i in range(G) if g[i] > least + 2.0 ** -50]
        rest = [i for i in range(G) if abs(g[i] - least) <= 2.0 ** -50]
        args = (L[t], b, h.k, opt["score"], G, n, opt["group_score"])
        assert any(np.array_equal(idx[t], os_.choose(*args, best=[*sure, *some]))
                   for some in itertools.combinations(rest, n - len(sure))), t


@pytest.mark.parametrize("score,gap", [("sigmoid", 1e-9), ("sigmoid", 1e-8), ("sigmoid", 3e-7),
                                       ("softmax", 1e-10), ("softmax", 1e-9)])
def test_keys_too_close_for_32_bits(score, gap):
    """Biases chosen so that score + bias differs by about `gap` from expert to expert."""
    T, E, k = 96, 64, 8
    r = np.random.default_rng(9)
    l = r.standard_normal(E).astype(np.float32)
    s = os_.scores(l.astype(np.float64), score)
    bias = (0.7 - s + gap * r.permutation(E)).astype(np.float32)
    # (the fp32 bias's own rounding keeps keys apart by far less than 32 bits of a key show)
    L = np.tile(l, (T, 1))
    L[T // 2:] = np.roll(L[T // 2:], 1, axis=1)
    for groups, keep in ((1, 1), (8, 2)):
        opt = options(score, groups, keep, "top2", True, 1.0)
        check_forward(MoESelect(T, E, k, **opt), torch.from_numpy(L).cuda(),
                      torch.from_numpy(bias).cuda(), opt)


def test_close_logits_without_a_bias():
    """Neighbouring fp32 values: the bits given to the place in a lane do not decide."""
    T, E, k = 300, 256, 8
    r = np.random.default_rng(2)
    base = np.float32(1.7).view(np.int32)
    l = (base + r.integers(0, 40, (T, E))).astype(np.int32).view(np.float32)
    l[::2] *= -1
    for groups, keep, gsc in ((1, 1, "max"), (8, 3, "max"), (8, 3, "top2")):
        opt = options("sigmoid", groups, keep, gsc, True, 1.0)
        ri, _ = os_.forward(l, None, k, **opt)
        idx, _ = MoESelect(T, E, k, **opt).forward(torch.from_numpy(l).cuda())
        if gsc == "top2":   # (sums of scores that agree to 1e-16: any of the closest groups)
            s = 1 / (1 + np.exp(-l.astype(np.float64)))
            two = -np.sort(-s.reshape(T, 8, 32), axis=2)[:, :, :2]
            g = two.sum(2)
            kept = np.zeros((T, 8), bool)
            np.put_along_axis(kept, idx.cpu().numpy() // 32, True, 1)
            least = np.where(kept, g, np.inf).min(1)
            third = -np.sort(-g, axis=1)[:, 2]
            assert (least >= third - 1e-15).all()
        else:
            assert np.array_equal(idx.cpu().numpy(), ri)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep,gsc", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2")])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(score, groups, keep, gsc, with_bias):
    """Logits of -inf and of the type's lowest value: last in rank, weight zero."""
    T, E, k = 64, 32, 4
    l = logits_of(T, E, "fp32", 3)
    l[:, ::3] = -float("inf")
    l[::4, 1::3] = torch.finfo(torch.float32).min
    l[5] = -float("inf")
    l[6, 3:] = -float("inf")
    l[7, :8] = -float("inf")          # a whole group
    l[8] = torch.finfo(torch.float32).min
    bias = bias_of(E, score) if with_bias else None
    for renorm in (True, False):
        opt = options(score, groups, keep, gsc, renorm, 1.0)
        idx, w = check_forward(MoESelect(T, E, k, **opt), l, bias, opt)
        assert not w[5].any() if score == "softmax" or renorm else True


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 3)])
def test_not_finite(with_bias, groups, keep):
    """Whatever the logits hold, the indices are distinct and in range, and other tokens' are right."""
    T, E, k = 40, 64, 6
    l = logits_of(T, E, "fp32")
    good = l.clone()
    l[1, 5] = float("nan")
    l[3, ::2] = float("nan")
    l[5] = float("nan")
    l[7, 9] = float("inf")
    l[9, ::5] = float("inf")
    bad = [1, 3, 5, 7, 9]
    bias = bias_of(E, "sigmoid") if with_bias else None
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            opt = options(score, groups, keep, "top2", renorm, 1.0)
            h = MoESelect(T, E, k, **opt)
            idx, w = h.forward(l, bias)
            i = idx.cpu().numpy()
            assert ((i >= 0) & (i < E)).all()
            assert all(len(set(row)) == k for row in i)
            gi, gw = h.forward(good, bias)
            rest = [t for t in range(T) if t not in bad]
            assert torch.equal(idx[rest], gi[rest]) and torch.equal(w[rest], gw[rest])
            if score == "sigmoid":       # an infinite logit is a score of one, a NaN is passed over
                assert 9 in i[7] and torch.isfinite(w[7]).all() and 5 not in i[1]
                assert set(i[9]) <= set(range(0, E, 5)) or groups > 1


def check_backward(T, E, k, opt, dtype, grad, aux, idx=None, seed=0):
    l = logits_of(T, E, dtype, seed)
    h = MoESelect(T, E, k, dtype=dtype, grad_dtype=grad, **opt)
    if idx is None:
        idx = h.forward(l, None)[0]
    r = np.random.default_rng(T + E)
    g = torch.from_numpy(r.standard_normal((T, k)).astype(np.float32)).cuda()
    x = torch.from_numpy(r.standard_normal((T, E)).astype(np.float32)).cuda() if aux else None
    got = h.backward(l, idx, g, dlogits_aux=x)
    assert got.dtype == DT[grad or dtype]
    o = dict(score=opt["score"], renormalise=opt["renormalise"], scale=opt["scale"])
    i = idx.cpu().numpy()
    want = os_.backward(f64(l), i, f64(g), **o)
    # the terms' sizes: the formula with every sign the same
    ag = np.abs(f64(g))
    size = np.zeros((T, E))
    for t in range(T):
        e = np.array([v for v in i[t] if 0 <= v < E], int)
        a = ag[t][[0 <= v < E for v in i[t]]]
        lt = f64(l)[t]
        if len(e) == 0:
            continue
        if o["renormalise"]:
            s = os_.scores(lt, o["score"])[e] if o["score"] == "sigmoid" else \
                os_.weights(lt, e, "softmax", True, 1.0)
            n = s.sum()
            np.add.at(size[t], e, (a + a @ s / n) * s / n)
        else:
            s = os_.scores(lt, o["score"])
            np.add.at(size[t], e, a * s[e])
            if o["score"] == "softmax":
                size[t] += s * (a @ s[e])
    size *= abs(o["scale"])
    if aux:
        want = want + f64(x)
        size += np.abs(f64(x))
    n = grad or dtype
    tol = 2 * wtol(E, k) * size + U[n] * np.abs(want) + SUB[n] + 1e-37
    bad = ~(np.abs(f64(got) - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], f64(got)[bad][:4], want[bad][:4])
    return h, l, idx, g


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 7, 3), (64, 8, 2), (33, 60, 4), (100, 128, 8),
                                   (41, 256, 8), (9, 512, 32), (5, 1020, 16), (300, 36, 6)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward(T, E, k, score, renorm):
    opt = options(score, 1, 1, "max", renorm, 2.5 if renorm else 1.0)
    for n, (dtype, grad) in enumerate((("fp32", None), ("fp32", "bf16"), ("bf16", None),
                                       ("fp16", None), ("fp16", "bf16"))):
        check_backward(T, E, k, opt, dtype, grad, aux=n % 2 == 1, seed=n)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_repeated_and_dropped_indices(score, renorm):
    T, E, k = 50, 40, 6
    r = np.random.default_rng(4)
    i = r.integers(0, E, (T, k))
    i[::3, 2] = i[::3, 0]
    i[1::3, 1:] = i[1::3, :1]
    i[5, 3], i[6, 0], i[7, :], i[8, 2] = -1, E, -7, 2 ** 31 - 1
    idx = torch.from_numpy(i.astype(np.int32)).cuda()
    check_backward(T, E, k, options(score, 1, 1, "max", renorm, 1.5), "fp32", None, True, idx)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """The oracle's gradient against central differences of its weights (fp64), at a fixed choice."""
    r = np.random.default_rng(1)
    l, g = r.standard_normal((3, 12)), r.standard_normal((3, 4))
    idx, _ = os_.forward(l, None, 4, score)
    d = os_.backward(l, idx, g, score, renorm, 1.7)

    def loss(x):
        return sum((os_.weights(x[t], idx[t], score, renorm, 1.7) * g[t]).sum() for t in range(3))
    for t in range(3):
        for e in range(12):
            h = np.zeros_like(l)
            h[t, e] = 1e-6
            assert abs((loss(l + h) - loss(l - h)) / 2e-6 - d[t, e]) < 1e-8


@pytest.mark.parametrize("T,E,k,groups,keep,gsc,score,dtype,renorm,with_bias", [
    (20011, 256, 8, 8, 4, "top2", "sigmoid", "fp32", True, True),
    (20011, 256, 8, 1, 1, "max", "softmax", "fp32", True, False),
    (20000, 256, 8, 1, 1, "max", "softmax", "bf16", False, True),
    (10001, 250, 6, 5, 2, "top2", "softmax", "fp32", True, True),
    (19999, 128, 8, 1, 1, "max", "softmax", "fp32", True, False),
    (12345, 128, 8, 8, 2, "max", "sigmoid", "fp16", True, True),
    (12345, 100, 7, 4, 3, "top2", "sigmoid", "fp32", False, False),
    (20000, 64, 4, 8, 4, "top2", "sigmoid", "fp32", True, True),
    (11111, 60, 6, 1, 1, "max", "sigmoid", "fp32", True, True),
    (30000, 32, 4, 4, 2, "max", "softmax", "bf16", True, False),
    (30001, 16, 4, 1, 1, "max", "softmax", "fp32", False, True),
    (40000, 8, 2, 1, 1, "max", "softmax", "fp32", True, False),
    (40001, 7, 7, 1, 1, "max", "sigmoid", "fp32", True, True),
    (40000, 12, 3, 4, 2, "top2", "sigmoid", "fp32", True, True),
    (10007, 256, 12, 16, 8, "top2", "sigmoid", "fp32", True, True),
    (10007, 128, 16, 1, 1, "max", "softmax", "fp32", True, True),
    (6000, 512, 8, 8, 3, "top2", "sigmoid", "fp32", True, True),
    (6001, 500, 10, 1, 1, "max", "softmax", "bf16", True, False),
    (5000, 1024, 8, 16, 4, "top2", "sigmoid", "fp32", True, True),
    (10007, 256, 8, 8, 3, "max", "sigmoid", "fp32", True, True)])
def test_many_tokens(T, E, k, groups, keep, gsc, score, dtype, renorm, with_bias):
    """As test_forward where the tokens fill the SMs, with fewer lanes a token."""
    opt = options(score, groups, keep, gsc, renorm, 1.5)
    h = MoESelect(T, E, k, dtype=dtype, **opt)
    l = logits_of(T, E, dtype, 1)
    l[5] = -float("inf")
    l[6, ::2] = -float("inf")
    l[7] = 0.25                                     # all alike
    l[8, : E // 2] = 1.0
    l[9, 3:] = float("nan")
    bias = bias_of(E, score) if with_bias else None
    if not with_bias and dtype == "fp32" and gsc != "top2":   # neighbouring values
        v = np.float32(0.7).view(np.int32) + np.random.default_rng(0).integers(0, 9, (50, E))
        l[100:150] = torch.from_numpy(v.astype(np.int32).view(np.float32)).cuda()
    idx, w = h.forward(l, bias)
    i, w = idx.cpu().numpy(), f64(w)
    assert ((i >= 0) & (i < E)).all() and len(set(i[9])) == k
    L, b = f64(l), None if bias is None else f64(bias)
    ok = [t for t in range(T) if t not in (9,)]
    ri, rw = os_.forward(L[ok], b, k, **opt)
    tied = groups > keep and gsc == "top2"          # (rows 5 to 8: sums that tie, see check_groups)
    keep_rows = np.array([not (tied and t in (5, 6, 7, 8)) for t in ok])
    bad = np.argwhere((i[ok] != ri).any(1) & keep_rows)[:, 0]
    assert len(bad) == 0, (len(bad), ok[bad[0]], i[ok][bad[0]], ri[bad[0]])
    off = (np.abs(w[ok] - rw) > wtol(E, k) * np.abs(rw) + 1e-37) & keep_rows[:, None]
    assert not off.any(), np.argwhere(off)[:5]


def test_near_keys_of_many_tokens():
    """Biases that bring score + bias together to 1e-8 and less, in one row in ten."""
    T, E, k = 20000, 256, 8
    r = np.random.default_rng(3)
    l = r.standard_normal((T, E)).astype(np.float32)
    s = os_.scores(l[0].astype(np.float64), "sigmoid")
    bias = (0.7 - s + np.where(np.arange(E) % 3 == 0, 1e-8, 1e-3) * r.permutation(E)).astype(np.float32)
    l[::10] = l[0]
    for groups, keep in ((1, 1), (8, 4)):
        opt = options("sigmoid", groups, keep, "top2", True, 1.0)
        h = MoESelect(T, E, k, **opt)
        idx = h.forward(torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda())[0].cpu().numpy()
        rows = np.concatenate([[0], np.arange(1, 2000)])
        ri, _ = os_.forward(l[rows], bias.astype(np.float64), k, **opt)
        assert np.array_equal(idx[rows], ri)
        assert (idx[::10] == idx[0]).all()


def test_rows_on_no_vector_boundary():
    """Logits and gradients whose storage begins between two vectors."""
    T, E, k = 33, 128, 8
    for dtype in ("fp32", "bf16"):
        l = logits_of(T, E, dtype)
        wide = torch.empty(T * E + 1, dtype=DT[dtype], device="cuda")
        odd = wide[1:].view(T, E)
        odd.copy_(l)
        opt = options("sigmoid", 8, 4, "top2", True, 1.0)
        h = MoESelect(T, E, k, dtype=dtype, **opt)
        a, b = h.forward(l), h.forward(odd)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        g = torch.randn((T, k), device="cuda")
        o = torch.empty(T * E + 1, dtype=DT[dtype], device="cuda")[1:].view(T, E)
        assert torch.equal(h.backward(l, a[0], g), h.backward(odd, a[0], g, dlogits=o))


def test_past_32_bit_offsets():
    T, E, k = (1 << 22) + 1000, 1024, 8
    l = torch.full((T, E), -1.0, dtype=torch.bfloat16, device="cuda")
    want = torch.tensor([1000, 3, 77, 512, 13, 1023, 0, 256], device="cuda")
    up = torch.tensor([9.0, 8.0, 7.0, 6.0, 5.0, 4.0, 3.0, 2.0], device="cuda").bfloat16()
    l[:, want] = up
    h = MoESelect(T, E, k, "sigmoid", dtype="bf16")
    idx, w = h.forward(l)
    assert bool((idx == want.int()).all())
    g = torch.randn((T, k), device="cuda")
    d = h.backward(l, idx, g)
    assert not d[:, 1:3].any()
    part = MoESelect(1000, E, k, "sigmoid", dtype="bf16")
    assert torch.equal(d[-1000:], part.backward(l[-1000:], idx[-1000:], g[-1000:]))


@pytest.mark.parametrize("opt", [
    dict(score="sigmoid", groups=4, topk_groups=2, group_score="top2", scale=2.5),
    dict(score="softmax", renormalise=False)])
def test_router(opt):
    """MoERouter with these options: its logits, the choice from them, and the same gradients as the
    plain router's products give for that logit gradient."""
    T, H, E, k = 300, 256, 32, 4
    gen = torch.Generator(device="cuda")
    gen.manual_seed(0)
    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    W = (0.1 * torch.randn((E, H), generator=gen, device="cuda")).bfloat16()
    bias = bias_of(E, opt["score"])
    r = MoERouter(T, H, E, k, select=opt)
    idx, w = r.forward(x, W, bias=bias)
    plain = MoERouter(T, H, E, k)
    plain.forward(x, W)
    assert torch.equal(plain.logits, r.logits)
    h = MoESelect(T, E, k, grad_dtype="bf16", **opt)
    i2, w2 = h.forward(r.logits, bias)
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    ri, _ = os_.forward(f64(r.logits), f64(bias), k, **{**options("softmax", 1, 1, "max", True, 1.0),
                                                      **opt})
    assert np.array_equal(idx.cpu().numpy(), ri)
    loss = MoEBalanceLoss(T, E, k)
    loss.forward(r.logits, idx)
    aux = loss.backward(r.logits, torch.tensor([0.1, 0.01], device="cuda"))
    g = torch.randn((T, k), generator=gen, device="cuda")
    for a in (None, aux):
        dx = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
        dx0 = f64(dx)
        dW = r.backward(x, W, idx, w, g, dx, dlogits_aux=a)
        dl = h.backward(r.logits, idx, g, dlogits_aux=a)
        assert torch.equal(dl, r.dlogits)
        d = f64(dl)
        want = d.T @ f64(x)
        # a product of T terms in fp32 and one rounding to bf16
        assert (np.abs(f64(dW) - want) <= 2 ** -8 * np.abs(want) +
                T * E24 * (np.abs(d).T @ np.abs(f64(x)))).all()
        want = dx0 + d @ f64(W)
        assert (np.abs(f64(dx) - want) <= 2 ** -8 * np.abs(want) + E24 * E * (
            np.abs(dx0) + np.abs(d) @ np.abs(f64(W)))).all()
    with pytest.raises(ValueError):
        plain.forward(x, W, bias=bias)


def test_captured_and_repeated():
    T, E, k = 1000, 256, 8
    l = logits_of(T, E, "fp32")
    h = MoESelect(T, E, k, "sigmoid", 8, 4, "top2")
    b = bias_of(E, "sigmoid")
    g = torch.randn((T, k), device="cuda")

    def go(s=None):
        idx, w = h.forward(l, b, stream=s)
        return [idx, w, h.backward(l, idx, g, stream=s)]
    want = [t.clone() for t in go()]
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


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(8, 2), (8, 8), (5, 3), (16, 4), (13, 13)])
def test_near_keys_of_few_experts(score, E, k):
    """Keys 1e-3 to 1e-10 apart, several together, in every other row; equal ones and -inf as well."""
    T = 4000
    r = np.random.default_rng(E + k)
    l = r.standard_normal((T, E)).astype(np.float32)
    l[::2] = l[0]
    l[3], l[5, ::2], l[7] = 0.5, -np.inf, -np.inf
    s = os_.scores(l[0].astype(np.float64), score)
    for gap in (1e-3, 1e-6, 1e-8, 1e-10):
        bias = (0.7 - s + gap * r.permutation(E)).astype(np.float32)
        bias[0] = bias[1] = bias[0]
        h = MoESelect(T, E, k, score)
        idx = h.forward(torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda())[0].cpu().numpy()
        ri, _ = os_.forward(l, bias.astype(np.float64), k, score)
        bad = np.argwhere((idx != ri).any(1))[:, 0]
        assert len(bad) == 0, (gap, len(bad), idx[bad[0]], ri[bad[0]])


@pytest.mark.parametrize("with_bias", [False, True])
def test_more_candidates_than_there_is_room_for(with_bias):
    """Few kept lanes and a large k leave no bound below the k-th key, and rows of equal keys none
    that helps: the whole row is ranked."""
    for T, E, k, groups, keep in ((20, 1024, 32, 32, 12), (33, 512, 20, 1, 1), (12000, 256, 8, 1, 1),
                                  (12000, 256, 8, 8, 4)):
        opt = options("sigmoid", groups, keep, "max", True, 1.0)
        l = logits_of(T, E, "fp32", 2)
        l[1::2] = 0.5
        l[3, E // 2:] = 0.25
        bias = None
        if with_bias:
            bias = bias_of(E, "sigmoid")
            bias[E // 4:] = 0.125
        rows = slice(0, 400)
        h = MoESelect(T, E, k, **opt)
        idx, w = h.forward(l, bias)
        ri, _ = os_.forward(f64(l[rows]), None if bias is None else f64(bias), k, **opt)
        assert np.array_equal(idx[rows].cpu().numpy(), ri)
        assert torch.equal(idx[5::2], idx[5].expand_as(idx[5::2]))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_renormalised_expert(score):
    """Its weight is `scale` whatever the logits are (but for the sigmoid's 1e-20 beside the sum): the gradient is
    zero, not what is left of two equal terms."""
    T, E = 700, 96
    l = logits_of(T, E, "fp32")
    h = MoESelect(T, E, 1, score, scale=2.5)
    idx, w = h.forward(l)
    assert (w == 2.5).all()
    assert not h.backward(l, idx, torch.randn((T, 1), device="cuda")).any()
