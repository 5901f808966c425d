"""Pins of the fp64 oracle of the training-step operators (oracle/train.py): torch's own
modules in fp64, brute force, central finite differences, closed-form cases, and planted
mistakes that the pins must catch."""
import numpy as np
import pytest
import torch

import oracle.train as ot


def _diff(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def _norm_case(T, H, seed):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, H)) * r.uniform(0.1, 5.0, H) + r.standard_normal(H),
            1 + 0.2 * r.standard_normal(H), r.standard_normal(H), r.standard_normal((T, H)))


@pytest.mark.parametrize("T,H", [(1, 1), (3, 2), (5, 17), (4, 128)])
def test_norm_against_autograd(T, H):
    x, w, b, dy = _norm_case(T, H, T * H)
    tx, tw, tb = (torch.tensor(a, requires_grad=True) for a in (x, w, b))
    y = torch.nn.functional.layer_norm(tx, (H,), tw, tb, 1e-5)
    y.backward(torch.tensor(dy))
    f = ot.norm_forward(x, w, b, 1e-5)
    g = ot.norm_backward(dy, x, w, 1e-5)
    assert np.allclose(f["y"], y.detach().numpy(), rtol=1e-11, atol=1e-12)
    # the terms of dx cancel: at H = 1 exactly, else relative to rstd |g|
    scale = f["rstd"].max() * np.abs(dy * w).max()
    assert np.abs(g["dx"] - tx.grad.numpy()).max() <= 1e-11 * scale
    assert np.allclose(g["dweight"], tw.grad.numpy(), rtol=1e-10, atol=1e-10)
    assert np.allclose(g["dbias"], tb.grad.numpy(), rtol=1e-11, atol=1e-12)


def test_norm_against_differences():
    x, w, b, dy = _norm_case(6, 33, 5)
    r = np.random.default_rng(6)
    g = ot.norm_backward(dy, x, w, 1e-5)
    L = lambda x_, w_, b_: float((ot.norm_forward(x_, w_, b_, 1e-5)["y"] * dy).sum())
    for arg, name, val in ((0, "dx", x), (1, "dweight", w), (2, "dbias", b)):
        v = r.standard_normal(val.shape)
        args = [x, w, b]

        def f(z):
            a = list(args)
            a[arg] = z
            return L(*a)
        assert np.isclose(_diff(f, val, v), (g[name] * v).sum(), rtol=1e-7, atol=1e-7)


def _balance_case(T, E, k, G, seed):
    r = np.random.default_rng(seed)
    logits = 2 * r.standard_normal((T, E))
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    off = np.concatenate([[0], np.sort(r.integers(0, T + 1, G - 1)), [T]])
    if G > 2:
        off[G // 2] = off[G // 2 - 1]         # a sequence without a token
    mask = r.random(T) < 0.8
    return logits, idx, off, mask


def test_balance_even_load_is_one():
    # uniform logits and an even routing: f = 1 for every expert, P = 1/E
    T, E, k = 24, 8, 2
    idx = (np.arange(T * k).reshape(T, k)) % E
    f = ot.balance_forward(np.zeros((T, E)), idx)
    assert np.isclose(f["losses"][0], 1.0) and np.isclose(f["losses"][1], np.log(E) ** 2)
    # every token on one expert that takes all the probability: E
    logits = np.full((T, E), -40.0)
    logits[:, 3] = 40.0
    f = ot.balance_forward(logits, np.full((T, 1), 3))
    assert np.isclose(f["losses"][0], E)


@pytest.mark.parametrize("T,E,k,G", [(12, 4, 1, 1), (30, 8, 2, 4), (25, 5, 3, 7)])
def test_balance_against_autograd_and_differences(T, E, k, G):
    logits, idx, off, mask = _balance_case(T, E, k, G, T)
    f = ot.balance_forward(logits, idx, G, off, mask)
    dl = np.array([0.7, -0.3])
    d = ot.balance_backward(logits, idx, dl, G, off, mask)
    t = torch.tensor(logits, requires_grad=True)
    p, ls = torch.softmax(t, 1), torch.logsumexp(t, 1)
    bal, live, n_all, zs = 0.0, 0, 0, 0.0
    for s in range(G):
        rows = [i for i in range(off[s], off[s + 1]) if mask[i]]
        if not rows:
            assert f["tokens"][s] == 0 and not f["counts"][s].any()
            continue
        cnt = np.bincount(idx[rows].reshape(-1), minlength=E)
        assert np.array_equal(cnt, f["counts"][s])
        live += 1
        n_all += len(rows)
        bal = bal + (torch.tensor(cnt * E / (k * len(rows))) * p[rows].mean(0)).sum()
        zs = zs + (ls[rows] ** 2).sum()
    loss = dl[0] * bal / live + dl[1] * zs / n_all
    assert np.isclose(float(loss.detach()), dl @ f["losses"], rtol=1e-12)
    loss.backward()
    assert np.allclose(d, t.grad.numpy(), rtol=1e-10, atol=1e-13)
    v = np.random.default_rng(1).standard_normal(logits.shape)
    num = _diff(lambda z: dl @ ot.balance_forward(z, idx, G, off, mask)["losses"], logits, v)
    assert np.isclose(num, (d * v).sum(), rtol=1e-6, atol=1e-9)
    assert not d[~mask].any()


def test_balance_rows_left_out():
    logits, idx, _, _ = _balance_case(10, 4, 2, 1, 3)
    logits[4] = -np.inf                       # nothing left by its mask
    logits[5, 1:] = -np.inf                   # one expert left
    f = ot.balance_forward(logits, idx)
    assert f["tokens"][0] == 9 and f["lse"][4] == 0.0 and np.isclose(f["lse"][5], logits[5, 0])
    f = ot.balance_forward(logits, idx, mask=np.zeros(10, bool))
    assert not f["losses"].any() and not f["counts"].any()


def test_clip():
    r = np.random.default_rng(0)
    gs = [r.standard_normal(n) for n in (5, 0, 300)]
    n, out = ot.grad_clip(gs, 1.0)
    assert np.isclose(n, np.linalg.norm(np.concatenate(gs)))
    assert np.isclose(np.linalg.norm(np.concatenate(out)), n / (n + 1e-6))
    n2, same = ot.grad_clip(gs, 2 * n)
    assert n2 == n and all(np.array_equal(a, b) for a, b in zip(gs, same))
    assert ot.grad_norm([]) == 0.0 and ot.grad_norm([np.array([3e30, 4e30])]) == 5e30


def test_planted_mistakes_fail_the_pins(monkeypatch):
    def caught(fn, *a):
        try:
            fn(*a)
        except AssertionError:
            return True
        return False

    good_b, good_f, good_bb = ot.norm_backward, ot.balance_forward, ot.balance_backward

    def no_xh_term(dy, x, weight, eps, dx_add=None):
        o = good_b(dy, x, weight, eps, dx_add)
        f = ot.norm_forward(x, weight, None, eps)
        g = np.asarray(dy) * weight
        o["dx"] = f["rstd"][:, None] * (g - g.mean(1, keepdims=True))
        return o

    monkeypatch.setattr(ot, "norm_backward", no_xh_term)
    assert caught(test_norm_against_autograd, 5, 17) and caught(test_norm_against_differences)
    monkeypatch.setattr(ot, "norm_backward", good_b)

    def mean_over_all(logits, idx, G=1, off=None, mask=None):
        o = good_f(logits, idx, G, off, mask)
        o["losses"] = o["losses"] * np.array([max((o["tokens"] > 0).sum(), 1) / G, 1.0])
        return o

    monkeypatch.setattr(ot, "balance_forward", mean_over_all)
    assert caught(test_balance_against_autograd_and_differences, 25, 5, 3, 7)
    monkeypatch.setattr(ot, "balance_forward", good_f)

    def no_jacobian(logits, idx, dl, G=1, off=None, mask=None):
        return good_bb(logits, idx, dl, G, off, mask) + 1e-4

    monkeypatch.setattr(ot, "balance_backward", no_jacobian)
    assert caught(test_balance_against_autograd_and_differences, 12, 4, 1, 1)
