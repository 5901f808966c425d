"""MoEResidualNorm.load_stats: which backward may follow it (no GPU needed: the library's call is replaced)."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEResidualNorm, build, resnorm

T, H = 4, 8


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture
def calls(monkeypatch):
    """The library's calls that pass the handle's checks."""
    made = []
    monkeypatch.setattr(resnorm, "_on", lambda device, fn, *args: made.append(fn))
    monkeypatch.setattr(resnorm, "_stream", lambda *args: 0)
    return made


def norm(**kw):
    return MoEResidualNorm(T, H, "fp32", device="cpu", **kw)


@pytest.mark.parametrize("with_f", [True, False])
def test_without_a_norm_behind(calls, with_f):
    """The kept norms are the same with and without a block's output, so either may follow."""
    h = norm(post=False)
    x, w = torch.zeros(T, H), torch.ones(H)
    f = x if with_f else None
    with pytest.raises(RuntimeError):
        h.backward(x, x, x, f, pre_weight=w)
    h.load_stats(rstd_out=torch.ones(T))
    dx, df, grads = h.backward(x, x, x, f, pre_weight=w)
    assert len(calls) == 1 and (df is not None) == with_f and set(grads) == {"pre_weight"}


@pytest.mark.parametrize("with_f", [True, False])
def test_with_a_norm_behind(calls, with_f):
    """rstd_f says whether there was one."""
    x, w, r = torch.zeros(T, H), torch.ones(H), torch.ones(T)
    h = norm()
    h.load_stats(r if with_f else None, r)
    h.backward(x, x, x, x if with_f else None, post_weight=w if with_f else None, pre_weight=w)
    with pytest.raises(ValueError):
        h.backward(x, x, x, None if with_f else x, post_weight=None if with_f else w, pre_weight=w)
    assert len(calls) == 1


@pytest.mark.parametrize("post", [True, False])
def test_after_a_forward(calls, post):
    """A backward without the f that the forward had is refused; a norm alone takes a backward alone."""
    x, w = torch.zeros(T, H), torch.ones(H)
    p = dict(post_weight=w if post else None, pre_weight=w)
    h = norm(post=post)
    h.forward(x, x, **p)
    h.backward(x, x, x, x, **p)
    with pytest.raises(ValueError):
        h.backward(x, x, x, pre_weight=w)
    h.forward(x, pre_weight=w)
    h.backward(x, x, x, pre_weight=w)
    assert len(calls) == 4
