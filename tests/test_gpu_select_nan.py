"""The choice of experts where a token's logits are NaN, or NaN and -inf: a NaN ranks as -inf, and is not lost
on the way to the weights (a NaN among the chosen; with a softmax that is not renormalised, or has a bias,
any of the row)."""
import numpy as np
import pytest
import torch

import oracle.selection as os_
from mixture_experts_layer_16_gb300 import MoESelect
from tests import gpu_util as G
from tests.test_gpu_select import bias_of, f64, logits_of, options

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def rows(T, E, dtype):
    l = logits_of(T, E, dtype)
    l[1] = NAN
    l[2], l[2, E // 2:] = -INF, NAN
    l[3], l[3, 0] = NAN, -INF
    l[4, E - 1] = NAN
    l[5] = -INF                      # nothing to choose from, and no NaN
    l[6, ::2] = NAN
    l[T - 1] = NAN
    return l


SHAPES = [(40, 8, 2, 1, 1), (40, 13, 4, 1, 1), (40, 64, 6, 1, 1), (40, 64, 6, 8, 3), (1400, 64, 6, 1, 1),
          (2600, 64, 6, 8, 3), (2600, 256, 8, 1, 1), (300, 250, 8, 5, 2)]


@pytest.mark.parametrize("T,E,k,groups,keep", SHAPES)
@pytest.mark.parametrize("score,dtype", [("softmax", "fp32"), ("softmax", "bf16"), ("sigmoid", "fp32")])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_bias", [False, True])
def test_forward(T, E, k, groups, keep, score, dtype, renorm, with_bias):
    l = rows(T, E, dtype)
    bias = bias_of(E, score) if with_bias else None
    for gsc in ("max", "top2") if groups > 1 else ("max",):
        opt = options(score, groups, keep, gsc, renorm, 1.5)
        idx, w = MoESelect(T, E, k, dtype=dtype, **opt).forward(l, bias)
        L, i, w = f64(l), idx.cpu().numpy(), f64(w)
        with np.errstate(invalid="ignore"):
            for t in (0, 1, 2, 3, 4, 5, 6, T - 2, T - 1):
                # without a bias the logits rank
                rank = np.where(np.isnan(L[t]), -np.inf, L[t]) if bias is None else L[t]
                want = os_.choose(rank, None if bias is None else f64(bias), k, score, groups, keep, gsc)
                assert np.array_equal(i[t], want), (t, i[t], want)
                chosen = np.isnan(L[t][i[t]])
                if score == "softmax" and (with_bias or not renorm):
                    nan = np.full(k, np.isnan(L[t]).any())
                else:
                    nan = np.full(k, chosen.any()) if renorm else chosen
                assert np.array_equal(np.isnan(w[t]), nan), (t, w[t], nan)
        if score == "softmax":
            assert not w[5].any()
