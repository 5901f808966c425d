"""Groups whose two largest keys are the two infinities: their sum, a NaN, ranks as -inf, and no more groups
than are kept take part."""
import numpy as np
import pytest
import torch

import oracle.selection as os_
from mixture_experts_layer_16_gb300 import MoESelect
from tests import gpu_util as G
from tests.test_gpu_select import f64, logits_of, options

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("T", [20, 1400, 2600])
@pytest.mark.parametrize("E,k,groups,keep", [(64, 6, 8, 2), (32, 4, 16, 3), (256, 8, 8, 4), (100, 5, 5, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinite_biases(T, E, k, groups, keep, score):
    n = E // groups
    l = logits_of(T, E, "fp32")
    bias = torch.zeros(E, device="cuda")
    for g in (1, groups - 1):                  # everything in it forbidden but one expert, which is forced
        bias[g * n:(g + 1) * n] = -INF
        bias[g * n + n // 2] = INF
    bias[2 * n:2 * n + n // 2] = -INF
    opt = options(score, groups, keep, "top2", True, 1.0)
    idx = MoESelect(T, E, k, **opt).forward(l, bias)[0].cpu().numpy()
    L, b = f64(l), f64(bias)
    with np.errstate(invalid="ignore"):
        for t in range(0, T, max(1, T // 50)):
            want = os_.choose(L[t], b, k, score, groups, keep, "top2")
            assert np.array_equal(idx[t], want), (t, idx[t], want)
