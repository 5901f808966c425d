"""Three saturated sigmoids whose keys are equal in 64 bits while the difference of two of them, with the
same bias, is known beyond that: decided pair by pair each can lie above the next.  Whatever the order, the
indices are distinct and their keys the largest."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoESelect
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
F = np.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def sigmoid(x):
    return 1 / (1 + np.exp(-np.float64(x)))


@pytest.mark.parametrize("E", [3, 8, 13, 16, 32])
@pytest.mark.parametrize("T", [4, 2600])
def test_circles(E, T):
    r = np.random.default_rng(E)
    for n in range(40):
        high = F(24 + 3 * r.random())
        low = F(high - F(0.5 + r.random()))
        bias = np.zeros(E, F)
        bias[1] = F(sigmoid(high) - sigmoid(low))
        l = np.full((T, E), -3, F)
        l[:, 0], l[:, 1], l[:, 2] = np.nextafter(high, F(0)), low, high
        for k in (1, 2, 3):
            h = MoESelect(T, E, k, "sigmoid")
            idx, w = h.forward(torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda())
            idx = idx.cpu().numpy()
            assert (idx == idx[0]).all(), (n, k)
            key = sigmoid(l[0]) + bias.astype(np.float64)
            assert len(set(idx[0])) == k and set(idx[0]) <= {0, 1, 2}, (n, k, idx[0])
            best = np.sort(key)[::-1][:k]
            assert (np.abs(key[idx[0]] - best) <= 2.0 ** -51).all(), (n, k, idx[0])
