"""Near keys of logits that lie far apart (a small score beside a bias as large): the scores' difference is
taken where neither a sigmoid or exponential below fp32's range nor its inverse above it enters.  The
oracle's keys differ by some 2^-24 of themselves or are equal, so that 64 bits tell them apart."""
import numpy as np
import pytest
import torch

import oracle.selection as os_
from mixture_experts_layer_16_gb300 import MoESelect
from tests import gpu_util as G
from tests.test_gpu_select import options

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def check(l, bias, k, opt):
    T, E = l.shape
    idx, _ = MoESelect(T, E, k, **opt).forward(torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda())
    idx = idx.cpu().numpy()
    rows, at = np.unique(l, axis=0, return_inverse=True)     # (few different ones)
    want = os_.forward(rows, bias.astype(np.float64), k, **opt)[0][at.ravel()]
    bad = np.argwhere((idx != want).any(1))[:, 0]
    assert len(bad) == 0, (len(bad), idx[bad[0]], want[bad[0]], l[bad[0]][want[bad[0]]])


def near(score, high, low):
    """Two experts whose keys are near one another: a logit of `high` without a bias, and one of `low`
    with a bias of as many ulps around the first one's score."""
    s = os_.scores(np.array([0.0, high]), score)[1]
    return np.float32(s) * (1 + np.float32(2.0 ** -23) * np.arange(-8, 9, dtype=np.float32))


@pytest.mark.parametrize("T", [40, 1400, 2600])
@pytest.mark.parametrize("E", [6, 13, 32, 64, 256])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("high,low", [(-20.0, -90.0), (-20.0, -100.0), (-30.0, -120.0), (-10.0, -3e38),
                                      (-5.0, -np.inf)])
def test_near_keys_of_far_logits(T, E, score, high, low):
    r = np.random.default_rng(E + T)
    biases = near(score, high, low)
    for k in (1, 3):
        for b in biases[::4]:
            bias = np.full(E, -1.0, np.float32)
            l = np.full((T, E), -4.0, np.float32)
            l[:, 2] = 0.0                        # (the softmax's largest; its key is -1 and a half or less)
            bias[2] = -2.0
            bias[3] = bias[5] = 0.0
            bias[4], bias[0], bias[1] = b, 0.0, np.float32(b) * np.float32(0.75)
            for t in range(T):                   # who has the score and who the bias
                l[t, [0, 1, 3, 4, 5]] = low
                l[t, r.integers(3, 6)] = high
            check(l, bias, k, options(score, 1, 1, "max", True, 1.0))


@pytest.mark.parametrize("T", [40, 2600])
@pytest.mark.parametrize("E", [3, 6, 16, 32])
def test_small_biases_beside_small_scores(T, E):
    """Biases of 0 and 1e-9 beside logits of -3 to -90: indices are distinct and in order."""
    r = np.random.default_rng(T + E)
    v = np.array([17.5, -3.0, -20.0, -20.5, -90.0, -91.0], np.float32)
    for k in range(1, min(E, 5)):
        l = v[r.integers(0, len(v), (T, E))]
        bias = np.array([0.0, 1e-9], np.float32)[r.integers(0, 2, E)]
        check(l, bias, k, options("sigmoid", 1, 1, "max", True, 1.0))
