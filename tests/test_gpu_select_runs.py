"""The order of experts with a bias where a run of identical keys lies between the last chosen place and
a larger key that fp32 does not tell apart from them.  Against the fp64 oracle; tolerances as in
test_gpu_select.py.  The numbers of tokens go through 32, 16 and 8 lanes a token."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoESelect
from tests import gpu_util as G
from tests.test_gpu_select import check_forward, options

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def tokens(a):
    return torch.from_numpy(a.astype(np.float32)).cuda()


@pytest.mark.parametrize("T", [4, 1400, 2600])
@pytest.mark.parametrize("E,k", [(32, 1), (32, 3), (64, 8), (256, 8), (250, 6), (24, 4)])
def test_saturated_sigmoids(T, E, k):
    """Logits of 20 and a few of 20.125, all of them a sigmoid of 1 in fp32, among logits of -3."""
    r = np.random.default_rng(T + E + k)
    l = np.full((T, E), -3.0)
    for t in range(T):
        n, m = int(r.integers(3, 12)), int(r.integers(1, k + 2))
        at = r.permutation(E)[:n + m]
        l[t, at[:n]], l[t, at[n:]] = 20.0, 20.125
    l[0] = -3.0
    l[0, :3], l[0, 3] = 20.0, 20.125
    bias = torch.zeros(E, device="cuda")
    opt = options("sigmoid", 1, 1, "max", True, 1.0)
    check_forward(MoESelect(T, E, k, **opt), tokens(l), bias, opt)


@pytest.mark.parametrize("T", [4, 1400, 2600])
@pytest.mark.parametrize("E,k,groups,keep", [(32, 8, 1, 1), (256, 8, 1, 1), (32, 8, 4, 4), (64, 5, 4, 2),
                                             (250, 9, 5, 3)])
def test_masked_experts_in_front(T, E, k, groups, keep):
    """Equal biases; one expert takes nearly all, those at -25 below it lie behind masked ones in fp32."""
    r = np.random.default_rng(T + E)
    l = np.full((T, E), -25.0)
    l[:, :E // 2] = -np.inf
    l[:, E // 2 + 1] = 0.0
    for t in range(1, T):
        l[t] = l[t, r.permutation(E)]
    bias = torch.full((E,), 0.05, device="cuda")
    opt = options("softmax", groups, keep, "max", True, 1.0)
    check_forward(MoESelect(T, E, k, **opt), tokens(l), bias, opt)


@pytest.mark.parametrize("T", [4, 1400, 2600])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_copied_experts(T, score):
    """Experts copied from one another (equal logits and biases), and one whose key is larger by 1e-9."""
    E, k = 96, 6
    r = np.random.default_rng(T)
    row = r.normal(-4.0, 0.3, E).astype(np.float32)
    row[10:20], row[60] = 1.0, np.float32(1.0) + np.float32(2.0 ** -23)
    bias = np.zeros(E, np.float32)
    bias[10:20] = bias[60] = 0.25
    l = np.tile(row, (T, 1))
    l[:, 30:33] = 2.0 + 0.1 * r.random((T, 3))
    opt = options(score, 1, 1, "max", False, 1.0)
    check_forward(MoESelect(T, E, k, **opt), tokens(l), torch.from_numpy(bias).cuda(), opt)
