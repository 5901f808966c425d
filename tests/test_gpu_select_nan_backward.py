"""The gradient through the choice of experts where a token's logits are NaN, or NaN and -inf: NaN where
the weights are."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoESelect
from tests import gpu_util as G
from tests.test_gpu_select import options
from tests.test_gpu_select_nan import rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("T,E,k", [(40, 8, 2), (40, 64, 6), (300, 250, 8), (2600, 256, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward(T, E, k, score, renorm):
    """Chosen experts' gradients are NaN where their weights are; other tokens' are not touched."""
    l = rows(T, E, "fp32")
    opt = options(score, 1, 1, "max", renorm, 1.5)
    h = MoESelect(T, E, k, **opt)
    idx, w = h.forward(l)
    g = torch.ones((T, k), device="cuda") + torch.arange(k, device="cuda")
    d = h.backward(l, idx, g)
    at = d.gather(1, idx.long())
    assert torch.equal(torch.isnan(at), torch.isnan(w))
    if score == "softmax" and not renorm:
        assert torch.equal(torch.isnan(d), torch.isnan(l).any(1, keepdim=True).expand(T, E))
    else:
        assert int(torch.isnan(d).sum()) == int(torch.isnan(at).sum())
    assert not d[5].any()
