"""The handles' backward without a forward, whose results it reads, is refused (no GPU needed)."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import build, train


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_norm_backward_needs_a_forward():
    n = train.MoELayerNorm(4, 8, "fp32", device="cpu")
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(RuntimeError, match="forward first"):
        n.backward(x, x, w)
    with pytest.raises(RuntimeError, match="forward first"):
        n.backward(x, x, w, dx_add=x, out=(torch.zeros(4, 8), torch.zeros(8), torch.zeros(8)))
    with pytest.raises(ValueError):             # (arguments are looked at first)
        n.backward(x, x, w[:3])


def test_balance_backward_needs_a_forward():
    b = train.MoEBalanceLoss(16, 8, 2, device="cpu")
    lg = torch.zeros(16, 8)
    with pytest.raises(RuntimeError, match="forward first"):
        b.backward(lg, torch.zeros(2))
    with pytest.raises(RuntimeError, match="forward first"):
        b.backward(lg, torch.zeros(2), dlogits=torch.zeros(16, 8))
    with pytest.raises(ValueError):
        b.backward(lg, torch.zeros(3))
