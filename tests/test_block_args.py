"""Refusals of MoEBlock before anything touches a device (no GPU needed)."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEBlock, build

T, H, I, E, K = 16, 128, 64, 8, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("kw", [dict(), dict(norm="rms"), dict(norm="rms", gate=True, first=False)])
def test_dnext_without_a_next_norm(kw):
    """A block that gives no `next` takes no gradient of it: refused, not dropped."""
    b = MoEBlock(T, H, I, E, K, device="cpu", **kw)
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dnext"):
        b.backward(x, {}, torch.zeros(2), dnext=x)
    with pytest.raises(RuntimeError):
        b.backward(x, {}, torch.zeros(2))
