"""A forward of MoEBlock that ends in an error half-way leaves nothing to a backward: its operators hold
statistics, logits and routing of two different inputs by then."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEBlock
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
T, H, I, E, K = 64, 128, 64, 8, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("kw", [dict(), dict(norm="rms", gate=True, select=dict(score="sigmoid"))])
def test_backward_after_a_failed_forward(kw):
    b = MoEBlock(T, H, I, E, K, **kw)
    p = MoEBlock.init_params(H, I, E, rms="norm" in kw)
    x, y, dout = (torch.randn((T, H), device="cuda").bfloat16() for _ in range(3))
    dl = torch.tensor([0.1, 0.01], device="cuda")
    b.forward(x, p)
    want = b.backward(dout, p, dl)
    b.forward(x, p)
    with pytest.raises(ValueError):                 # behind the norm and the router
        b.forward(y, p, mask=torch.ones(T, device="cuda"))
    with pytest.raises(RuntimeError):
        b.backward(dout, p, dl)
    b.forward(x, p)
    got = b.backward(dout, p, dl)
    assert torch.equal(want[0], got[0]) and all(torch.equal(want[1][n], got[1][n]) for n in want[1])
