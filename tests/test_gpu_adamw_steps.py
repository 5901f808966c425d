"""MoEAdamW.steps and set_step beside a step that has not run yet: both wait for the device, whichever stream
the step is on."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEAdamW
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("states", ["fp32", "8bit"])
def test_a_step_on_another_stream(states):
    p, g = [torch.randn(1000, device="cuda")], [torch.randn(1000, device="cuda")]
    o = MoEAdamW(p, states=states)
    o.step(p, g, 1e-3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def later():
        with torch.cuda.stream(s):
            torch.cuda._sleep(200_000_000)       # about 0.1 s
        o.step(p, g, 1e-3, stream=s)
    later()
    assert o.steps() == 2
    later()
    o.set_step(7)
    assert o.steps() == 7
    o.step(p, g, 1e-3)
    assert o.steps() == 8
