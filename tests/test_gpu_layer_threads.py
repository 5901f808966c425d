"""Two host threads, each with a layer of its own width."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoELayer
from mixture_experts_layer_16_gb300.inputs import custom_inputs
from tests import gpu_util as G
from tests.test_gpu_threads import together

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def layer_job(H, prec):
    def make(s):
        d = custom_inputs(96, H, 128, 8, 2, seed=H)
        v = G.upload(d)
        layer = MoELayer(96, H, 128, 8, 2, prec)
        y = torch.empty((96, H), dtype=torch.bfloat16, device="cuda")
        return lambda: layer.forward(v["x"], v["topk_idx"], v["topk_w"], v["W_gate"], v["W_up"],
                                     v["W_down"], y=y, stream=s), (y,)
    return make


@pytest.mark.parametrize("prec", ["bf16", "mxfp8"])
def test_layers_of_two_widths_in_two_threads(prec):
    together([layer_job(128, prec), layer_job(4096, prec)], 2000)
