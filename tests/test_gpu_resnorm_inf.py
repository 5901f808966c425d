"""The residual norm's backward without a norm behind the block where the block's output is infinite: its
own gradient is scale gate D, which does not depend on f."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEResidualNorm
from tests import gpu_util as G
from tests.test_gpu_resnorm import TYPES, data

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("T,H", [(4, 256), (400, 256), (400, 2048), (330, 5000), (40, 129), (4, 9000),
                                 (4, 9001)])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("pre", [False, True])
def test_infinite_output(T, H, types, gate, pre):
    d = data(T, H, *types, False, gate, pre)
    h = MoEResidualNorm(T, H, *types, post=False, gate=gate, pre=pre, scale=0.7)
    p = dict(gate=d["gate"], pre_weight=d["pre_weight"])
    out, _ = h.forward(d["x"], d["f"], **p)
    args = (d["dout"], d["dn"] if pre else None, out)
    dx, df, grads = h.backward(*args, d["f"], **p)
    f = d["f"].clone()
    f[2, 7], f[3, H - 1] = INF, -INF
    dx2, df2, grads2 = h.backward(*args, f, **p)
    assert torch.equal(dx, dx2) and torch.equal(df, df2)
    if pre:
        assert torch.equal(grads["pre_weight"], grads2["pre_weight"])
    if gate == "channel":
        a, b = grads["gate"], grads2["gate"]
        rest = torch.ones(H, dtype=torch.bool, device="cuda")
        rest[7] = rest[H - 1] = False
        assert torch.equal(a[rest], b[rest]) and torch.isinf(b[~rest]).all()
    if gate == "token":
        a, b = grads["gate"], grads2["gate"]
        rest = torch.ones(T, dtype=torch.bool, device="cuda")
        rest[2] = rest[3] = False
        assert torch.equal(a[rest], b[rest])
        if not pre:      # (with a norm in front an infinite f leaves no finite out to a forward)
            want = torch.stack([INF * dx[2, 7].sign(), -INF * dx[3, H - 1].sign()]).to(b.dtype)
            assert torch.equal(b[2:4], want)
