"""MoELayerNorm at the ends of its range of rows: the most that its shape admits (2^31 - 1), and
few rows of fp32 around what a single CTA takes in the backward."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoELayerNorm
from mixture_experts_layer_16_gb300 import binding as B
from tests import gpu_util as G
from tests.test_gpu_norm import go

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


@pytest.mark.parametrize("T", [(1 << 31) - 200, (1 << 31) - 1])
def test_norm_most_rows(T):
    """One column: mean = x, y = bias, rstd = eps^-1/2, dx = dx_add, dweight = 0, dbias = sum dy (a
    few powers of two: exact in any order)."""
    eps, at = 2.0 ** -16, torch.tensor([0, 5, 1 << 30, T // 3, T - 2, T - 1], device="cuda")
    x = torch.empty((T, 1), dtype=BF, device="cuda").random_(0, 200)
    w, b = (torch.full((1,), v, dtype=BF, device="cuda") for v in (1.5, -0.75))
    n = MoELayerNorm(T, 1, eps=eps)
    for t in (n.mean, n.rstd):
        t.fill_(-1.0)
    y = n.forward(x, w, b, y=torch.full_like(x, 9.0))
    for a in range(0, T, 1 << 28):
        e = min(T, a + (1 << 28))
        assert torch.equal(n.mean[a:e], x[a:e, 0].float())
        assert bool(((n.rstd[a:e] - 256.0).abs() <= 2.0 ** -14).all())   # (2 ulp)
        assert bool((y[a:e] == -0.75).all())
    dy = torch.zeros_like(x)
    dy[at, 0] = torch.tensor([1, 2, 4, 8, 16, 32], dtype=BF, device="cuda")
    dx, dw, db = n.backward(dy, x, w, dx_add=x, out=(y, torch.empty_like(w), torch.empty_like(b)))
    assert float(dw) == 0.0 and float(db) == 63.0
    for a in range(0, T, 1 << 28):
        assert torch.equal(dx[a:a + (1 << 28)], x[a:a + (1 << 28)])


@pytest.mark.parametrize("H", [1024, 1000, 515, 2048, 260])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 8, 9, 15, 16, 17, 32, 33])
def test_norm_backward_few_fp32_rows(T, H):
    go(T, H, "fp32", "fp32", bias=T % 2 == 0, add=T % 3 == 0)


@pytest.mark.parametrize("H,most", [(1024, 8), (512, 16), (2048, 4)])
def test_norm_backward_launches_of_few_fp32_rows(H, most):
    """One launch for up to two rows for each group of a single CTA in two units a thread, two
    above."""
    for T in (most, most + 1, 2 * most, 2 * most + 1):
        n = MoELayerNorm(T, H, "fp32")
        x, w = torch.randn((T, H), device="cuda"), torch.ones(H, device="cuda")
        n.forward(x, w, w)
        B.mm_moe_profile_start()
        n.backward(x, x, w)
        k = B.mm_moe_profile_stop()
        assert k["norm_bwd"][1] == 1 and k["norm_bwd_finish"][1] == (T > most), (T, k)
