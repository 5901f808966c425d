"""The router's backward with the choice of experts refuses a gradient of the logits over what other
CTAs still read, as the choice's own backward does (no GPU needed)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_16_gb300 import binding as B
from mixture_experts_layer_16_gb300 import build

P = [(1 << 30) * (i + 1) for i in range(9)]     # aligned addresses that are never read
LOGITS, AUX, DLOGITS = 2, 5, 6
T, E = 16, 64


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


@pytest.mark.parametrize("over", [LOGITS, AUX])
@pytest.mark.parametrize("by", [0, 64, T * E * 4 - 16, 16 - T * E * 2])
def test_overlap(lib, over, by):
    shape = ctypes.byref(B.make_shape(T, 128, 64, E, 4))
    q = ctypes.byref(B.Select(T, E, 4, 2, 0, 1, 8, 2, 1, 1, 1.0))
    a = P + [None]
    a[DLOGITS] = P[over] + by
    assert lib.mm_moe_router_select_backward(shape, q, *a) == B.MM_MOE_EINVAL
    a[DLOGITS] = P[over] + T * E * 4                 # behind them
    if not torch.cuda.is_available():                # (where there is a GPU it would run)
        assert lib.mm_moe_router_select_backward(shape, q, *a) != B.MM_MOE_EINVAL
