"""Outputs of the training-step operators laid over operands that are still read: refused by the C
ABI before anything touches a device (no GPU needed; the addresses are never read)."""
import ctypes

import pytest

from mixture_experts_layer_16_gb300 import binding as B
from mixture_experts_layer_16_gb300 import build

EI = B.MM_MOE_EINVAL
A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


# (where dx or y begins, in elements after x or dy's first; its stride; the other's stride), for 6
# rows of 8 elements
OVER = [(0, 8, 8), (8, 8, 8), (-8, 8, 8), (40, 8, 8), (-40, 8, 8), (47, 8, 8), (1, 8, 8),
        (0, 20, 20), (7, 20, 20), (13, 20, 20), (-13, 20, 20), (100, 20, 20), (93, 20, 20),
        (0, 8, 20), (0, 20, 8), (47, 20, 8), (8, 8, 20), (-47, 8, 20), (20, 32, 20)]


@pytest.mark.parametrize("at,ld,ldo", OVER)
def test_norm_overlaps_are_refused(lib, at, ld, ldo):
    s = ctypes.byref(B.NormShape(6, 8, B.MM_MOE_DT_BF16, B.MM_MOE_DT_BF16, 1e-5))
    P = [A * (i + 1) for i in range(12)]
    other = P[9] + 2 * at
    if at != 0 or ld != ldo:
        assert lib.mm_moe_norm_forward(s, P[9], ldo, P[1], P[2], other, ld, P[3], P[4], None) == EI
        assert lib.mm_moe_norm_backward(s, P[0], 8, P[1], 8, P[2], P[3], P[4], P[9], ldo, other, ld,
                                        P[5], P[6], P[7], None) == EI
    assert lib.mm_moe_norm_backward(s, P[9], ldo, P[1], 8, P[2], P[3], P[4], None, 0, other, ld,
                                    P[5], P[6], P[7], None) == EI
    assert lib.mm_moe_norm_backward(s, P[0], 8, P[9], ldo, P[2], P[3], P[4], None, 0, other, ld,
                                    P[5], P[6], P[7], None) == EI


@pytest.mark.parametrize("dtype,size", [(B.MM_MOE_DT_F32, 4), (B.MM_MOE_DT_F16, 2)])
@pytest.mark.parametrize("at", [0, 1, -1, 8, 127, -127])
def test_balance_gradient_over_the_logits_is_refused(lib, at, dtype, size):
    s = ctypes.byref(B.BalanceShape(16, 8, 2, 1, dtype))
    P = [A * (i + 1) for i in range(8)]
    assert lib.mm_moe_balance_backward(s, P[0], None, None, P[1], P[2], P[3], P[0] + size * at, P[4],
                                       None) == EI
