"""MoEGradClip on both sides of its changes of chunk length and list: up to 32 tensors of at most
4096 * 152 elements together in short chunks (one for every SM), more elements or tensors in
long ones.

Bounds as in test_gpu_gradclip.py: 40 e of the norm, an element's half ulp plus 48 e, e = 2^-24;
half the smallest subnormal step where the output type has fewer bits."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEGradClip
from tests import gpu_util as G
from tests.test_gpu_gradclip import E32, SUB, U

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def check(sizes, dtype, out):
    gen = torch.Generator("cuda").manual_seed(len(sizes) + sum(sizes))
    g = [torch.randn(n, device="cuda", generator=gen).to(DT[dtype]) for n in sizes]
    want = float(sum((t.double() ** 2).sum() for t in g)) ** 0.5
    clip = MoEGradClip(64)
    norm = clip.norm(g)
    o = [torch.full((n,), 9.0, dtype=DT[out], device="cuda") for n in sizes]
    assert torch.equal(clip.clip(g, 0.5, out=o), norm)
    assert abs(float(norm) - want) <= 40 * E32 * want
    coef = 0.5 / (want + 1e-6)
    for a, b in zip(o, g):
        ref = b.double() * coef
        assert ((a.double() - ref).abs() <= (U[DT[out]] + 48 * E32) * ref.abs() + SUB[DT[out]]).all()
    if out == dtype:
        clip.clip(g, 0.5)
        assert all(torch.equal(a, b) for a, b in zip(g, o))


@pytest.mark.parametrize("total", [4096 * 152 - 1, 4096 * 152, 4096 * 152 + 1, 4096 * 153])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32")])
def test_gradclip_at_the_last_short_chunk(total, dtype, out):
    sizes = [1, 4095, 4096, 4097, 16385]
    check(sizes + [total - sum(sizes)], dtype, out)
    check([total], dtype, out)


@pytest.mark.parametrize("n", [31, 32, 33])
@pytest.mark.parametrize("last", [1, 4096, 4096 * 152])
def test_gradclip_at_the_longest_short_list(n, last):
    check([1 + 37 * i % 5000 for i in range(n - 1)] + [last], "bf16", "bf16")
    check([4096] * (n - 1) + [last], "fp32", "fp32")
