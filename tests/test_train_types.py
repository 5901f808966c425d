"""Gradients that are no tensors (None for a parameter without one) are named in a TypeError, as the
other handles name theirs (no GPU needed)."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import build, train


@pytest.mark.parametrize("bad", [None, 1.0, [1.0, 2.0]])
def test_clip_names_what_is_no_tensor(bad):
    build.build()
    c = train.MoEGradClip(4, device="cpu")
    g = torch.ones(4, 6)
    with pytest.raises(TypeError, match=r"grads\[1\]"):
        c.norm([g, bad])
    with pytest.raises(TypeError, match=r"grads\[0\]"):
        c.clip([bad, g], 1.0)
    with pytest.raises(TypeError, match=r"out\[1\]"):
        c.clip([g, g], 1.0, out=[g, bad])
