"""A few training steps of one MoE block, x + MoE(LayerNorm(x)), on synthetic data: the block's
forward with the router's balance and z losses, its backward, clipping by the global
gradient norm into fp32 gradients, and an Adam update of fp32 master weights.

    python examples/train_block.py [--tokens 4096] [--steps 20] [--prec bf16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_layer_16_gb300 import MoEBlock, MoEGradClip  # noqa: E402
from mixture_experts_layer_16_gb300.block import PARAMS  # noqa: E402


def train(T=4096, H=512, I=256, E=16, k=4, prec="bf16", steps=20, lr=3e-3, max_norm=0.5,
          balance_coef=1e-2, z_coef=1e-3, sequences=8, seed=0, log=print):
    """Returns one (mse, balance loss, z loss, gradient norm) per step."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randn((T, H), generator=gen, device="cuda").to(torch.bfloat16)
    target = x.float() + 0.3 * torch.tanh(x.float() @ torch.randn(
        (H, H), generator=gen, device="cuda") / H ** 0.5)
    seq_offsets = torch.linspace(0, T, sequences + 1, device="cuda").to(torch.int32)
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[int(seq_offsets[1]) - T // (4 * sequences):int(seq_offsets[1])] = False   # padding

    block = MoEBlock(T, H, I, E, k, prec, sequences)
    params = MoEBlock.init_params(H, I, E, seed)
    master = [params[n].float() for n in PARAMS]
    grads32 = [torch.empty_like(m) for m in master]
    moment = [(torch.zeros_like(m), torch.zeros_like(m)) for m in master]
    clip = MoEGradClip(len(PARAMS))
    dlosses = torch.tensor([balance_coef, z_coef], device="cuda")
    history = []
    for step in range(steps):
        out, losses, _ = block.forward(x, params, seq_offsets, mask)
        err = (out.float() - target) * mask[:, None]
        mse = err.square().mean()
        dout = (2.0 / T * err).to(torch.bfloat16)        # of the squared error per token
        _, grads = block.backward(dout, params, dlosses)
        norm = clip.clip([grads[n] for n in PARAMS], max_norm, out=grads32)
        for m, g, (m1, m2), name in zip(master, grads32, moment, PARAMS):
            m1.lerp_(g, 0.1)
            m2.lerp_(g.square(), 0.01)
            b1, b2 = 1 - 0.9 ** (step + 1), 1 - 0.99 ** (step + 1)
            m.sub_(lr / b1 * m1 / ((m2 / b2).sqrt() + 1e-8))
            params[name].copy_(m)
        history.append((mse, losses.clone(), norm))
    history = [(float(m), float(l[0]), float(l[1]), float(n)) for m, l, n in history]
    for step, (mse, bal, z, n) in enumerate(history):
        log(f"step {step:3d}  mse {mse:.5f}  balance {bal:.4f}  z {z:.4f}  grad norm {n:.4f}")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--prec", default="bf16")
    a = ap.parse_args()
    train(T=a.tokens, steps=a.steps, prec=a.prec)
