"""Trains a small MoE block to reproduce the output of another one: norm, router, experts, balance
loss, clipping and AdamW together.

    python -m mixture_experts_layer_14_gb300.train_block [--dtype mxfp8] [--states mxfp8] [--steps N]
"""

import argparse

import torch

from . import MOK_BF16, MOK_MXFP8, AdamW, MoEBlock, dims, grad_norm
from .synthetic import LayerShape, make_layer


def train(steps=40, dtype="bf16", states="f32", T=512, d=256, E=8, k=2, F=256, lr=2e-3, device="cuda",
          report=None):
    """Trains a block to reproduce another one's output; the mean squared errors, step by step."""
    code = {"bf16": MOK_BF16, "mxfp8": MOK_MXFP8}[dtype]
    D = dims(T, d, E, k, F, F, 1, code)
    shape = LayerShape("block", T, d, E, k, F, F, 1, 0.0, "none", dtype, True, 31)
    target, W = (make_layer(shape, device, seed_base=c) for c in (31, 32))
    x, norm = W.pop("x"), torch.ones(d, dtype=torch.float32, device=device)
    target["norm"], W["norm"] = norm, norm.clone()
    residual = target["x"].float()
    want = MoEBlock(D, target).forward(x, residual)[0].float()
    block = MoEBlock(D, W, alpha=1e-2, z_coef=1e-4)
    names, params = block.parameters()
    opt = AdamW(params, weight_decay=[0.0 if n == "norm" else 0.01 for n in names], states=states)
    errors = []
    for step in range(steps):
        y, _ = block.forward(x, residual, training=True)
        diff = y.float() - want
        errors.append(diff.square().mean())
        g = block.gradients(block.backward((diff * (2.0 / diff.numel())).to(torch.bfloat16)))
        clip = grad_norm(g, 1.0)
        opt.step(g, lr, clip=clip)
        block.requantise()
        if report is not None:
            report(step, float(errors[-1]), float(block.aux["loss"][0]), float(clip[0]))
    return torch.stack(errors).tolist()


def main():
    ap = argparse.ArgumentParser(description="Trains one small MoE block.")
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--dtype", choices=("bf16", "mxfp8"), default="bf16")
    ap.add_argument("--states", choices=("f32", "mxfp8"), default="f32")
    a = ap.parse_args()
    train(a.steps, a.dtype, a.states, report=lambda s, e, b, n: print(
        f"step {s:3d}  error {e:.5f}  balance loss {b:.5f}  gradient norm {n:.4f}"))


if __name__ == "__main__":
    main()
