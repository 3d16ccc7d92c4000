"""Train one MoE layer's experts on one GPU to follow another layer's.

    python examples/train_experts.py [--precision bf16|mxfp8] [--state-bits 32|8] [--steps 60]

Token rows are grouped by expert; a step is forward, backward over
micro-batches (bf16: gradients added up in float32; mxfp8: one batch, bf16
gradients), the gradients' global norm and the AdamW step, which writes the
bf16 weights that the next forward multiplies (bf16) or quantizes (mxfp8).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp8_block_scaled_04_amd as mx  # noqa: E402
from mxfp8_block_scaled_04_amd.bf16_layer import Bf16Layer  # noqa: E402
from mxfp8_block_scaled_04_amd.moe_layer import MoELayer  # noqa: E402
from mxfp8_block_scaled_04_amd.optimizer import AdamW  # noqa: E402


def weights(G, H, I, seed, device):
    gen = torch.Generator(device=device).manual_seed(seed)
    w1 = torch.randn((G, 2 * I, H), generator=gen, device=device) * H ** -0.5
    w2 = torch.randn((G, H, I), generator=gen, device=device) * I ** -0.5
    return mx.swiglu_interleave(w1).bfloat16().contiguous(), w2.bfloat16()


def train(precision="bf16", state_bits=32, steps=60, sizes=(300, 0, 84, 640), H=256, I=256, lr=3e-3, micro=2, seed=0,
          device="cuda", report=None):
    """Returns the loss (mean squared error) before every step."""
    G, M = len(sizes), sum(sizes)
    offsets = torch.tensor([sum(sizes[:g]) for g in range(G + 1)], dtype=torch.int32, device=device)
    gen = torch.Generator(device=device).manual_seed(seed)
    xs = [torch.randn((M, H), generator=gen, device=device).bfloat16() for _ in range(micro)]
    T1, T2 = weights(G, H, I, seed + 1, device)
    teacher = Bf16Layer(offsets, M, H, I, device)
    targets = [teacher.forward(x, T1, T2).clone() for x in xs]

    W1, W2 = weights(G, H, I, seed + 2, device)
    if precision == "bf16":
        layer = Bf16Layer(offsets, M, H, I, device, fp32_grads=True)
    else:
        layer, xs, targets = MoELayer(offsets, M, H, I, device), xs[:1], targets[:1]
    optimizer = AdamW([W1, W2], [layer.dW1, layer.dW2], lr=lr, weight_decay=0.01, state_bits=state_bits, max_norm=1.0)
    losses = []
    for step in range(steps):
        loss = 0.0
        if precision != "bf16":
            layer.quantize_weights(W1, W2)
        for k, (x, target) in enumerate(zip(xs, targets)):
            y = layer.forward(x, W1, W2) if precision == "bf16" else layer.forward(x)
            error = y.float() - target.float()
            loss += float(error.square().mean()) / len(xs)
            dY = (error * (2.0 / (error.numel() * len(xs)))).bfloat16()
            if precision == "bf16":
                layer.backward(x, dY, W1, W2, accumulate=k > 0)
            else:
                layer.backward(dY)
        optimizer.step()
        losses.append(loss)
        if report is not None and (step % 10 == 0 or step == steps - 1):
            report(f"step {step:3d}  loss {loss:.5f}  gradient norm {float(optimizer.norm[0]):.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--precision", choices=("bf16", "mxfp8"), default="bf16")
    ap.add_argument("--state-bits", type=int, choices=(32, 8), default=32)
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    train(a.precision, a.state_bits, a.steps, report=print)
