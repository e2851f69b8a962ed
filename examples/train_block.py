"""A small network of a convolution, a gated feed-forward block and a linear
head, trained for some steps and then asked row by row: the library's operators
as a program uses them together.

    python examples/train_block.py [--steps 30] [--dtype bf16]

A convolution (its weights stay) turns 8 x 8 images into 64 positions of
`width` features; each position goes through the block, with its residual, and
the head predicts `targets` numbers for it.  Every step is forward, backward,
clipping by the global gradient norm, and a plain gradient step on float32
master weights.  At the end the block's answer for single rows is compared with
its answer for all rows.  Prints the loss."""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import implicit_gemm_cnn_gb300 as conv  # noqa: E402

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def train(steps=30, dtype="bf16", images=16, width=128, hidden=320, targets=24, rate=0.2, max_norm=0.5, seed=0):
    """(losses, gradient norms, the largest difference between rows alone and together)"""
    dt = DTYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    pixels = normal(images, 8, 8, 8).to(dt)
    stem = normal(width, 8, 3, 3, scale=72 ** -0.5).to(dt)
    master = {"gate": normal(hidden, width, scale=width ** -0.5), "up": normal(hidden, width, scale=width ** -0.5),
              "down": normal(width, hidden, scale=hidden ** -0.5), "head": normal(targets, width, scale=width ** -0.5),
              "bias": torch.zeros(targets, device="cuda")}
    want = normal(images * 64, targets)
    # the convolution's [n][channel][position] as [n * position][channel] rows
    rows = conv.conv2d(pixels, stem, pads=1, act="silu").flatten(2).transpose(1, 2).reshape(-1, width).contiguous()
    losses, norms = [], []
    for _ in range(steps):
        w = {k: v.to(dt) for k, v in master.items()}
        mid, saved = conv.gated_ffn(rows, w["gate"], w["up"], w["down"], residual=rows, save=True)
        out = conv.linear(mid, w["head"], w["bias"])
        off = out.float() - want
        losses.append(off.square().mean())
        dout = (off * (2.0 / off.shape[0])).to(dt)  # of the squares' sum per row
        dmid, dhead, dbias, _ = conv.linear_backward(dout, mid, w["head"], need_dbias=True)
        _, dgate, dup, ddown = conv.gated_ffn_backward(dmid, rows, w["gate"], w["up"], w["down"], saved)
        grads = [dgate, dup, ddown, dhead, dbias]
        norms.append(conv.clip_grad_norm(grads, max_norm))
        for v, d in zip(master.values(), grads):
            v.sub_(d.float(), alpha=rate)
    # an answer for one row at a time
    w = {k: v.to(dt) for k, v in master.items()}
    together = conv.gated_ffn(rows, w["gate"], w["up"], w["down"], residual=rows)
    alone = torch.cat([conv.gated_ffn(rows[i:i + 1], w["gate"], w["up"], w["down"], residual=rows[i:i + 1])
                       for i in range(8)])
    apart = (alone.float() - together[:8].float()).abs().max().item()
    return [v.item() for v in losses], [v.item() for v in norms], apart


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    a.add_argument("--steps", type=int, default=30)
    a.add_argument("--dtype", choices=sorted(DTYPES), default="bf16")
    a = a.parse_args()
    losses, norms, apart = train(a.steps, a.dtype)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}  gradient norm {norms[i]:.3f}")
    print(f"last loss {losses[-1]:.4f}; rows alone and together differ by at most {apart:.3g}")
