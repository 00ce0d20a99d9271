"""Training steps of one linear layer with 8-bit products and an orthogonalised update.

A step quantises the activations, the weights and the output's gradient to 8 bits (each in both directions from
one read), makes the three products of the layer from them, lets the weight gradient's product accumulate the
momentum (beta = momentum, fp32), and folds the orthogonalised momentum into the weights (alpha = -rate,
beta = 1 - rate * decay):

    python examples/fp8_muon_step.py [--tokens 4096] [--inputs 2048] [--outputs 1024] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_matmul_gb300 as mpg  # noqa: E402


def forward(x, w):
    """y = x W^T and what the backward pass needs of it."""
    xq, xs, xqt, xst = mpg.fp8_quantize(x, transpose=True)
    wq, ws, wqt, wst = mpg.fp8_quantize(w, block="tile", transpose=True)
    return mpg.gemm_fp8(xq, xs, wq, ws), (xqt, xst, wqt, wst)


def backward(dy, saved, momentum, mu, need_dx=True):
    """The input's gradient, and momentum <- mu * momentum + dy^T x."""
    xqt, xst, wqt, wst = saved
    # gradients differ in size from token to token: e5m2's range, a scale for each block of a token
    dq, ds, dqt, dst = mpg.fp8_quantize(dy, fmt="e5m2", transpose=True)
    dx = mpg.gemm_fp8(dq, ds, wqt, wst) if need_dx else None
    mpg.gemm_fp8(dqt, dst, xqt, xst, C=momentum, beta=mu)
    return dx


def update(w, momentum, rate, decay):
    """W <- (1 - rate * decay) W - rate * scale * NS(momentum); the scale gives the update of a wide or tall matrix
    the root mean square of a square one's."""
    scale = max(1.0, w.shape[0] / w.shape[1]) ** 0.5
    mpg.orthogonalize(momentum, O=w, alpha=-rate * scale, beta=1.0 - rate * decay)


def train(tokens=4096, inputs=2048, outputs=1024, steps=20, rate=0.03, mu=0.9, decay=0.01, seed=0, say=None):
    """Fits a random linear map; returns the losses."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    teacher = torch.randn((outputs, inputs), generator=g, device=dev) / inputs ** 0.5
    w = torch.zeros((outputs, inputs), device=dev)
    momentum = torch.zeros_like(w)
    losses = []
    for i in range(steps):
        x = torch.randn((tokens, inputs), generator=g, device=dev)
        target = x @ teacher.t()
        y, saved = forward(x.bfloat16(), w)
        diff = y.float() - target
        losses.append(float(diff.square().mean()))
        backward((diff * (2.0 / diff.numel())).bfloat16(), saved, momentum, mu, need_dx=False)
        update(w, momentum, rate, decay)
        if say:
            say(f"step {i:3d}  loss {losses[-1]:.5f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("inputs", 2048), ("outputs", 1024), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    mpg.build()
    train(a.tokens, a.inputs, a.outputs, a.steps, say=print)
