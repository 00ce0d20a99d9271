"""Training steps of a gated feed-forward layer under a vocabulary's loss.

A step computes  y = silu(x Wg^T) * (x Wu^T),  h = y Wd^T  and the cross entropy of  h Wv^T  against the targets (the
logits are never kept), takes all gradients, clips them together, and updates the layer's matrices by their
orthogonalised gradients and the vocabulary's by its clipped one:

    python examples/gated_lm_step.py [--tokens 4096] [--hidden 1024] [--inner 2752] [--vocab 8192] [--steps 10]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_matmul_gb300 as mpg  # noqa: E402

IGNORE = -100


def product(a, b):
    """a @ b of 16-bit matrices (transposed views too), rounded once to their type."""
    c = torch.empty((a.shape[0], b.shape[1]), dtype=a.dtype, device=a.device)
    return mpg.gemm(a, b, c, mode="bf16" if a.dtype == torch.bfloat16 else "fp16")


def gradients(x, target, wg, wu, wd, wv):
    """The mean loss over the tokens that count, and the gradients of x, wg, wu, wd and wv."""
    y, *kept = mpg.gated_gemm(x, wg, wu, keep=True)
    h = product(y, wd.t())
    loss, lse = mpg.linear_cross_entropy(h, wv, target, ignore_index=IGNORE)
    share = 1.0 / (target != IGNORE).sum().clamp(min=1).float()
    dh, dwv = mpg.linear_cross_entropy_backward(h, wv, target, lse, share.expand(target.shape), ignore_index=IGNORE)
    dy = product(dh, wd)
    dwd = product(dh.t(), y)
    dx, dwg, dwu = mpg.gated_gemm_backward(dy, x, wg, wu, kept=kept)
    return loss.sum() * share, (dx, dwg, dwu, dwd, dwv)


def step(x, target, weights, masters, max_norm=1.0, rate=0.02):
    """One update of the fp32 masters of (wg, wu, wd, wv) and of their 16-bit copies; returns (loss, norm)."""
    loss, (_, *grads) = gradients(x, target, *weights)
    clipped = [torch.empty_like(m) for m in masters]
    norm = mpg.clip_grad_norm(grads, max_norm, out=clipped)
    for m, d in zip(masters[:3], clipped[:3]):
        mpg.orthogonalize(d, O=m, alpha=-rate, beta=1.0)
    masters[3].sub_(clipped[3], alpha=rate)
    for w, m in zip(weights, masters):
        w.copy_(m)
    return loss, norm


def draw(tokens, hidden, inner, vocab, seed=0, dtype=torch.bfloat16, ignored=0.1):
    """(x, target, weights, masters) of a random layer."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return scale * torch.randn(shape, generator=g, device="cuda")
    masters = [normal(inner, hidden, scale=hidden ** -0.5), normal(inner, hidden, scale=hidden ** -0.5),
               normal(hidden, inner, scale=inner ** -0.5), normal(vocab, hidden, scale=hidden ** -0.5)]
    target = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    target[torch.rand(tokens, generator=g, device="cuda") < ignored] = IGNORE
    return normal(tokens, hidden).to(dtype), target, [m.to(dtype) for m in masters], masters


def train(tokens=4096, hidden=1024, inner=2752, vocab=8192, steps=10, say=None):
    x, target, weights, masters = draw(tokens, hidden, inner, vocab)
    losses = []
    for i in range(steps):
        loss, norm = step(x, target, weights, masters)
        losses.append(float(loss))
        if say:
            say(f"step {i:3d}  loss {losses[-1]:.4f}  gradient norm {float(norm):.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 1024), ("inner", 2752), ("vocab", 8192), ("steps", 10)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    mpg.build()
    train(a.tokens, a.hidden, a.inner, a.vocab, a.steps, say=print)
