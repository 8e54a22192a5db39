"""A training step of a small language model whose output projection is its
embedding table, on the library's products.

    python examples/train_tied.py [steps]

The model: e = scale * W[tokens], h = e W1^T, and a loss over the vocabulary on the
logits h W^T, with the same W. A step looks the tokens up (embedding), keeps e in 8
bits for the backward pass (ckpt8_save), forms h (gemm), takes the loss and its
gradients without ever keeping the logits (linear_cross_entropy and its backward),
forms dW1 from the 8-bit e (ckpt8_weight_grad) and de = dh W1 (gemm), adds the
lookup's share to the projection's gradient of W (embedding_backward with beta = 1),
and scales both gradients so that their norm stays within a limit
(clip_grad_norm), all without waiting for the GPU. Places with the token or the
target -100 are padding. Random text is learnt by plain gradient descent; the mean
loss and the norm are printed every few steps."""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_14_gb300 as g14  # noqa: E402


def gradients(w: torch.Tensor, w1: torch.Tensor, tokens: torch.Tensor, targets: torch.Tensor,
              scale: float, fp32_mode: str | None = None, keep8: bool = True):
    """(loss per place, dw, dw1) of the mean loss: w (V, D) and w1 (D, D) in one
    dtype, tokens and targets vectors. keep8: the weight gradient from e in 8 bits,
    else from e itself."""
    targets = torch.where(tokens == -100, -100, targets)
    part = (targets != -100).sum().clamp(min=1)
    e = g14.embedding(w, tokens, scale=scale)
    kept = g14.ckpt8_save(e) if keep8 else None
    mode = fp32_mode if w.dtype == torch.float32 else None
    h = g14.gemm(e, w1.t(), fp32_mode=mode).to(w.dtype)
    loss, lse = g14.linear_cross_entropy(h, w, targets, fp32_mode=fp32_mode)
    dloss = torch.ones(tokens.numel(), device=w.device) / part
    dh, dw = g14.linear_cross_entropy_backward(h, w, targets, lse, dloss, fp32_mode=fp32_mode)
    dw1 = g14.ckpt8_weight_grad(dh, kept, fp32_mode=fp32_mode) if keep8 else \
        g14.gemm(dh.t(), e, fp32_mode=mode)
    de = g14.gemm(dh, w1, fp32_mode=mode).to(w.dtype)
    g14.embedding_backward(de, tokens, out=dw, scale=scale, beta=1.0)
    return loss, dw, dw1


def train(steps: int = 30, rows: int = 600, width: int = 256, vocab: int = 5000, rate: float = 0.5,
          limit: float = 1.0, seed: int = 0) -> list[tuple[float, float]]:
    """Runs the steps on the current GPU; returns the mean loss and the norm of each."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    # fp32 weights are updated, 16-bit copies of them are multiplied
    w = torch.randn(vocab, width, device="cuda", generator=g) / math.sqrt(width)
    w1 = torch.randn(width, width, device="cuda", generator=g) / math.sqrt(width)
    text = torch.randint(0, vocab, (rows + 1,), device="cuda", generator=g)
    tokens, targets = text[:-1].clone(), text[1:].clone()
    targets[::7] = -100
    tokens[-5:] = -100
    # fp32 gradients, clipped from the 16-bit ones; the lists are kept with them
    dw32, dw132 = torch.empty_like(w), torch.empty_like(w1)
    clipped = g14.GradList([dw32, dw132])
    out = []
    for _ in range(steps):
        loss, dw, dw1 = gradients(w.bfloat16(), w1.bfloat16(), tokens, targets, math.sqrt(width))
        norm = g14.clip_grad_norm([dw, dw1], limit, out=clipped)
        w -= rate * dw32
        w1 -= rate * dw132
        out.append((loss, norm))
    if g14.check_device_error(torch.cuda.current_stream().cuda_stream):
        raise RuntimeError("a kernel recorded an error")
    part = int(((tokens != -100) & (targets != -100)).sum())
    return [(float(loss.sum()) / part, float(norm)) for loss, norm in out]


if __name__ == "__main__":
    n = int(sys.argv[1]) if len(sys.argv) > 1 else 30
    for step, (value, size) in enumerate(train(n)):
        if step % 5 == 0 or step == n - 1:
            print(f"step {step:3d}  mean loss {value:.4f}  gradient norm {size:.3f}")
