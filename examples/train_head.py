"""A training step of a small model's last two layers on the library's products.

    python examples/train_head.py [steps]

The model: h = x W1^T, then a loss over a vocabulary on the logits h W2^T. A
step forms h with gemm, keeps x in 8 bits for the backward pass (ckpt8_save)
and lets go of it, takes the loss and its gradients without ever keeping the
logits (linear_cross_entropy and its backward), and forms dW1 from the 8-bit
x (ckpt8_weight_grad). Rows with the target -100 are padding: they hold NaN
here, which reaches nothing. Random tokens' targets are learnt by plain
gradient descent; the mean loss is printed every few steps."""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_14_gb300 as g14  # noqa: E402


def train(steps: int = 30, rows: int = 600, width: int = 256, hidden: int = 320, vocab: int = 5000,
          rate: float = 2.0, seed: int = 0) -> list[float]:
    """Runs the steps on the current GPU; returns the mean loss of each."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return scale * torch.randn(*shape, device="cuda", generator=g)

    # fp32 weights are updated, 16-bit copies of them are multiplied
    w1 = normal(hidden, width, scale=1 / math.sqrt(width))
    w2 = normal(vocab, hidden, scale=1 / math.sqrt(hidden))
    x_all = normal(rows, width, scale=1.0).bfloat16()
    targets = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    targets[::7] = -100
    part = (targets != -100)
    dloss = torch.full((rows,), 1.0 / int(part.sum()), device="cuda")
    losses = []
    for _ in range(steps):
        w1h, w2h = w1.bfloat16(), w2.bfloat16()
        x = x_all
        h = g14.gemm(x, w1h.t()).bfloat16()
        h[~part] = float("nan")  # what padding rows hold does not matter
        kept = g14.ckpt8_save(x)
        del x
        loss, lse = g14.linear_cross_entropy(h, w2h, targets)
        dh, dw2 = g14.linear_cross_entropy_backward(h, w2h, targets, lse, dloss)
        dw1 = g14.ckpt8_weight_grad(dh, kept)
        w1 -= rate * dw1
        w2 -= rate * dw2.float()
        losses.append(float(loss.sum() * dloss[0]))
    if g14.check_device_error(torch.cuda.current_stream().cuda_stream):
        raise RuntimeError("a kernel recorded an error")
    return losses


if __name__ == "__main__":
    n = int(sys.argv[1]) if len(sys.argv) > 1 else 30
    for step, value in enumerate(train(n)):
        if step % 5 == 0 or step == n - 1:
            print(f"step {step:3d}  mean loss {value:.4f}")
