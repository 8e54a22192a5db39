"""Runs lookups, their gradients, norms and clipping on whichever library GEMM14_LIB
names and writes their outputs and device status (tests/test_step_checks.py runs it on
the build with device-side bounds checks):

    python step_checks_worker.py OUT.npz
"""
import os
import sys

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import dense_gemm_14_gb300 as g14  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# T, V, D, dtype, dtype of the gradient, beta: few tokens, ranked, sorted by 8 and by 16 SMs, rows at any address
CASES = [(1, 700, 72, "bf16", "bf16", 0.0), (300, 61, 129, "f16", "f32", 1.0), (1000, 1031, 1032, "bf16", "bf16", 0.5),
         (3000, 300, 264, "f32", "f32", 1.0), (8192, 40, 1024, "bf16", "f32", 0.0), (12000, 50021, 200, "f16", "f16", 1.0),
         (30000, 5000, 136, "bf16", "f32", 1.0), (9000, 17, 65, "bf16", "bf16", 1.0)]


def run_all():
    out = []
    for T, V, D, dtype, to, beta in CASES:
        g = torch.Generator().manual_seed(T + V)
        dy = torch.randn(T, D, generator=g).to(DT[dtype]).cuda()
        tokens = (torch.rand(T, generator=g) ** 4 * V).long()
        tokens[torch.randperm(T, generator=g)[:T // 8]] = -100
        tokens = tokens.cuda()
        dw = torch.randn(V, D, generator=g).to(DT[to]).cuda()
        out.append(g14.embedding_backward(dy, tokens, out=dw, scale=0.5, beta=beta))
        out.append(g14.embedding(dw, tokens, scale=2.0, dtype=DT[dtype]))
    norm, each = g14.grad_norm(out, each=True)
    clipped = [torch.empty_like(x, dtype=torch.float32) for x in out]
    out += [norm, each, g14.clip_grad_norm(out, 1.0, out=clipped), *clipped]
    status = g14.check_device_error(torch.cuda.current_stream().cuda_stream)
    return [x.float().cpu().numpy() for x in out], status


if __name__ == "__main__":
    arrays, status = run_all()
    np.savez(sys.argv[1], lib=g14.lib_path(), status=status,
             **{f"a{i}": a for i, a in enumerate(arrays)})
