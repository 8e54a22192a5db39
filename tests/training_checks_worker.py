"""Runs training products on whichever library GEMM14_LIB names and writes
their outputs and device status (tests/test_training_checks.py runs it on the
build with device-side bounds checks):

    python training_checks_worker.py OUT.npz
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

# T, V, D, dtype, rows that take part
CE = [(1, 700, 72, "bf16", 1), (61, 1031, 136, "f16", 50), (128, 512, 64, "bf16", 128),
      (300, 700, 129, "bf16", 300), (700, 600, 80, "f16", 257), (300, 513, 37, "f32", 200),
      (2100, 20000, 320, "bf16", 1500)]
# T, N, K, dtype, beta, output pad: split tiles, whole ones, half-width ones
WGRAD = [(1, 64, 96, "bf16", 1.0, 0), (200, 600, 1001, "f16", 1.0, 3), (4096, 300, 520, "bf16", 0.0, 0),
         (2048, 256, 256, "f32", 1.0, 1), (1500, 5000, 4600, "bf16", 1.0, 4)]


def run_all():
    out = []
    for T, V, D, dtype, keep in CE:
        g = torch.Generator().manual_seed(T + V)
        h = torch.randn(T, D, generator=g).to(DT[dtype]).cuda()
        w = (torch.randn(V, D, generator=g) / D ** 0.5).to(DT[dtype]).cuda()
        y = torch.randint(0, V, (T,), generator=g)
        y[torch.randperm(T, generator=g)[keep:]] = -100
        y = y.cuda()
        up = torch.full((T,), 1.0, device="cuda")
        mode = "3xtf32" if dtype == "f32" else None
        loss, lse = g14.linear_cross_entropy(h, w, y, fp32_mode=mode)
        dh, dw = g14.linear_cross_entropy_backward(h, w, y, lse, up, fp32_mode=mode)
        out += [loss, lse, dh, dw]
    for T, N, K, dtype, beta, pad in WGRAD:
        g = torch.Generator().manual_seed(T + N)
        c = g14.ckpt8_save(torch.randn(T, K, generator=g).to(DT[dtype]).cuda())
        dy = torch.randn(T, N, generator=g).to(DT[dtype]).cuda()
        dw = torch.ones(N, K + pad, device="cuda")
        g14.ckpt8_weight_grad(dy, c, out=dw[:, :K], beta=beta,
                              fp32_mode="3xtf32" if dtype == "f32" else None)
        out.append(dw)
    status = g14.check_device_error(torch.cuda.current_stream().cuda_stream)
    return [x.float().cpu().numpy() for x in out], status


if __name__ == "__main__":
    arrays, status = run_all()
    np.savez(sys.argv[1], lib=g14.lib_path(), status=status,
             **{f"a{i}": a for i, a in enumerate(arrays)})
