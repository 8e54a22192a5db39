"""The linear cross entropy where the vocabulary goes in more than one piece
(384 MiB of dZ, of logits, or of a copied W each), against the definition in
64 bits with the bounds of test_linear_ce.py. Every call gets a workspace of
exactly the bytes that the query names, with a guard behind it."""
import os
import subprocess
import sys

import pytest
import torch

import dense_gemm_14_gb300 as g14
from dense_gemm_14_gb300 import build
from test_linear_ce import DT, IGNORE, U, reference

pytestmark = pytest.mark.gpu

GUARD = 1 << 20
CODE = {"bf16": 1, "f16": 2, "fp32": 0, "tf32": 3, "3xtf32": 4}

# mode, rows, rows that take part, V, D; the pieces they make
CASES = [
    ("3xtf32", 64, 64, 39168, 2048),     # few rows, W split: 2, the last with tiles to spare
    ("3xtf32", 100, 71, 62000, 1728),    # 2
    ("bf16", 61, 50, 51500, 4097),       # few rows, W copied: 2
    ("f16", 128, 128, 95000, 2051),      # 2
    ("bf16", 5, 5, 800000, 64),          # few rows, W as it is: 2 of the backward call
    ("bf16", 4096, 4096, 100000, 72),    # 3 of the backward call
    ("f16", 1500, 1100, 270001, 40),     # 3 of the backward call
    ("f16", 300, 300, 50000, 4099),      # W copied: 2
    ("3xtf32", 300, 300, 70000, 1000),   # 2 of either
    ("3xtf32", 513, 257, 150000, 33),    # 3 of the backward call
    ("fp32", 300, 300, 400000, 24),      # the library's products: 2
    ("tf32", 300, 211, 400000, 24),
]


def make(mode, T, keep, V, D):
    dtype = mode if mode in DT else "f32"
    g = torch.Generator(device="cuda").manual_seed(T + V + D)
    h = torch.randn(T, D, device="cuda", generator=g).to(DT[dtype])
    w = (2.0 / D ** 0.5 * torch.randn(V, D, device="cuda", generator=g)).to(DT[dtype])
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    y[:3] = torch.tensor([V - 1, 0, V // 2], device="cuda")
    y[torch.randperm(T, device="cuda", generator=g)[keep:]] = IGNORE
    up = (torch.rand(T, device="cuda", generator=g) + 0.5) * (1024.0 / T if dtype == "f16" else 1.0 / T)
    with torch.device("cuda"):
        r = reference(h, w, y, up)
    h[y == IGNORE] = float("nan")
    return dtype, h, w, y, up, r


def raw(mode, backward, h, w, y, *rest):
    """One call with a workspace of the queried size, all of it but the flag words (zeros before
    a first use) holding NaN patterns, and a guard behind it."""
    (T, D), V = h.shape, w.shape[0]
    need = g14.linear_ce_workspace_bytes(CODE[mode], backward, T, V, D, h.data_ptr(), D, w.data_ptr(), D)
    assert need > 0
    ws = torch.full((need + GUARD,), 0xff, dtype=torch.uint8, device="cuda")
    ws[:min(need, 1 << 16)] = 0
    call = g14.linear_ce_backward if backward else g14.linear_ce_forward
    call(CODE[mode], T, V, D, h.data_ptr(), D, w.data_ptr(), D, y.data_ptr(), IGNORE, *rest,
         ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert g14.check_device_error(torch.cuda.current_stream().cuda_stream) == 0
    assert bool((ws[need:] == 0xff).all()), "written past the workspace"


@pytest.mark.parametrize("mode,T,keep,V,D", CASES)
def test_several_pieces(mode, T, keep, V, D):
    dtype, h, w, y, up, r = make(mode, T, keep, V, D)
    loss, lse = torch.empty(2, T, device="cuda")
    raw(mode, 0, h, w, y, loss.data_ptr(), lse.data_ptr())
    # (TF32: its bound, 4e-3 of |h||w|, in place of fp32's in the logits and each product)
    tf32 = mode == "tf32"
    hz = torch.where((y != IGNORE).unsqueeze(1), h, 0.0).double()
    d = (4e-3 if tf32 else 1e-5) * (hz.abs() @ w.double().abs().t()).amax(dim=1)
    tol = torch.where(y != IGNORE, 2 * d + 1e-4, 0.0) if tf32 else r["tol"]
    for got, want in ((loss, r["loss"]), (lse, r["lse"])):
        assert bool(((got.double() - want).abs() <= tol).all()), float(((got.double() - want).abs() - tol).max())

    dh, dw = torch.empty_like(h), torch.empty_like(w)
    raw(mode, 1, h, w, y, lse.data_ptr(), up.data_ptr(), dh.data_ptr(), D, dw.data_ptr(), D)
    u = U[dtype]
    small = (r["ref"] * 2.0 ** -40, 2.0 ** -25) if dtype == "f16" else (0.0, 1e-30)
    if tf32:
        p = (r["dz"].abs() + up.double().unsqueeze(1)) * (y != IGNORE).unsqueeze(1)
        e = p * torch.expm1(2 * d + 1e-4).unsqueeze(1) + 4e-3 * r["dz"].abs()
        e = e + 4e-3 * e
    else:
        e = r["perr"] + (u + 1e-5) * r["dz"].abs() + small[0]
    for got, want, bound in ((dh, r["dh"], e @ r["w"].abs()), (dw, r["dw"], e.t() @ r["h"].abs())):
        diff = (got.double() - want).abs()
        assert bool((diff <= bound + u * (want.abs() + bound) + small[1]).all()), float(diff.max())
    # the tensor-level calls give the same bits
    mode32 = mode if dtype == "f32" else None
    loss2, lse2 = g14.linear_cross_entropy(h, w, y, ignore_index=IGNORE, fp32_mode=mode32)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    dh2, dw2 = g14.linear_cross_entropy_backward(h, w, y, lse, up, ignore_index=IGNORE, fp32_mode=mode32)
    assert torch.equal(dh, dh2) and torch.equal(dw, dw2)


def test_several_pieces_on_the_checked_build():
    """The same on the build whose stores of statistics, dZ, slots and outputs are checked
    against their buffers: no check fails (the device status is part of the test above)."""
    if os.environ.get("GEMM14_LIB"):
        pytest.skip("this is that run")
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", __file__],
                       capture_output=True, text=True, timeout=900,
                       env=dict(os.environ, GEMM14_LIB=build.build(checked=True)))
    assert r.returncode == 0, r.stdout[-3000:]
