"""Infinite logits of the linear cross entropy's forward pass, as the header states them."""
import math

import pytest
import torch

import dense_gemm_14_gb300 as g14
from test_linear_ce import check_loss, make, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [4, 70, 300])
@pytest.mark.parametrize("dtype,mode", [("bf16", None), ("f16", None), ("f32", "fp32"), ("f32", "tf32")])
def test_infinite_logits(T, dtype, mode):
    h, w, y, up = make(T, 600, 64, dtype, T, spread=2.0)
    y[:] = torch.arange(T) % 300
    h[:, 0] = 0.0
    w[:, 0] = 0.0
    r = reference(h, w, y)
    if mode == "tf32":  # its bound, 4e-3 of |h||w|
        d = (h.double().abs() @ w.double().abs().t()).amax(dim=1)
        r["tol"] = 8e-3 * d + 1e-4
    inf = float("inf")
    # all logits of one row at +infinity, or at -infinity
    for row, sign in ((0, 1.0), (2, -1.0)):
        x, m = h.clone(), w.clone()
        m[:, 0] = 2.0
        x[row, 0] = sign * inf
        loss, lse = (v.cpu() for v in g14.linear_cross_entropy(x.cuda(), m.cuda(), y.cuda(), fp32_mode=mode))
        keep = torch.arange(T) != row
        check_loss(loss[keep], lse[keep], {k: r[k][keep] for k in ("loss", "lse", "tol")})
        assert math.isnan(loss[row])
        assert math.isnan(lse[row]) if sign > 0 else lse[row] == -inf
    # one logit of each row at -infinity, which is one row's target
    x, m = h.clone(), w.clone()
    x[:, 0] = 1.0
    m[1, 0] = -inf
    loss, lse = (v.cpu() for v in g14.linear_cross_entropy(x.cuda(), m.cuda(), y.cuda(), fp32_mode=mode))
    others = torch.arange(600) != 1
    off = y == 1
    assert bool((loss[off] == inf).all())
    yy = y - (y > 1).long()
    yy[off] = 0
    s = reference(h, w[others], yy)
    tol = r["tol"] if mode == "tf32" else s["tol"]
    assert bool(((lse.double() - s["lse"]).abs() <= tol).all())
    assert bool(((loss.double() - s["loss"]).abs() <= tol)[~off].all())
