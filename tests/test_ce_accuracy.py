"""How far gradients may be off beside their own roundings:
rows whose target is learnt, where dZ of the target is a small difference."""
import pytest
import torch

import dense_gemm_14_gb300 as g14

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # 2^-p, p significant bits


@pytest.mark.parametrize("T", [32, 100, 129, 300])
@pytest.mark.parametrize("D", [1024, 4096, 8192])
@pytest.mark.parametrize("dtype,mode", [(torch.bfloat16, None), (torch.float16, None),
                                        (torch.float32, "3xtf32"), (torch.float32, "fp32")])
def test_gradients_of_learnt_rows(T, D, dtype, mode):
    """Rows of p_y in 0.99 .. 0.9995. dZ_y = p_y - 1 cancels: it is as good as the logits of the
    forward and the backward call are alike. With equal logits p_y is off by 1.5e-6: half an ulp
    of lse in 8 .. 16 (4.8e-7) and of its parts, and 2^-22 of an exponential in either call (2.4e-7
    each). dH of such a row is about (p_y - 1) w_y; dZ's rounding adds u of it (the other
    columns' are small beside it: half of u), the result's u."""
    g = torch.Generator(device="cuda").manual_seed(T + D)
    V = 1000
    w = (1.28 / D ** 0.5 * torch.randn(V, D, device="cuda", generator=g)).to(dtype)
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    wy = w[y].float()
    norm = wy.norm(dim=1, keepdim=True)
    lean = (11.5 + 5.0 * torch.rand(T, 1, device="cuda", generator=g)) / norm
    h = torch.randn(T, D, device="cuda", generator=g)
    h = (h - (h * wy).sum(dim=1, keepdim=True) * wy / norm ** 2 + lean * wy / norm).to(dtype)
    z = h.double() @ w.double().t()
    rows = torch.arange(T, device="cuda")
    p = torch.softmax(z, dim=1)
    rest = 1.0 - p[rows, y]
    learnt = (rest > 5e-4) & (rest < 1e-2) & (torch.logsumexp(z, dim=1) < 16)
    assert int(learnt.sum()) > T // 3
    p[rows, y] = -(p.sum(dim=1) - p[rows, y])  # without the cancellation
    up = torch.full((T,), 64.0, device="cuda")
    want = 64.0 * p @ w.double()
    lse = g14.linear_cross_entropy(h, w, y, fp32_mode=mode)[1]
    dh = g14.linear_cross_entropy_backward(h, w, y, lse, up, need_dw=False, fp32_mode=mode)[0]
    off = (dh.double() - want).norm(dim=1) / want.norm(dim=1)
    allowed = 2.5 * U[dtype] + 1.5e-6 / rest
    assert bool((off <= allowed)[learnt].all()), float((off / allowed)[learnt].max())


@pytest.mark.parametrize("dtype,V,D", [(torch.float16, 262144, 19456), (torch.bfloat16, 700000, 19456)])
def test_sums_over_a_large_vocabulary(dtype, V, D):
    """dH over a vocabulary whose sum no tile's split shortens (76 tiles, one a cluster), its
    largest term, the target's, first: every product after it is added to it, and an
    accumulator that truncates loses a little each time. As for any few rows, the result is
    its rounding off, and 10 % of that for all else (sums 1e-5 of |dZ||W|)."""
    g = torch.Generator(device="cuda").manual_seed(V)
    h = torch.randn(1, D, device="cuda", generator=g).to(dtype)
    w = torch.empty(V, D, device="cuda", dtype=dtype)
    for v in range(0, V, 16384):
        w[v:v + 16384] = 0.02 * torch.randn(min(16384, V - v), D, device="cuda", generator=g)
    y = torch.zeros(1, device="cuda", dtype=torch.int64)
    up = torch.full((1,), 64.0, device="cuda")
    z = torch.cat([h.double() @ w[v:v + 16384].double().t() for v in range(0, V, 16384)], dim=1)
    p = torch.softmax(z, dim=1)
    p[0, 0] = -p[0, 1:].sum()
    p *= 64.0
    want = sum(p[:, v:v + 16384] @ w[v:v + 16384].double() for v in range(0, V, 16384))
    lse = g14.linear_cross_entropy(h, w, y)[1]
    dh = g14.linear_cross_entropy_backward(h, w, y, lse, up, need_dw=False)[0]
    once = float((want.to(dtype).double() - want).norm())
    off = float((dh.double() - want).norm())
    assert off <= 1.1 * once + 1e-5 * float(want.norm()), (off, once)
