"""A whole step of a model whose output projection is its embedding table
(examples/train_tied.py): lookup, products, linear cross entropy, the gradients of
both uses of the table in one matrix, their norm and clipping.

The gradients in fp32 are held to the formulas in 64 bits. Each product is within
1e-5 of the product of its operands' magnitudes (the library's fp32 bound), and each
later stage carries the error of the one before it; the bounds are worked out from
the magnitudes below (`bounds`). They are also held to differences of the loss in 64
bits along random directions, within the same bounds summed along the direction
(central differences of a step of 1e-4: their own error, of the order of 1e-8 of the
slope's scale, is covered by 1e-6 of it)."""
import math
import os
import sys

import numpy as np
import pytest
import torch

import dense_gemm_14_gb300 as g14

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

E, U = 1e-5, 2.0 ** -24


def model(T=150, V=97, D=40, seed=3):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(V, D, generator=g) / math.sqrt(D)
    w1 = torch.randn(D, D, generator=g) / math.sqrt(D)
    tokens = torch.randint(0, V, (T,), generator=g)
    tokens[T // 3:T // 2] = 11  # one token at many places
    targets = torch.randint(0, V, (T,), generator=g)
    targets[::6], tokens[5], tokens[-1] = -100, -100, -100
    return w, w1, tokens, targets, 3.0


def exact(w, w1, tokens, targets, scale):
    """(mean loss, dw, dw1) and the magnitudes that the bounds need, in 64 bits."""
    w, w1 = w.double(), w1.double()
    V, T = w.size(0), len(tokens)
    e = torch.where((tokens >= 0).unsqueeze(1), scale * w[tokens.clamp(min=0)], 0.0)
    h = e @ w1.t()
    part = (tokens != -100) & (targets != -100)
    z = h @ w.t()
    lse = torch.logsumexp(z, 1)
    at = targets.clamp(min=0)
    loss = torch.where(part, lse - z.gather(1, at.unsqueeze(1)).squeeze(1), 0.0).sum() / part.sum()
    p = torch.softmax(z, 1)
    one = torch.nn.functional.one_hot(at, V).double()
    g = (part.double() / part.sum()).unsqueeze(1)
    dz = (p - one) * g
    dh = dz @ w
    de = dh @ w1
    dw = dz.t() @ h
    dw.index_add_(0, tokens.clamp(min=0), torch.where((tokens >= 0).unsqueeze(1), scale * de, 0.0))
    return loss, dw, dh.t() @ e, (e, h, p, one, g, dz, dh, de)


def bounds(w, w1, tokens, scale, parts):
    """How far fp32 may be off, element by element, for dw and dw1."""
    e, h, p, one, g, dz, dh, de = (x.abs() for x in parts)
    w, w1 = w.double().abs(), w1.double().abs()
    hb = e @ w1.t()                              # magnitudes behind h
    dh_err = 2 * E * hb                          # (e itself is off by 2^-24)
    z_err = dh_err @ w.t() + E * (hb @ w.t())
    worst = z_err.amax(1, keepdim=True)
    dz_err = g * (2 * p * (worst + E) + E * (p + one))
    dzb = dz + dz_err
    dhe = dz_err @ w + E * (dzb @ w)
    dhb = dh + dhe
    dee = dhe @ w1 + E * ((dz @ w) @ w1)
    dw = dz_err.t() @ hb + dzb.t() @ dh_err + E * (dzb.t() @ hb)
    place = (tokens >= 0).double().unsqueeze(1) * scale
    m = len(tokens) + 4
    dw.index_add_(0, tokens.clamp(min=0), place * (dee + m * U * (de + dee)))
    dw1 = dhe.t() @ e + 2 * E * (dhb.t() @ e)
    return dw * 1.01, dw1 * 1.01


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [None, "3xtf32"])
@pytest.mark.parametrize("T", [150, 1500])
def test_gradients_of_a_tied_model(T, mode):
    import train_tied
    w, w1, tokens, targets, scale = model(T)
    loss, dw, dw1 = train_tied.gradients(w.cuda(), w1.cuda(), tokens.cuda(), targets.cuda(), scale, mode, keep8=False)
    want, want_w, want_w1, parts = exact(w, w1, tokens, targets, scale)
    tol_w, tol_w1 = bounds(w, w1, tokens, scale, parts)
    part = int(((tokens != -100) & (targets != -100)).sum())
    assert abs(float(loss.double().sum()) / part - float(want)) <= 1e-4
    for got, exact_, tol in ((dw, want_w, tol_w), (dw1, want_w1, tol_w1)):
        off = (got.cpu().double() - exact_).abs()
        assert bool((off <= tol).all()), float((off / tol).max())
    # against differences of the loss
    g = torch.Generator().manual_seed(1)
    for _ in range(3):
        a, b = torch.randn(w.shape, generator=g).double(), torch.randn(w1.shape, generator=g).double()
        step = 1e-4
        up = exact(w.double() + step * a, w1.double() + step * b, tokens, targets, scale)[0]
        down = exact(w.double() - step * a, w1.double() - step * b, tokens, targets, scale)[0]
        slope = float((up - down) / (2 * step))
        got = float((dw.cpu().double() * a).sum() + (dw1.cpu().double() * b).sum())
        size = float((tol_w * a.abs()).sum() + (tol_w1 * b.abs()).sum())
        whole = float((want_w * a).abs().sum() + (want_w1 * b).abs().sum())
        assert abs(got - slope) <= size + 1e-6 * whole, (got, slope)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_clipped_step_in_16_bits(dtype):
    """The step's own gradients, clipped into fp32: N and f are those of the gradients that it left."""
    import train_tied
    w, w1, tokens, targets, scale = model(700, 301, 64)
    w, w1, tokens, targets = w.to(dtype).cuda(), w1.to(dtype).cuda(), tokens.cuda(), targets.cuda()
    _, dw, dw1 = train_tied.gradients(w, w1, tokens, targets, scale)
    assert dw.dtype == dtype and dw1.dtype == torch.float32
    true = math.sqrt(float(dw.double().square().sum() + dw1.double().square().sum()))
    outs = [torch.empty(dw.shape, device="cuda"), torch.empty_like(dw1)]
    norm = g14.clip_grad_norm([dw, dw1], 0.5 * true, out=outs)
    assert abs(float(norm) - true) <= 10.1 * U * true
    limit = float(torch.tensor(0.5 * true, dtype=torch.float32))
    for x, y in zip((dw, dw1), outs):
        want = x.double() * (limit / true)
        assert bool(((y.double() - want).abs() <= 13 * U * want.abs() + 2.0 ** -149).all())
    # the same again, on another stream and in a graph, bit for bit
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _, dw_s, dw1_s = train_tied.gradients(w, w1, tokens, targets, scale)
        norm_s = g14.clip_grad_norm([dw_s, dw1_s], 0.5 * true)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(norm, norm_s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, dw_g, dw1_g = train_tied.gradients(w, w1, tokens, targets, scale)
        norm_g = g14.clip_grad_norm([dw_g, dw1_g], 0.5 * true)
    for _ in range(3):
        dw_g.fill_(math.nan)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, norm_g) and torch.equal(dw_g, dw_s) and torch.equal(dw1_g, dw1_s)
    assert g14.check_device_error(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.gpu
def test_the_example_runs():
    import train_tied
    for loss, norm in train_tied.train(steps=4):
        assert np.isfinite(loss) and norm > 0


# ---- what the calls write of their workspaces

@pytest.mark.gpu
@pytest.mark.parametrize("T,V,D,dtype", [(1025, 300, 8, 1), (3000, 70, 1032, 2), (8192, 9, 264, 0), (9000, 50021, 33, 1),
                                         (40000, 5, 4096, 1), (70000, 300001, 16, 0), (20000, 700, 513, 1)])
def test_nothing_is_written_beside_the_workspace(T, V, D, dtype):
    types = (torch.float32, torch.bfloat16, torch.float16)
    g = torch.Generator(device="cuda").manual_seed(T)
    dy = torch.randn(T, D, device="cuda", generator=g).to(types[dtype])
    tokens = (torch.rand(T, device="cuda", generator=g) ** 4 * V).long()
    dw = torch.empty(V, D, device="cuda")
    need = g14.embedding_backward_workspace_bytes(dtype, T, V, D)
    flags = 608  # the flag words of split products, at a workspace's start
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    g14.embedding_backward_raw(dtype, 0, T, V, D, dy.data_ptr(), D, tokens.data_ptr(), 8, -100, 1.0, 0.0, dw.data_ptr(), D,
                               ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert bool((ws[need:] == 0xA5).all()) and bool((ws[:flags] == 0xA5).all())
    assert torch.equal(dw, g14.embedding_backward(dy, tokens, rows=V, dtype=torch.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 50, 545, 1200])
def test_nothing_is_written_beside_the_norms_workspace(n):
    g = torch.Generator(device="cuda").manual_seed(n)
    xs = [torch.randn(100 + 3000 * (i % 7), device="cuda", generator=g) for i in range(n - 1)]
    xs.append(torch.randn(3_000_001, device="cuda", generator=g))
    grads = g14.GradList(xs)
    need = g14.grad_workspace_bytes(n)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    norm, each = torch.zeros((), device="cuda"), torch.zeros(n, device="cuda")
    g14.grad_clip_raw(n, grads._args, None, 1.0, 1e9, norm.data_ptr(), each.data_ptr(), ws.data_ptr(), need,
                      torch.cuda.current_stream().cuda_stream)
    assert bool((ws[need:] == 0xA5).all()) and bool((ws[:608] == 0xA5).all())
    want, want_each = g14.grad_norm(grads, each=True)
    assert torch.equal(norm, want) and torch.equal(each, want_each)
