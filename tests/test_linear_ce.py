"""Softmax cross entropy of a projection's outputs (gemm14_linear_ce_forward /
_backward) against the definition in 64 bits, element by element.

Bounds, from the arithmetic the header states. Logits are products with fp32
accumulation: |dz_tv| <= d_t = 1e-5 max_v (|h_t||w_v|), the library's fp32
bound (its 16-bit products accumulate in fp32 and meet it too). lse is
1-Lipschitz in the largest logit error; its exponentials, sum and logarithm add
at most 4e-6 (1 + |lse|) (fp32 sums of up to 2^13 terms per thread in a tree of
partial sums, fp32 exponents). So loss and lse are within
2 d_t + 4e-6 (1 + |lse| + |z_y|).
dZ = (p - 1_y) g: the error of p is p (2 d_t + 1e-5), of rounding dZ to the
type u |dZ| (u = 2^-8 bf16, 2^-11 fp16, 2^-24 fp32; fp16 also ref 2^-40 where
dZ, held in units of ref 2^-15, is subnormal); the products add
1e-5 |dZ||W|; the result is rounded once (u, fp16: 2^-25 where subnormal)."""
import math

import numpy as np
import pytest
import torch

import dense_gemm_14_gb300 as g14

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # 2^-p, p significant bits
IGNORE = -100
P = 0x10000  # an aligned address that is never dereferenced


def make(T, V, D, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, D, generator=g).to(DT[dtype])
    w = (spread / max(D, 1) ** 0.5 * torch.randn(V, D, generator=g)).to(DT[dtype])
    y = torch.randint(0, V, (T,), generator=g)
    up = (torch.rand(T, generator=g) + 0.5) / max(T, 1)
    if dtype == "f16":
        up = up * 1024.0  # a loss scale: gradients inside fp16's range
    return h, w, y, up


def reference(h, w, y, up=None, ignore=IGNORE):
    """loss, lse, dH, dW and their bounds' parts, in 64 bits, rows that take part only."""
    h, w = h.double(), w.double()
    T, V = h.shape[0], w.shape[0]
    valid = (y != ignore)
    if up is not None:
        grad_valid = valid & (up != 0)
    z = h @ w.t()
    lse = torch.logsumexp(z, dim=1)
    at = torch.where(valid, y, 0).unsqueeze(1)
    zy = z.gather(1, at).squeeze(1)
    d = 1e-5 * (h.abs() @ w.abs().t()).amax(dim=1)
    out = {"loss": torch.where(valid, lse - zy, 0.0), "lse": torch.where(valid, lse, 0.0),
           "tol": torch.where(valid, 2 * d + 4e-6 * (1 + lse.abs() + zy.abs()), 0.0)}
    if up is not None:
        g = torch.where(grad_valid, up.double(), 0.0).unsqueeze(1)
        p = torch.exp(z - lse.unsqueeze(1))
        dz = p.clone()
        dz.scatter_add_(1, at, -torch.ones(T, 1, dtype=torch.float64))
        dz = dz * g
        perr = (p * g.abs()) * (2 * d.unsqueeze(1) + 1e-5)
        hv = torch.where(grad_valid.unsqueeze(1), h, 0.0)
        out.update(dh=dz @ w, dw=dz.t() @ hv, dz=dz, perr=perr, h=hv, w=w,
                   ref=float(torch.where(grad_valid, up.abs().double(), 0.0).max()) if T else 0.0)
    return out


def check_loss(loss, lse, r):
    for got, want in ((loss, r["loss"]), (lse, r["lse"])):
        diff = (got.cpu().double() - want).abs()
        assert bool((diff <= r["tol"]).all()), (float((diff - r["tol"]).max()), float(diff.max()))


def check_grads(dh, dw, r, dtype):
    u = U[dtype]
    small = (r["ref"] * 2.0 ** -40, 2.0 ** -25) if dtype == "f16" else (0.0, 1e-37)
    e = r["perr"] + (u + 1e-5) * r["dz"].abs() + small[0]
    for got, want, bound in ((dh, r["dh"], e @ r["w"].abs()), (dw, r["dw"], e.t() @ r["h"].abs())):
        if got is None:
            continue
        tol = bound + u * (want.abs() + bound) + small[1]
        diff = (got.cpu().double() - want).abs()
        assert bool((diff <= tol).all()), float((diff - tol).max())


def on_gpu(x, pad=0, offset=0):
    """x on the GPU as a view with `pad` extra elements a row and a start `offset` elements in."""
    if x.dim() == 1:
        return x.cuda()
    rows, cols = x.shape
    buf = torch.full((offset + rows * (cols + pad) + 8,), float("nan"), dtype=x.dtype, device="cuda")
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(x.cuda())
    return view


def both(h, w, y, up, dtype, mode=None, **kw):
    loss, lse = g14.linear_cross_entropy(h, w, y, fp32_mode=mode)
    dh, dw = g14.linear_cross_entropy_backward(h, w, y, lse, up, fp32_mode=mode, **kw)
    assert g14.check_device_error(torch.cuda.current_stream().cuda_stream) == 0
    return loss, lse, dh, dw


SIZES = [(1, 1, 1), (1, 7, 3), (2, 256, 8), (3, 255, 64), (5, 257, 65), (61, 1000, 200),
         (128, 512, 72), (129, 300, 128), (257, 1031, 136), (300, 4099, 96), (1023, 770, 40),
         (16, 40000, 64), (7, 5000, 1000), (8, 333, 4104), (13, 4000, 777), (32, 2049, 2050),
         (31, 100, 6000), (4, 70, 12000)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_loss_and_gradients(T, V, D, dtype):
    h, w, y, up = make(T, V, D, dtype, 100 * T + V + D, spread=2.0)
    r = reference(h, w, y, up)
    loss, lse, dh, dw = both(on_gpu(h), on_gpu(w), y.cuda(), up.cuda(), dtype)
    check_loss(loss, lse, r)
    check_grads(dh, dw, r, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("mode", ["fp32", "3xtf32"])
@pytest.mark.parametrize("T,V,D", [(3, 255, 64), (257, 1031, 136), (300, 600, 37)])
def test_fp32_modes(T, V, D, mode):
    h, w, y, up = make(T, V, D, "f32", T + V + D, spread=2.0)
    r = reference(h, w, y, up)
    loss, lse, dh, dw = both(on_gpu(h), on_gpu(w), y.cuda(), up.cuda(), "f32", mode)
    check_loss(loss, lse, r)
    check_grads(dh, dw, r, "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,D", [(5, 300, 64), (257, 1031, 136)])
def test_tf32_mode(T, V, D):
    """TF32's bound, 4e-3 of |h||w|, in place of fp32's in the logits and in each product."""
    h, w, y, up = make(T, V, D, "f32", T + V + D)
    r = reference(h, w, y, up)
    loss, lse, dh, dw = both(on_gpu(h), on_gpu(w), y.cuda(), up.cuda(), "f32", "tf32")
    d = 4e-3 * (h.double().abs() @ w.double().abs().t()).amax(dim=1)
    for got, want in ((loss, r["loss"]), (lse, r["lse"])):
        assert bool(((got.cpu().double() - want).abs() <= 2 * d + 1e-4).all())
    p = torch.exp(h.double() @ w.double().t() - r["lse"].unsqueeze(1)) * up.double().unsqueeze(1)
    e = p * torch.expm1(2 * d + 1e-4).unsqueeze(1) + 4e-3 * r["dz"].abs()
    e = e + 4e-3 * e
    assert bool(((dh.cpu().double() - r["dh"]).abs() <= e @ r["w"].abs() + 1e-30).all())
    assert bool(((dw.cpu().double() - r["dw"]).abs() <= e.t() @ r["h"].abs() + 1e-30).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hp,ho,wp,wo", [(1, 0, 0, 0), (0, 0, 1, 0), (3, 1, 5, 1), (8, 8, 16, 8),
                                         (0, 2, 0, 3)])
def test_pitches_and_offsets(hp, ho, wp, wo, dtype):
    h, w, y, up = make(150, 700, 72, dtype, 7, spread=2.0)
    r = reference(h, w, y, up)
    loss, lse, dh, dw = both(on_gpu(h, hp, ho), on_gpu(w, wp, wo), y.cuda(), up.cuda(), dtype)
    check_loss(loss, lse, r)
    check_grads(dh, dw, r, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,keep", [(1, 0), (5, 1), (300, 0), (300, 1), (300, 150), (700, 257), (700, 256)])
def test_rows_that_take_no_part(T, keep, dtype):
    """Ignored rows hold NaN and infinities: their loss, lse and dH are 0 and nothing of them reaches dW."""
    h, w, y, up = make(T, 600, 80, dtype, T + keep, spread=2.0)
    off = torch.randperm(T, generator=torch.Generator().manual_seed(T))[keep:]
    y[off] = IGNORE
    r = reference(h, w, y, up)
    h[off[0::2]] = float("nan")
    h[off[1::2]] = float("inf")
    up[off[0::3]] = float("nan")
    loss, lse, dh, dw = both(on_gpu(h), on_gpu(w), y.cuda(), up.cuda(), dtype)
    check_loss(loss, lse, r)
    check_grads(dh, dw, r, dtype)
    assert not dh[off.cuda()].any() and not loss[off.cuda()].any() and not lse[off.cuda()].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_upstream_rows_add_nothing(dtype):
    h, w, y, up = make(300, 400, 64, dtype, 5)
    up[::3] = 0.0
    r = reference(h, w, y, up)
    loss, lse = g14.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda())
    h[::3] = float("nan")
    dh, dw = g14.linear_cross_entropy_backward(h.cuda(), w.cuda(), y.cuda(), lse, up.cuda())
    check_grads(dh, dw, r, dtype)
    dh, dw = g14.linear_cross_entropy_backward(h.cuda(), w.cuda(), y.cuda(), lse,
                                               torch.zeros(300, device="cuda"))
    assert not dh.any() and not dw.any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [3, 300])
def test_bad_targets_and_nonfinite_logits_stay_in_their_rows(T, dtype):
    V = 500
    h, w, y, up = make(T, V, 64, dtype, 11)
    y[0], y[1] = V, -1  # not rows of W, not ignore_index
    clean = reference(h, w, y.clamp(0, V - 1), up)
    loss, lse, dh, dw = both(h.cuda(), w.cuda(), y.cuda(), up.cuda(), dtype)
    assert torch.isnan(loss[:2]).all() and torch.isnan(dh[:2]).all() and torch.isnan(dw).all()
    diff = (loss[2:].cpu().double() - clean["loss"][2:]).abs()
    assert bool((diff <= clean["tol"][2:]).all())
    h[2, 3] = float("nan")
    loss, lse = g14.linear_cross_entropy(h.cuda(), w.cuda(), y.clamp(0, V - 1).cuda())
    assert torch.isnan(loss[2]) and torch.isnan(lse[2])
    keep = torch.arange(T) != 2
    diff = (loss.cpu().double() - clean["loss"]).abs()[keep]
    assert bool((diff <= clean["tol"][keep]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [512, 768, 960, 1024, 1500, 4096])
@pytest.mark.parametrize("dtype,mode", [(torch.bfloat16, None), (torch.float16, None),
                                        (torch.float32, "3xtf32")])
def test_small_losses_of_learnt_rows(D, dtype, mode):
    """Tensor cores truncate, which moves all logits one way and adds up in the small
    losses of learnt rows. 1e-6 of the losses' norm is what the statistics' fp32
    roundings leave: 2^-24 of lse and of z_y (each about twice a loss here), of
    their terms and of products summed in any order."""
    g = torch.Generator(device="cuda").manual_seed(D)
    T, V = 600, 1000
    w = (0.02 * torch.randn(V, D, device="cuda", generator=g)).to(dtype)
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    lean = 8.0 * torch.rand(T, 1, device="cuda", generator=g) / (0.02 * D ** 0.5)
    wy = w[y].float()
    h = (torch.randn(T, D, device="cuda", generator=g) + lean * wy / wy.norm(dim=1, keepdim=True)).to(dtype)
    z = h.double() @ w.double().t()
    want = torch.logsumexp(z, dim=1) - z[torch.arange(T, device="cuda"), y]
    loss = g14.linear_cross_entropy(h, w, y, fp32_mode=mode)[0]
    assert float((loss.double() - want).norm()) <= 1e-6 * float(want.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("T,keep", [(1, 1), (5, 3), (16, 16), (64, 40), (65, 65), (128, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gradients_of_few_rows_are_rounded_once(T, keep, dtype):
    """dZ in two parts is off by 2^-16 (2^-22) at most, sums by 1e-5: beside the
    rounding of the gradient itself, 0.0017 (0.0002) of its norm, under 1 % of it."""
    g = torch.Generator(device="cuda").manual_seed(T)
    V, D = 3001, 520
    w = (0.02 * torch.randn(V, D, device="cuda", generator=g)).to(dtype)
    y = torch.randint(0, V, (T,), device="cuda", generator=g)
    lean = 8.0 * torch.rand(T, 1, device="cuda", generator=g) / (0.02 * D ** 0.5)
    wy = w[y].float()
    h = (torch.randn(T, D, device="cuda", generator=g) + lean * wy / wy.norm(dim=1, keepdim=True)).to(dtype)
    up = 100.0 * (0.5 + torch.rand(T, device="cuda", generator=g))
    p = torch.softmax(h.double() @ w.double().t(), dim=1)
    p[torch.arange(T, device="cuda"), y] -= 1.0
    p *= up.double()[:, None]
    p[keep:] = 0.0
    y[keep:] = IGNORE
    lse = g14.linear_cross_entropy(h, w, y, ignore_index=IGNORE)[1]
    got = g14.linear_cross_entropy_backward(h, w, y, lse, up, ignore_index=IGNORE)
    for a, want in zip(got, (p @ w.double(), p.t() @ h.double())):
        once = (want.to(dtype).double() - want).norm()
        assert float((a.double() - want).norm()) <= 1.1 * float(once) + 1e-5 * float(want.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_entries_masked_with_the_lowest_value_and_large_logits(dtype):
    """Vocabulary entries shut out by logits near the type's lowest value; others spread over +-60."""
    h, w, y, up = make(70, 600, 64, dtype, 13, spread=60.0)
    h[:, 0] = 1.0
    w[:, 0] = 0.0
    w[300:, 0] = torch.finfo(DT[dtype]).min / 2
    w[300:, 1:] = 0.0
    y = y % 300
    r = reference(h[:, 1:], w[:300, 1:], y, up)
    tol = reference(h[:, 1:], w[:300, 1:], y)["tol"]
    loss, lse, dh, dw = both(h.cuda(), w.cuda(), y.cuda(), up.cuda(), dtype)
    assert bool(((loss.cpu().double() - r["loss"]).abs() <= tol).all())
    assert not dw[300:].any()
    check_grads(dh[:, 1:], dw[:300, 1:], r, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 70, 300])
@pytest.mark.parametrize("dtype,mode", [("bf16", None), ("f16", None), ("f32", "fp32"), ("f32", "3xtf32")])
def test_entries_at_the_lowest_value_and_at_minus_infinity(T, dtype, mode):
    """Entries shut out by the type's lowest value itself (which, as an fp32, rounds to no finite
    bf16), or by minus infinity in the forward pass: the others' loss and gradients are as without them."""
    h, w, y, up = make(T, 600, 64, dtype, 31, spread=2.0)
    h[:, 0] = 1.0
    w[:, 0] = 0.0
    w[300:] = 0.0
    w[300:, 0] = torch.finfo(DT[dtype]).min
    y = y % 300
    r = reference(h[:, 1:], w[:300, 1:], y, up)
    loss, lse, dh, dw = both(h.cuda(), w.cuda(), y.cuda(), up.cuda(), dtype, mode)
    check_loss(loss, lse, r)
    assert not dw[300:].any()
    check_grads(dh[:, 1:], dw[:300, 1:], r, dtype)
    w[300:, 0] = -float("inf")
    if mode != "3xtf32" or T <= 32:  # (an infinite operand is no number in split arithmetic)
        check_loss(*g14.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), fp32_mode=mode), r)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_gradient_alone_is_the_same(dtype):
    h, w, y, up = (x.cuda() for x in make(300, 700, 72, dtype, 3))
    loss, lse, dh, dw = both(h, w, y, up, dtype)
    assert torch.equal(both(h, w, y, up, dtype, need_dw=False)[2], dh)
    assert torch.equal(both(h, w, y, up, dtype, need_dh=False)[3], dw)


@pytest.mark.gpu
def test_no_rows():
    h, w = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), torch.ones(9, 64, device="cuda", dtype=torch.bfloat16)
    e = torch.empty(0, device="cuda")
    loss, lse, dh, dw = both(h, w, torch.empty(0, dtype=torch.int64, device="cuda"), e, "bf16")
    assert loss.shape == (0,) and dh.shape == (0, 64) and not dw.any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [1, 500])
def test_runs_repeat_bit_for_bit_on_any_stream(T, dtype):
    h, w, y, up = make(T, 3000, 136, dtype, 17)
    h, w, y, up = h.cuda(), w.cuda(), y.cuda(), up.cuda()
    first = both(h, w, y, up, dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    loss, lse = g14.linear_cross_entropy(h, w, y, stream=side)
    dh, dw = g14.linear_cross_entropy_backward(h, w, y, lse, up, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(first, (loss, lse, dh, dw)):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graph_capture_replays(dtype):
    h, w, y, up = (x.cuda() for x in make(300, 1500, 72, dtype, 19))
    want = both(h, w, y, up, dtype)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(h, w, y, up, dtype)  # the stream's workspace exists before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        loss, lse = g14.linear_cross_entropy(h, w, y)
        dh, dw = g14.linear_cross_entropy_backward(h, w, y, lse, up)
    for _ in range(3):
        for x in (loss, lse, dh, dw):
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (loss, lse, dh, dw)):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_gradients_match_differences():
    """Central differences of the objective along random directions, on fp32
    data with the fp32 mode. The objective F = sum up loss is known to
    sum |up| tol; the third derivative of log-sum-exp along a direction is at
    most (range of the logits' change)^3, so with step e the difference is off by
    at most sum |up| (tol / e + e^2 R^3 / 6 * 2)."""
    T, V, D = 37, 211, 24
    h, w, y, up = make(T, V, D, "f32", 23, spread=2.0)
    g = torch.Generator().manual_seed(4)
    dirs = [(torch.randn(T, D, generator=g), None), (None, torch.randn(V, D, generator=g) / D ** 0.5)]
    hc, wc, yc = h.cuda(), w.cuda(), y.cuda()
    loss, lse, dh, dw = both(hc, wc, yc, up.cuda(), "f32")
    e = 2.0 ** -7
    for dh_dir, dw_dir in dirs:
        hd = dh_dir if dh_dir is not None else torch.zeros(T, D)
        wd = dw_dir if dw_dir is not None else torch.zeros(V, D)
        values = []
        for sign in (1, -1):
            moved = g14.linear_cross_entropy((h + sign * e * hd).cuda(), (w + sign * e * wd).cuda(), yc)[0]
            values.append(float((moved.double().cpu() * up.double()).sum()))
        change = (h.double() @ wd.double().t() + hd.double() @ w.double().t())
        R = (change.amax(dim=1) - change.amin(dim=1))
        tol = reference(h, w, y)["tol"]
        # the moved operands are rounded to fp32: 2^-24 of h and w in each logit
        moved_err = 2.0 ** -23 * (h.double().abs() @ w.double().abs().t()).amax(dim=1) * 2
        allowed = float((up.double() * ((tol * 2 + 2 * moved_err) / (2 * e) + e ** 2 * R ** 3 / 3)).sum())
        got = float((dh.cpu().double() * hd.double()).sum() + (dw.cpu().double() * wd.double()).sum())
        assert abs((values[0] - values[1]) / (2 * e) - got) <= allowed + 1e-5 * abs(got)


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """W of 2.3e9 elements: targets and logits from both ends of it."""
    V, D = 70001, 32768
    g = torch.Generator(device="cuda").manual_seed(29)
    h = torch.randn(3, D, device="cuda", generator=g).bfloat16()
    w = torch.empty(V, D, device="cuda", dtype=torch.bfloat16)
    for v in range(0, V, 8192):
        w[v:v + 8192] = (torch.randn(min(8192, V - v), D, device="cuda", generator=g) / D ** 0.5).bfloat16()
    y = torch.tensor([V - 1, 0, 65537], device="cuda")
    z = torch.cat([h.double() @ w[v:v + 8192].double().t() for v in range(0, V, 8192)], dim=1)
    za = max(float((h.double().abs() @ w[v:v + 8192].double().abs().t()).max()) for v in range(0, V, 8192))
    lse = torch.logsumexp(z, dim=1)
    want = lse - z[torch.arange(3, device="cuda"), y]
    loss, got_lse = g14.linear_cross_entropy(h, w, y)
    tol = 2e-5 * za + 4e-6 * (1 + lse.abs() + (lse - want).abs())
    assert bool(((loss.double() - want).abs() <= tol).all())
    up = torch.ones(3, device="cuda")
    dh, dw = g14.linear_cross_entropy_backward(h, w, y, got_lse, up)
    # dW of the rows at both ends: dZ^T H of the 3 rows
    for v in (0, 65537, V - 1):
        dz = torch.exp(z[:, v] - lse) - (y == v).double()
        want_dw = dz @ h.double()
        bound = (dz.abs() * (2.0 ** -8 + 1e-5) + (dz.abs() + (y == v).double()) * (2e-5 * za + 1e-5)) @ h.double().abs()
        assert bool(((dw[v].double() - want_dw).abs() <= bound + 2.0 ** -8 * (want_dw.abs() + bound)).all())


# ---- refusals (host only)

def forward(T=4, V=8, D=8, H=P, ldh=8, W=P, ldw=8, y=P, loss=P, lse=P, ws=P, n=1 << 30, dtype=1):
    return g14.linear_ce_forward(dtype, T, V, D, H, ldh, W, ldw, y, IGNORE, loss, lse, ws, n,
                                 check=False)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(V=0), dict(D=0), dict(V=-3), dict(T=1 << 31), dict(ldh=7), dict(ldw=7),
    dict(H=0), dict(W=0), dict(y=0), dict(loss=0), dict(lse=0), dict(H=P + 1), dict(W=P + 1),
    dict(y=P + 4), dict(loss=P + 2), dict(dtype=7), dict(dtype=-1), dict(dtype=0, H=P + 2)])
def test_forward_refusals(bad):
    assert forward(**bad) == g14.GEMM14_ERR_INVALID_ARG


def test_forward_of_no_rows_is_ok():
    assert forward(T=0, H=0, y=0, loss=0, lse=0, ws=0, n=0) == g14.GEMM14_OK


def backward(T=4, V=8, D=8, H=P, ldh=8, W=P, ldw=8, y=P, lse=P, g=P, dH=P, lddh=8, dW=P, lddw=8,
             ws=P, n=1 << 30, dtype=1):
    return g14.linear_ce_backward(dtype, T, V, D, H, ldh, W, ldw, y, IGNORE, lse, g, dH, lddh, dW,
                                  lddw, ws, n, check=False)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(V=0), dict(D=0), dict(ldh=7), dict(ldw=7), dict(lddh=7), dict(lddw=7),
    dict(H=0), dict(W=0), dict(y=0), dict(lse=0), dict(g=0), dict(dH=P + 1), dict(dW=P + 1),
    dict(dtype=5)])
def test_backward_refusals(bad):
    assert backward(**bad) == g14.GEMM14_ERR_INVALID_ARG


def test_backward_of_nothing_is_ok():
    assert backward(dH=0, dW=0) == g14.GEMM14_OK


def test_workspace_query_is_host_only():
    n = g14.linear_ce_workspace_bytes(1, 0, 8192, 131072, 2048, P, 2048, P, 2048, 152)
    m = g14.linear_ce_workspace_bytes(1, 1, 8192, 131072, 2048, P, 2048, P, 2048, 152)
    # pieces, not the logits: 8192 x 131072 of them would take 2 GiB in 16 bits
    assert 0 < n <= m < 1 << 30
    assert g14.linear_ce_workspace_bytes(1, 0, 0, 8, 8, P, 8, P, 8, 152) == 0
    assert g14.linear_ce_workspace_bytes(1, 0, 4, 8, 8, P, 7, P, 8, 152) == 0


@pytest.mark.gpu
def test_a_row_wider_than_a_grid_of_narrow_blocks():
    """One fp32 row of more than 65535 x 1024 columns; logits 0 and 2, so that
    every sum has one term and only exp and log round (2^-20 of values below 3)."""
    D = 65535 * 1024 + 5
    h, w = torch.zeros(1, D, device="cuda"), torch.zeros(2, D, device="cuda")
    h[0, -1], w[1, -1] = 1.0, 2.0
    y, up = torch.ones(1, dtype=torch.int64, device="cuda"), torch.ones(1, device="cuda")
    loss, lse = g14.linear_cross_entropy(h, w, y)
    p0 = 1.0 / (1.0 + math.exp(2.0))
    assert abs(float(lse) - math.log(1.0 + math.exp(2.0))) < 3e-6
    assert abs(float(loss) + math.log(1.0 - p0)) < 3e-6
    dh, dw = g14.linear_cross_entropy_backward(h, w, y, lse, up)
    assert abs(float(dh[0, -1]) + 2.0 * p0) < 6e-6
    assert abs(float(dw[0, -1]) - p0) < 3e-6 and abs(float(dw[1, -1]) + p0) < 3e-6
    assert int(torch.count_nonzero(dh)) == 1 and int(torch.count_nonzero(dw)) == 2


def test_sizes_whose_tiles_pass_32_bits_are_refused():
    """Within 255 of 2^31 a count of whole tiles does not fit 32 bits."""
    most = (1 << 31) - 256
    for bad in (dict(T=most + 1), dict(V=most + 1), dict(D=most + 1, ldh=1 << 31, ldw=1 << 31)):
        assert forward(**bad) == g14.GEMM14_ERR_INVALID_ARG
        assert backward(**bad) == g14.GEMM14_ERR_INVALID_ARG
    assert g14.linear_ce_workspace_bytes(1, 0, 4, most, 8, P, 8, P, 8, 152) > 0
    assert g14.linear_ce_workspace_bytes(1, 0, 4, most + 1, 8, P, 8, P, 8, 152) == 0


@pytest.mark.gpu
def test_small_workspace_is_refused_with_the_bytes_needed():
    h, w, y, _ = make(4, 300, 64, "bf16", 1)
    h, w, y = h.cuda(), w.cuda(), y.cuda()
    out = torch.zeros(8, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    args = (1, 4, 300, 64, h.data_ptr(), 64, w.data_ptr(), 64, y.data_ptr(), IGNORE,
            out.data_ptr(), out.data_ptr() + 16)
    need = g14.linear_ce_workspace_bytes(1, 0, 4, 300, 64, h.data_ptr(), 64, w.data_ptr(), 64)
    for ptr, n in ((ws.data_ptr(), 256), (None, 1 << 30), (ws.data_ptr() + 8, 1 << 30)):
        if n < need or ptr is None or ptr % 16:
            assert g14.linear_ce_forward(*args, ptr, n, check=False) == g14.GEMM14_ERR_INVALID_ARG
            assert str(need) in g14.last_error_string()


def test_tensor_call_refusals():
    h, w, y = torch.zeros(3, 4), torch.zeros(5, 4), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        g14.linear_cross_entropy(h, w, y)          # not on a GPU
    with pytest.raises(TypeError):
        g14.linear_cross_entropy(h.double(), w, y)
    with pytest.raises(ValueError):
        g14.linear_cross_entropy(h.half(), w.half(), y, fp32_mode="tf32")
