"""Rows of a table looked up by token (gemm14_embedding_forward) and the gradient
of the lookup (gemm14_embedding_backward), against the formulas in 64 bits.

Bounds. A looked-up value is one fp32 product (2^-24 of it, none where scale is 1)
rounded once to the output's type (half a step, eps / 2; half the smallest
subnormal below the normal numbers). A gradient's sum of m terms in fp32, in any
order, is off by at most (m - 1) 2^-24 of the sum of their magnitudes (to first
order), its product with scale and the fma with beta by 2^-24 of theirs each, and it
is rounded once to the output's type. The first-order bounds are widened by 1 %."""
import math

import pytest
import torch

import dense_gemm_14_gb300 as g14

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODE = {"f32": 0, "bf16": 1, "f16": 2}
P = 0x10000
U = 2.0 ** -24


def half_step(want, dtype):
    """Half a step of a type at values, in 64 bits."""
    f = torch.finfo(dtype)
    return torch.clamp(want.abs(), min=f.smallest_normal) * (f.eps / 2)


def view_of(x, pad, offset, fill=0.0):
    """x as rows of a larger pitch, from an offset; (buffer, view)."""
    rows, cols = x.shape
    buf = torch.full((offset + rows * (cols + pad) + 64,), fill, dtype=x.dtype, device="cuda")
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(x.cuda())
    return buf, v


def tokens_of(T, V, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "same":
        return torch.full((T,), V // 2)
    if kind == "text":  # the r-th most frequent in proportion to 1 / r
        u = torch.rand(T, generator=g, dtype=torch.float64)
        return (torch.exp(u * math.log(V + 1)).long() - 1).clamp(0, V - 1)
    if kind == "runs":  # long runs of few tokens
        return (torch.arange(T) // 37 * 7919) % V
    if kind == "ends":
        return torch.where(torch.rand(T, generator=g) < 0.5, 0, V - 1)
    return torch.randint(0, V, (T,), generator=g)


# ---- the lookup

def lookup_check(table, tokens, got, scale, ignore, out_dtype):
    V = table.size(0)
    flat = tokens.reshape(-1).cpu()
    w = table.cpu().double()
    real = (flat != ignore) & (flat >= 0) & (flat < V)
    want = w[torch.where(real, flat, 0)] * float(torch.tensor(scale, dtype=torch.float32))
    want = torch.where(real.unsqueeze(1), want, torch.where(flat == ignore, 0.0, math.nan).unsqueeze(1))
    y = got.reshape(flat.numel(), -1).cpu().double()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    bad = torch.isnan(want)
    want, y = want[~bad], y[~bad]
    limit = torch.finfo(out_dtype).max
    wide = want.abs() > limit
    assert bool((y[wide].abs() >= limit).all())
    want, y = want[~wide], y[~wide]
    tol = half_step(want, out_dtype) * 1.01 + (0.0 if scale == 1.0 else U * 1.01) * want.abs()
    assert bool(((y - want).abs() <= tol).all())
    if scale == 1.0 and table.dtype == out_dtype:
        assert torch.equal(y, want)


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 50, 4096), (3, 7, 8), (5, 100, 33), (64, 1000, 64),
                                   (257, 300, 769), (1000, 50, 1000), (33, 9, 5000), (4097, 301, 40)])
def test_lookup(T, V, D, dtype, out):
    g = torch.Generator().manual_seed(T + D)
    table = torch.randn(V, D, generator=g).to(DT[dtype]).cuda()
    tokens = tokens_of(T, V, "uniform", T)
    for scale in (1.0, math.sqrt(D)):
        for wide in (torch.int64, torch.int32):
            t = tokens.to(wide).cuda()
            y = g14.embedding(table, t, scale=scale, dtype=DT[out])
            assert y.shape == (T, D) and y.dtype == DT[out]
            lookup_check(table, tokens, y, scale, -100, DT[out])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "bf16"), ("f32", "bf16"),
                                       ("bf16", "f32")])
@pytest.mark.parametrize("pad,offset,opad,ooffset", [(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1),
                                                     (3, 5, 2, 7), (8, 8, 16, 8), (4, 4, 4, 4)])
@pytest.mark.parametrize("D", [1, 7, 64, 130])
def test_lookup_pitches_and_offsets(D, pad, offset, opad, ooffset, dtype, out):
    T, V = 70, 41
    g = torch.Generator().manual_seed(D)
    _, table = view_of(torch.randn(V, D, generator=g).to(DT[dtype]), pad, offset)
    tokens = tokens_of(T, V, "ends", 1).cuda()
    tokens[::5], tokens[3] = -100, V
    buf = torch.full((ooffset + T * (D + opad) + 32,), 7.0, dtype=DT[out], device="cuda")
    y = buf[ooffset:ooffset + T * (D + opad)].view(T, D + opad)
    g14.embedding_raw(CODE[dtype], CODE[out], T, V, D, table.data_ptr(), D + pad, tokens.data_ptr(), 8,
                      -100, 0.5, y.data_ptr(), D + opad, torch.cuda.current_stream().cuda_stream)
    lookup_check(table, tokens, y[:, :D], 0.5, -100, DT[out])
    assert bool((y[:, D:] == 7.0).all()) and bool((buf[:ooffset] == 7.0).all())
    assert bool((buf[ooffset + T * (D + opad):] == 7.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("ignore", [-100, 0, 5])
def test_tokens_that_take_no_part(ignore):
    table = torch.randn(10, 24, device="cuda")
    table[5] = float("nan")
    tokens = torch.tensor([[0, 5, 9], [10, -1, 1 << 40], [-(1 << 40), ignore, 3]], device="cuda")
    y = g14.embedding(table, tokens, ignore_index=ignore)
    assert y.shape == (3, 3, 24)
    lookup_check(table, tokens, y, 1.0, ignore, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_special_values_are_looked_up_as_they_are(dtype):
    f = torch.finfo(DT[dtype])
    row = torch.tensor([0.0, -0.0, f.max, f.min, f.tiny, f.smallest_normal / 4, math.inf, -math.inf])
    table = row.to(DT[dtype]).repeat(3, 2).cuda()
    y = g14.embedding(table, torch.tensor([2, 0], device="cuda"))
    assert torch.equal(y.view(torch.int32 if dtype == "f32" else torch.int16),
                       table[:2].view(torch.int32 if dtype == "f32" else torch.int16))


@pytest.mark.gpu
def test_lookup_beyond_32_bits():
    """A table of 2.3e9 values and an output as large: their last rows."""
    V, D = 70001, 32768
    table = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    table[-3:] = torch.randn(3, D, device="cuda").bfloat16()
    tokens = torch.zeros(V, dtype=torch.int64, device="cuda")
    tokens[-3:] = torch.tensor([V - 1, V - 3, V - 2])
    y = g14.embedding(table, tokens)
    assert torch.equal(y[-3:], table[[V - 1, V - 3, V - 2]]) and not y[:-3].any()


# ---- its gradient

def gradient_check(dy, tokens, got, scale, ignore, beta=0.0, dw0=None):
    V, D = got.shape
    flat = tokens.reshape(-1).cpu().long()
    real = (flat != ignore) & (flat >= 0) & (flat < V)
    d = dy.reshape(flat.numel(), D).cpu().double()[real]
    at = flat[real]
    s = abs(scale)
    want = torch.zeros(V, D, dtype=torch.float64).index_add_(0, at, d) * scale
    size = torch.zeros(V, D, dtype=torch.float64).index_add_(0, at, d.abs()) * s
    terms = torch.bincount(at, minlength=V).double().unsqueeze(1)
    if beta:
        old = dw0.cpu().double() * beta
        want, size = want + old, size + old.abs()
    bad = torch.isnan(want)
    y = got.cpu().double()
    assert torch.equal(torch.isnan(y), bad)
    tol = 1.01 * (terms + 3) * U * size + half_step(want, got.dtype) * 1.01
    off = (y - want).abs()
    assert bool((off[~bad] <= tol[~bad]).all()), float((off / tol)[~bad].max())


PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


def gradient_case(T, V, D, dtype, out, kind, seed=0):
    g = torch.Generator().manual_seed(T * 7 + D + seed)
    dy = torch.randn(T, D, generator=g).to(DT[dtype])
    tokens = tokens_of(T, V, kind, T + V)
    if T > 4:
        tokens[torch.randperm(T, generator=g)[:T // 9]] = -100
        tokens[1], tokens[2] = V, -1  # outside: add nothing
    dw0 = torch.randn(V, D, generator=g).to(DT[out])
    return dy, tokens, dw0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["uniform", "text", "same", "runs"])
@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (2, 3, 8), (31, 5, 33), (255, 1000, 64), (256, 77, 769),
                                   (257, 77, 769), (2048, 300, 16), (2049, 4000, 40), (5000, 513, 200),
                                   (700, 900, 2056), (1024, 60, 1032), (1025, 60, 1032), (8192, 900, 72), (8193, 900, 72),
                                   (20000, 700, 24), (3000, 37, 264)])
def test_gradient(T, V, D, dtype, out, kind):
    dy, tokens, dw0 = gradient_case(T, V, D, dtype, out, kind)
    dy_, t_ = dy.cuda(), tokens.cuda()
    got = g14.embedding_backward(dy_, t_, rows=V, dtype=DT[out])
    assert got.shape == (V, D) and got.dtype == DT[out]
    gradient_check(dy, tokens, got, 1.0, -100)
    for scale, beta in ((0.75, 1.0), (-2.0, 0.5)):
        dw = dw0.cuda()
        g14.embedding_backward(dy_, t_, out=dw, scale=scale, beta=beta)
        gradient_check(dy, tokens, dw, scale, -100, beta, dw0)
    again = g14.embedding_backward(dy_, t_.int(), rows=V, dtype=DT[out])
    assert torch.equal(again, got)  # the same order, whatever the tokens' type


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("T", [40, 900, 2500])
@pytest.mark.parametrize("D,pad,offset,opad,ooffset", [(64, 1, 0, 0, 0), (64, 0, 1, 0, 0), (64, 0, 0, 1, 0),
                                                       (64, 0, 0, 0, 1), (130, 3, 5, 2, 7), (7, 1, 1, 1, 1),
                                                       (1001, 0, 0, 0, 0), (1000, 8, 8, 8, 8)])
def test_gradient_pitches_and_offsets(T, D, pad, offset, opad, ooffset, dtype, out):
    """NaN beside the rows of dY, in rows that take no part and (beta = 0) in dW reaches
    nothing; what lies beside dW's rows stays as it is."""
    V = 61
    dy, tokens, _ = gradient_case(T, V, D, dtype, out, "text")
    tokens[tokens == 17] = 16  # a row without tokens
    dy[tokens == -100] = math.nan
    dy[1] = dy[2] = math.nan  # tokens outside [0, V)
    _, dyv = view_of(dy, pad, offset, math.nan)
    buf = torch.full((ooffset + V * (D + opad) + 32,), math.nan, dtype=DT[out], device="cuda")
    whole = buf[ooffset:ooffset + V * (D + opad)].view(V, D + opad)
    dw = whole[:, :D]
    g14.embedding_backward(dyv, tokens.cuda(), out=dw)
    gradient_check(dy, tokens, dw, 1.0, -100)
    assert bool((dw[17] == 0).all())
    before = dw.cpu()
    dw[17] = math.nan
    g14.embedding_backward(dyv, tokens.cuda(), out=dw, scale=-0.5, beta=1.0)
    assert bool(torch.isnan(dw[17]).all())  # neither read nor written
    dw[17] = before[17].cuda()
    gradient_check(dy, tokens, dw, -0.5, -100, 1.0, before)
    g14.embedding_backward(dyv, tokens.cuda(), out=dw, scale=0.0, beta=-1.0)
    assert bool(torch.isnan(whole[:, D:]).all()) and bool(torch.isnan(buf[:ooffset]).all())
    assert bool(torch.isnan(buf[ooffset + V * (D + opad):]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("scale,beta", [(0.75, 0.5), (0.0, -1.0), (-2.0, 1.0)])
@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("T,V,D,pad,offset,opad,ooffset,kind", [
    (1100, 61, 7, 1, 1, 1, 1, "text"), (2500, 3001, 130, 3, 5, 2, 7, "text"), (4096, 40, 257, 0, 0, 0, 0, "uniform"),
    (5000, 900, 1001, 0, 0, 0, 0, "text"), (6000, 513, 257, 0, 1, 1, 0, "runs"), (5000, 7, 64, 0, 0, 1, 0, "uniform"),
    (5000, 7, 64, 1, 0, 0, 0, "same"), (20000, 4001, 333, 0, 0, 0, 0, "text"), (40000, 300, 65, 1, 3, 0, 1, "text")])
def test_gradient_of_rows_anywhere_with_any_factors(T, V, D, pad, offset, opad, ooffset, kind, dtype, out, scale, beta):
    """Ranked and sorted places, sums at any address and joins; rows without tokens (whose
    beta is theirs too), and what lies beside dW's rows."""
    dy, tokens, dw0 = gradient_case(T, V, D, dtype, out, kind)
    tokens[tokens == V - 3] = V - 2  # a row without tokens
    _, dyv = view_of(dy, pad, offset, math.nan)
    buf, dw = view_of(dw0, opad, ooffset, math.nan)
    g14.embedding_backward(dyv, tokens.cuda(), out=dw, scale=scale, beta=beta)
    gradient_check(dy, tokens, dw, scale, -100, beta, dw0)
    assert torch.equal(dw[V - 3].cpu(), (dw0[V - 3].float() * beta).to(DT[out]))
    dw.fill_(math.nan)
    assert bool(torch.isnan(buf).all())  # nothing beside the rows was written


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,D", [(70000, 300001, 4), (300000, 50, 8), (131072, 1 << 20, 3), (3000, 1 << 19, 1)])
@pytest.mark.parametrize("kind", ["uniform", "text", "ends"])
def test_many_tokens_and_large_vocabularies(T, V, D, kind):
    dy, tokens, _ = gradient_case(T, V, D, "bf16", "f32", kind)
    got = g14.embedding_backward(dy.cuda(), tokens.cuda(), rows=V, dtype=torch.float32)
    gradient_check(dy, tokens, got, 1.0, -100)
    assert torch.equal(got, g14.embedding_backward(dy.cuda(), tokens.cuda(), rows=V, dtype=torch.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 200, 3000, 10000])
@pytest.mark.parametrize("beta", [0.0, 1.0, 0.5])
def test_no_token_takes_part(T, beta):
    dw0 = torch.randn(90, 40, device="cuda")
    dw = dw0.clone() if beta else torch.full_like(dw0, math.nan)
    dy = torch.full((T, 40), math.nan, device="cuda")
    tokens = torch.full((T,), 33, device="cuda")
    g14.embedding_backward(dy, tokens, out=dw, beta=beta, ignore_index=33)
    assert torch.equal(dw, dw0 * beta if beta else torch.zeros_like(dw0))


@pytest.mark.gpu
def test_infinities_and_nan_stay_in_their_rows():
    for T in (100, 1000, 4000):
        dy = torch.randn(T, 48, device="cuda")
        tokens = torch.arange(T, device="cuda") % 20
        dy[3, 5], dy[4, 6], dy[24, 6], dy[7, 7] = math.inf, math.inf, -math.inf, math.nan
        got = g14.embedding_backward(dy, tokens, rows=20)
        assert got[3, 5] == math.inf and torch.isnan(got[4, 6]) and torch.isnan(got[7, 7])
        got[3, 5] = got[4, 6] = got[7, 7] = 0
        assert bool(torch.isfinite(got).all())


@pytest.mark.gpu
def test_shapes_of_a_batch():
    tokens = tokens_of(60, 30, "text", 1).view(4, 15).cuda()
    dy = torch.randn(4, 15, 64, device="cuda")
    a = g14.embedding_backward(dy, tokens, rows=30)
    assert torch.equal(a, g14.embedding_backward(dy.view(60, 64), tokens.view(60), rows=30))
    table = torch.randn(30, 64, device="cuda")
    y = g14.embedding(table, tokens)
    assert y.shape == (4, 15, 64) and torch.equal(y, table[tokens])
    one = g14.embedding(table, torch.tensor(7, device="cuda"))
    assert one.shape == (64,) and torch.equal(one, table[7])
    back = g14.embedding_backward(one, torch.tensor(7, device="cuda"), rows=30)
    assert torch.equal(back[7], one) and not back[:7].any() and not back[8:].any()
    assert g14.embedding(table, torch.empty(0, 3, dtype=torch.int64, device="cuda")).shape == (0, 3, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [64, 900, 1500])
def test_gradient_against_differences(T):
    """L = sum(r * embedding(W, tokens)) is linear in W: its derivative along a direction
    is the difference of two values, formed here from looked-up rows in 64 bits."""
    V, D, scale = 211, 72, 3.0
    g = torch.Generator().manual_seed(5)
    tokens = tokens_of(T, V, "text", 2).cuda()
    tokens[::6] = -100
    r = torch.randn(T, D, generator=g).cuda()
    w = torch.randint(-64, 64, (V, D), generator=g).float().cuda() / 64  # exact steps
    way = torch.randint(-8, 9, (V, D), generator=g).float().cuda()

    def loss(table):
        return (r.double() * g14.embedding(table, tokens, scale=scale).double()).sum()

    dw = g14.embedding_backward(r, tokens, rows=V, scale=scale)
    slope = float((loss(w + way / 64) - loss(w - way / 64)) * 32)
    got = float((dw.double() * way.double()).sum())
    size = float(r.abs().double().sum()) * scale * 8
    # each entry of dw is within (m + 1) 2^-24 of its terms' magnitudes, m <= T, and the
    # direction at most 8; the looked-up values and their differences are exact
    assert abs(got - slope) <= (T + 2) * U * size


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    T, V, D = 70001, 70001, 32768
    dy = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    dy[-2:] = torch.randn(2, D, device="cuda").bfloat16()
    tokens = torch.zeros(T, dtype=torch.int64, device="cuda")
    tokens[-2:] = V - 1
    dw = g14.embedding_backward(dy, tokens, rows=V)
    want = (dy[-2].float() + dy[-1].float()).bfloat16()
    assert torch.equal(dw[-1], want) and not dw[:-1].any()


# ---- streams, captures, threads

@pytest.mark.gpu
@pytest.mark.parametrize("T", [100, 4000, 20000])
def test_on_another_stream_and_repeated(T):
    dy, tokens, _ = gradient_case(T, 500, 264, "bf16", "bf16", "text")
    dy, tokens = dy.cuda(), tokens.cuda()
    want = g14.embedding_backward(dy, tokens, rows=500)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [g14.embedding_backward(dy, tokens, rows=500, stream=side) for _ in range(5)]
    rows = g14.embedding(want, tokens, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(want, x) for x in got)
    assert torch.equal(rows.nan_to_num(1e30), g14.embedding(want, tokens).nan_to_num(1e30))


@pytest.mark.gpu
def test_back_to_back_calls_share_the_workspace():
    cases = [gradient_case(T, V, D, "bf16", "f32", kind) for T, V, D, kind in
             [(3000, 400, 512, "same"), (300, 90, 64, "text"), (9000, 5000, 128, "uniform"), (2500, 3, 2048, "ends")] * 3]
    cases = [(dy.cuda(), t.cuda(), w.size(0)) for dy, t, w in cases]
    got = [g14.embedding_backward(dy, t, rows=V, dtype=torch.float32) for dy, t, V in cases]
    torch.cuda.synchronize()
    for (dy, t, V), x in zip(cases, got):
        gradient_check(dy.cpu(), t.cpu(), x, 1.0, -100)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [120, 3000, 10000])
@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_captured_and_replayed_on_other_tokens(T, beta):
    V, D = 300, 136
    dy, tokens, dw0 = gradient_case(T, V, D, "bf16", "bf16", "text")
    d, t, dw, table = dy.cuda(), tokens.cuda(), dw0.cuda(), dw0.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g14.embedding_backward(d, t, out=dw.clone(), beta=beta)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rows = g14.embedding(table, t)
        g14.embedding_backward(d, t, out=dw, beta=beta)
        g14.embedding_backward(d, t, out=dw, scale=0.5, beta=1.0)
    for seed in (1, 2):
        dy2, tokens2, dw2 = gradient_case(T, V, D, "bf16", "bf16", "uniform" if seed == 1 else "same", seed)
        d.copy_(dy2)
        t.copy_(tokens2)
        dw.copy_(dw2)
        graph.replay()
        torch.cuda.synchronize()
        first = dw2.cuda()
        g14.embedding_backward(d, t, out=first, beta=beta)
        g14.embedding_backward(d, t, out=first, scale=0.5, beta=1.0)
        assert torch.equal(first, dw)
        lookup_check(table, t, rows, 1.0, -100, torch.bfloat16)


# ---- refusals (host only)

@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=9), dict(dtype_out=4), dict(T=-1), dict(V=0), dict(D=0), dict(V=-1),
    dict(T=(1 << 31) - 255), dict(V=(1 << 31) - 255), dict(D=(1 << 31) - 255), dict(ldw=63), dict(ldo=63),
    dict(W=0), dict(out=0), dict(tokens=0), dict(token_bytes=2), dict(tokens=P + 4), dict(W=P + 1),
    dict(out=P + 1), dict(scale=math.inf), dict(scale=math.nan)])
def test_lookup_refusals(bad):
    a = dict(dtype=1, dtype_out=1, T=4, V=8, D=64, W=P, ldw=64, tokens=P, token_bytes=8, ignore=-100, scale=1.0,
             out=P, ldo=64) | bad
    assert g14.embedding_raw(*a.values(), check=False) == g14.GEMM14_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=9), dict(dtype_out=2), dict(dtype=0), dict(T=-1), dict(V=0), dict(D=0),
    dict(T=(1 << 31) - 255), dict(V=(1 << 31) - 255), dict(lddy=63), dict(lddw=63), dict(dY=0), dict(dW=0),
    dict(tokens=0), dict(token_bytes=3), dict(tokens=P + 4), dict(dY=P + 1), dict(dW=P + 1), dict(scale=math.inf),
    dict(beta=math.nan), dict(ws=P + 8)])
def test_gradient_refusals(bad):
    a = dict(dtype=1, dtype_out=1, T=4, V=8, D=64, dY=P, lddy=64, tokens=P, token_bytes=8, ignore=-100, scale=1.0,
             beta=0.0, dW=P, lddw=64, ws=P, n=1 << 30) | bad
    assert g14.embedding_backward_raw(*a.values(), check=False) == g14.GEMM14_ERR_INVALID_ARG


def test_workspace_sizes():
    need = g14.embedding_backward_workspace_bytes
    assert need(1, 100, 1000, 64, 152) == 0 and need(1, 5000, 1000, 64, 152) > 5000 * 16
    assert need(9, 5000, 10, 64, 152) == 0 and need(1, 5000, 0, 64, 152) == 0 and need(1, -1, 10, 64, 152) == 0
    big = need(1, 1 << 20, 1 << 20, 4096, 152)
    # sixteen bytes a place, and slots that do not grow: two rows of 4096 floats for each
    # of two waves of 4 ranges an SM
    assert (1 << 24) < big <= (1 << 24) + 2 * 608 * 2 * 4096 * 4 + (1 << 16)


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("V,D", [(1, 1), (50021, 769), (300, 4096), (1 << 30, 8)])
def test_the_tokens_that_need_no_workspace(V, D, dtype):
    """The tensor-level call asks for none up to as many tokens as the library needs none for."""
    from dense_gemm_14_gb300 import training
    few = training._FEW_TOKENS
    for sms in (1, 152):
        need = [g14.embedding_backward_workspace_bytes(dtype, T, V, D, sms) for T in (0, 1, few // 2, few, few + 1, 2 * few)]
        assert need[:4] == [0] * 4 and min(need[4:]) > 0


@pytest.mark.gpu
def test_small_workspace_is_refused():
    T = 5000
    dy, t = torch.randn(T, 64, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    dw = torch.zeros(8, 64, device="cuda")
    need = g14.embedding_backward_workspace_bytes(0, T, 8, 64)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for ptr, n in ((ws.data_ptr(), need - 1), (None, 0)):
        assert g14.embedding_backward_raw(0, 0, T, 8, 64, dy.data_ptr(), 64, t.data_ptr(), 8, -100, 1.0, 0.0,
                                          dw.data_ptr(), 64, ptr, n, check=False) == g14.GEMM14_ERR_INVALID_ARG
        assert str(need) in g14.last_error_string()


def test_tensor_call_refusals():
    w, t = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        g14.embedding(w, t)  # not on a GPU
    with pytest.raises(TypeError):
        g14.embedding(w.double(), t)
    with pytest.raises(TypeError):
        g14.embedding(w, t, dtype=torch.int8)
    with pytest.raises(TypeError):
        g14.embedding_backward(w.double(), t, rows=4)
    with pytest.raises(ValueError):
        g14.embedding_backward(torch.zeros(4, 8), t, rows=4)  # a row too many


@pytest.mark.gpu
def test_tensor_call_refusals_on_the_gpu():
    w, t = torch.zeros(4, 8, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    dy = torch.zeros(3, 8, device="cuda")
    for bad in (t.cpu(), t.repeat(2)[::2]):
        with pytest.raises(ValueError):
            g14.embedding(w, bad)
    with pytest.raises(TypeError):
        g14.embedding(w, t.short())
    with pytest.raises(ValueError):
        g14.embedding(w.t(), t)
    for kwargs in (dict(), dict(rows=4, beta=1.0), dict(rows=5, out=w), dict(out=w[:, :7]), dict(out=w, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            g14.embedding_backward(dy, t, **kwargs)
    with pytest.raises(TypeError):
        g14.embedding_backward(dy.bfloat16(), t, rows=4, dtype=torch.float16)
    with pytest.raises(ValueError):
        g14.embedding_backward(dy, t, out=w.t()[:, :3])
    with pytest.raises(ValueError):
        g14.embedding_backward(torch.zeros(3, 8, 3, device="cuda").transpose(1, 2)[:, :1], t.view(3, 1), rows=4)
    assert g14.check_device_error(torch.cuda.current_stream().cuda_stream) == 0
