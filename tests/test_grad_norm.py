"""The norm of many gradients taken together and their clipping (gemm14_grad_norm,
gemm14_grad_clip), against the formulas in 64 bits.

Bounds. At most 64 squares are added in fp32, 16 in a row into each of four sums and
those by twos: 18 roundings on a value's way, 18 2^-24 of the sum of squares (all of
them positive) to first order; what is added in fp64 adds nothing of that order. The
norm has half of that, and its own rounding: 10 2^-24. The factor has the norm's
error before that rounding (9 2^-24) and its own (2^-24), a product 2^-24 and its
rounding to the output's type half a step: (11 2^-24 + eps / 2) of the value, half a
step of the smallest subnormal below. First-order bounds are widened by 1 %."""
import math

import pytest
import torch

import dense_gemm_14_gb300 as g14

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
P = 0x10000
U = 2.0 ** -24


def squares(x):
    return float(x.double().square().sum())


def norm_check(got, want):
    got = float(got)
    if math.isfinite(want) and want <= torch.finfo(torch.float32).max:
        assert abs(got - want) <= 10.1 * U * want + 2.0 ** -150, (got, want)
    else:
        assert got == want or (math.isnan(got) and math.isnan(want)) or (want > 3.4e38 and got == math.inf)


def f32(x):
    """A limit as the call takes it."""
    return float(torch.tensor(x, dtype=torch.float32))


def factor_of(norm, max_norm, scale):
    max_norm = f32(max_norm)
    return scale * max_norm / norm if math.isfinite(norm) and norm > max_norm else scale


def out_check(y, x, factor):
    want = x.cpu().double() * factor
    f = torch.finfo(y.dtype)
    tol = 1.01 * (11 * U * want.abs() + torch.clamp(want.abs(), min=f.smallest_normal) * f.eps / 2)
    off = (y.cpu().double() - want).abs()
    fine = torch.isfinite(want) & (want.abs() <= f.max)
    assert bool((off[fine] <= tol[fine]).all()), float((off / tol)[fine].max())
    assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want))


def tensors_of(shapes, dtypes, seed, gap=0, offset=0):
    """Tensors one after the other in flat buffers, `gap` elements apart, the first from `offset`."""
    g = torch.Generator().manual_seed(seed)
    at = {d: offset for d in dtypes}
    places = []
    for i, s in enumerate(shapes):
        d = dtypes[i % len(dtypes)]
        places.append((d, at[d], s))
        at[d] += math.prod(s) + gap
    buffers = {d: torch.full((n + 16,), math.nan, dtype=DT[d], device="cuda") for d, n in at.items()}
    out = []
    for d, start, s in places:
        n = math.prod(s)
        x = buffers[d][start:start + n].view(s)
        x.copy_((torch.randn(s, generator=g) * math.exp(float(torch.randn((), generator=g)))).to(DT[d]))
        out.append(x)
    return out, buffers


SHAPES = [
    [(1,)], [(7,)], [(4096,)], [(4097,), (1,), (3, 5)], [(300, 1001), (1001,), (17, 64, 33)],
    [(2048,)] * 40, [(5,)] * 200, [(1000, 1000), (0,), (3, 0, 2), (1,)], [(131, 77)] * 30 + [(3000000,)],
    [(1 << 20,)] * 3 + [(3,)] * 100,
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtypes", [["f32"], ["bf16"], ["f16"], ["bf16", "f32"], ["f16", "f32", "bf16"]])
@pytest.mark.parametrize("gap,offset", [(0, 0), (0, 1), (5, 3), (8, 8)])
@pytest.mark.parametrize("shapes", SHAPES, ids=range(len(SHAPES)))
def test_norm_and_clipping(shapes, gap, offset, dtypes):
    xs, buffers = tensors_of(shapes, dtypes, len(shapes) + gap, gap, offset)
    each_sq = [squares(x) for x in xs]
    true = math.sqrt(math.fsum(each_sq))
    for scale in (1.0, -0.25):
        norm, each = g14.grad_norm(xs, scale=scale, each=True)
        norm_check(norm, abs(scale) * true)
        assert each.shape == (len(xs),)
        for e, s in zip(each.tolist(), each_sq):
            norm_check(e, abs(scale) * math.sqrt(s))
    assert torch.equal(norm, g14.grad_norm(g14.GradList(xs), scale=-0.25))
    before = {d: b.clone() for d, b in buffers.items()}
    olds = [x.clone() for x in xs]
    # within the limit: nothing is written
    norm_check(g14.clip_grad_norm(xs, 2 * true), true)
    assert all(torch.equal(b.nan_to_num(7.0), before[d].nan_to_num(7.0)) for d, b in buffers.items())
    # into others of each type, at another place
    for out in ("same", "f32"):
        ys, ybuf = tensors_of(shapes, dtypes if out == "same" else ["f32"], 9, gap + 1, offset + 1)
        zs = [y.clone() for y in ys]
        norm, each = g14.clip_grad_norm(xs, 0.3 * true, scale=0.5, out=ys, each=True)
        norm_check(norm, 0.5 * true)
        for y, x in zip(ys, xs):
            out_check(y, x, factor_of(0.5 * true, 0.3 * true, 0.5))
        for y, z in zip(ys, zs):
            y.copy_(z)
        want = tensors_of(shapes, dtypes if out == "same" else ["f32"], 9, gap + 1, offset + 1)[1]
        assert all(torch.equal(b.nan_to_num(7.0), want[d].nan_to_num(7.0)) for d, b in ybuf.items())
    # in place
    norm = g14.clip_grad_norm(xs, 0.1 * true)
    norm_check(norm, true)
    for x, old in zip(xs, olds):
        out_check(x, old, factor_of(true, 0.1 * true, 1.0))
        x.copy_(old)
    assert all(torch.equal(b.nan_to_num(7.0), before[d].nan_to_num(7.0)) for d, b in buffers.items())
    assert g14.check_device_error(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,cols,pad,offset,opad,ooffset", [
    (1, 1, 3, 0, 0, 0), (300, 5, 3, 1, 4, 2), (37, 64, 8, 0, 8, 0), (129, 130, 1, 1, 0, 0), (5, 9000, 7, 3, 2, 1),
    (2, 2041, 7, 0, 0, 3), (3, 1017, 0, 1, 1, 0), (4000, 1, 1, 0, 1, 1), (64, 4096, 64, 0, 0, 0)])
def test_rows_of_a_pitch(rows, cols, pad, offset, opad, ooffset, dtype, out):
    g = torch.Generator().manual_seed(rows + cols)

    def pitched(kind, pad, offset):
        buf = torch.full((offset + rows * (cols + pad) + 32,), math.nan, dtype=DT[kind], device="cuda")
        return buf, buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]

    xbuf, x = pitched(dtype, pad, offset)
    x.copy_(torch.randn(rows, cols, generator=g))
    ybuf, y = pitched(out, opad, ooffset)
    b = torch.randn(77, generator=g).cuda()
    true = math.sqrt(squares(x) + squares(b))
    norm, each = g14.grad_norm([b, x], each=True)
    norm_check(norm, true)
    norm_check(each[1], math.sqrt(squares(x)))
    bo = torch.zeros_like(b)
    norm_check(g14.clip_grad_norm([b, x], 0.5, out=[bo, y]), true)
    out_check(y, x, factor_of(true, 0.5, 1.0))
    out_check(bo, b, factor_of(true, 0.5, 1.0))
    y.fill_(math.nan)
    assert bool(torch.isnan(ybuf).all())  # nothing beside the rows was written
    old = x.clone()
    g14.clip_grad_norm([b, x], 0.5)
    out_check(x, old, factor_of(true, 0.5, 1.0))
    x.fill_(math.nan)
    assert bool(torch.isnan(xbuf).all())


@pytest.mark.gpu
def test_other_layouts():
    x = torch.randn(30, 20, 8, 6, device="cuda").to(memory_format=torch.channels_last)
    t = torch.randn(50, 70, device="cuda").t()
    wide = torch.randn(6, 10, 40, device="cuda")[:, :, :17]  # rows of one pitch
    true = math.sqrt(squares(x) + squares(t) + squares(wide))
    norm_check(g14.grad_norm([x, t, wide]), true)
    old = [x.clone(), t.clone(), wide.clone()]
    norm_check(g14.clip_grad_norm([x, t, wide], 1.0), true)
    for a, b in zip((x, t, wide), old):
        out_check(a, b, 1.0 / true)
    out = [torch.empty_like(x), torch.empty(50, 70, device="cuda").t()]
    now = math.sqrt(squares(x) + squares(t))
    g14.clip_grad_norm([x, t], 0.5 * now, out=out)
    out_check(out[0], x, factor_of(now, 0.5 * now, 1.0))
    out_check(out[1], t, factor_of(now, 0.5 * now, 1.0))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [15, 16, 17, 72, 73, 544, 545, 577, 1500])
def test_long_lists(n):
    """Lists of one and several launches, tensors of all sizes among them."""
    g = torch.Generator().manual_seed(n)
    sizes = torch.exp(torch.rand(n, generator=g) * 9).long().tolist()
    sizes[n // 2] = 200001
    sizes[n // 3] = 0
    xs, _ = tensors_of([(s,) for s in sizes], ["bf16", "f32"], n, 1, 1)
    each_sq = [squares(x) for x in xs]
    true = math.sqrt(math.fsum(each_sq))
    grads = g14.GradList(xs)
    assert len(grads) == n and grads.tensors[3] is xs[3]
    norm, each = g14.grad_norm(grads, each=True)
    norm_check(norm, true)
    for e, s in zip(each.tolist(), each_sq):
        norm_check(e, math.sqrt(s))
    olds = [x.clone() for x in xs]
    outs = [torch.full_like(x, math.nan, dtype=torch.float32) for x in xs]
    norm, each2 = g14.clip_grad_norm(grads, 1.0, out=outs, each=True)
    assert torch.equal(each, each2)
    for y, x in zip(outs, olds):
        out_check(y, x, factor_of(true, 1.0, 1.0))
    g14.clip_grad_norm(grads, 1.0)
    for x, old in zip(xs, olds):
        out_check(x, old, factor_of(true, 1.0, 1.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_values_of_any_size(dtype):
    """Squares beyond what fp32 holds, and beyond its smallest, count as they should; zeros are zeros."""
    f = torch.finfo(DT[dtype])
    small = f.smallest_normal
    for values in ([f.max] * 100, [f.max, small], [small / 4] * 1000, [small] * 3000, [0.0] * 5000, [-0.0] * 9,
                   [1e-3] * 10 + [small] * 10, [3e4] * 70, [0.0] * 4000 + [small / 2]):
        x = torch.tensor(values, dtype=torch.float64).to(DT[dtype]).cuda()
        norm, each = g14.grad_norm([x], each=True)
        norm_check(norm, math.sqrt(squares(x)))
        assert torch.equal(each[0], norm)
        # to a norm of 1, where the factor is a number that fp32 holds
        true = math.sqrt(squares(x))
        if 1e-3 < true < 1e36:
            y = torch.empty_like(x, dtype=torch.float32)
            g14.clip_grad_norm([x], min(1.0, true / 2), out=[y])
            out_check(y, x, factor_of(true, min(1.0, true / 2), 1.0))
    huge = torch.full((4,), f.max, dtype=DT[dtype], device="cuda")
    got = g14.clip_grad_norm([huge], 1.0)
    if dtype == "f16":
        norm_check(got, 2.0 * f.max)
    else:
        assert got == math.inf  # beyond fp32; the factor is worked out in 64 bits all the same
    assert abs(float(huge.double().square().sum()) - 1.0) <= 2 * (f.eps / 2 + 11 * U) * 1.01


@pytest.mark.gpu
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_a_norm_that_is_no_number_clips_nothing(value):
    x, y = torch.randn(5000, device="cuda"), torch.randn(300, device="cuda").bfloat16()
    x[4321] = value
    old = [x.clone(), y.clone()]
    norm, each = g14.clip_grad_norm([x, y], 1e-3, each=True)
    want = math.nan if math.isnan(value) else math.inf
    norm_check(norm, want)
    norm_check(each[0], want)
    norm_check(each[1], math.sqrt(squares(y)))
    assert torch.equal(x.nan_to_num(9.0), old[0].nan_to_num(9.0)) and torch.equal(y, old[1])
    out = [torch.empty_like(x), torch.empty_like(y)]
    g14.clip_grad_norm([x, y], 1e-3, scale=0.5, out=out)
    assert torch.equal(out[0].nan_to_num(9.0), (x * 0.5).nan_to_num(9.0)) and torch.equal(out[1], y * 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [50, 600001, 5000001])  # one launch, two, three for the clipping
def test_finite_elements_are_clipped_where_their_norm_is_beyond_fp32(n):
    x = torch.full((n,), 3e38, device="cuda")
    true = math.sqrt(squares(x))
    assert true > torch.finfo(torch.float32).max
    y = torch.empty_like(x)
    norm, each = g14.clip_grad_norm([x], 2.0, out=[y], each=True)
    assert norm == math.inf and each[0] == math.inf and g14.grad_norm([x]) == math.inf
    out_check(y, x, 2.0 / true)
    # the same norm for an element that is infinite: nothing is clipped
    x[n // 2] = math.inf
    assert g14.clip_grad_norm([x], 2.0, scale=0.5, out=[y]) == math.inf
    assert torch.equal(y, x * 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1.0, -0.25])
@pytest.mark.parametrize("dtype,out,size,limits", [
    ("f32", "f32", 1e37, (1e-3, 1e-7)), ("bf16", "bf16", 1e37, (1e-3, 1e-7)), ("bf16", "f32", 1e37, (1e-3, 1e-7)),
    ("f32", "f32", 3.0, (1e-37, 1e-40)), ("f16", "f32", 1e4, (1e-33, 1e-38))])
@pytest.mark.parametrize("shapes", [[(300,), (7,)], [(600001,), (17, 33)], [(400, 30)] * 90],
                         ids=["one launch", "two launches", "long"])
def test_factors_below_the_normal_numbers(shapes, dtype, out, size, limits, scale):
    """A limit so far below the norm that fp32 does not hold the factor to 24 bits, or at all: the
    bounds are those of any other factor. Rows of a pitch and unaligned ones among them."""
    xs, _ = tensors_of(shapes, [dtype], len(shapes), 3, 1)
    xs.append(torch.ones(40, 70, dtype=DT[dtype], device="cuda")[:, 1:67])
    for x in xs:
        x.copy_(x.float().clamp(-4, 4) * size)
    true = abs(scale) * math.sqrt(math.fsum(squares(x) for x in xs))
    for limit in limits:
        assert abs(scale) * f32(limit) / true < 2.0 ** -126
        ys = [torch.full_like(x, math.nan, dtype=DT[out]) for x in xs]
        norm = g14.clip_grad_norm(xs, limit, scale=scale, out=ys)
        norm_check(norm, true)
        for y, x in zip(ys, xs):
            out_check(y, x, factor_of(true, limit, scale))
    if dtype == out:
        olds = [x.clone() for x in xs]
        g14.clip_grad_norm(xs, limits[0], scale=scale)
        for x, old in zip(xs, olds):
            out_check(x, old, factor_of(true, limits[0], scale))


@pytest.mark.gpu
def test_limits():
    x = torch.randn(1000, device="cuda")
    old, true = x.clone(), math.sqrt(squares(x))
    norm_check(g14.clip_grad_norm([x], math.inf), true)
    assert torch.equal(x, old)
    g14.clip_grad_norm([x], math.inf, scale=2.0)
    assert torch.equal(x, old * 2)
    g14.clip_grad_norm([x], 0.0)
    assert not x.any()
    norm_check(g14.clip_grad_norm([x], 0.0), 0.0)  # nothing to clip
    assert g14.grad_norm([]) == 0 and g14.clip_grad_norm([], 1.0) == 0
    norm, each = g14.grad_norm([torch.empty(0, device="cuda")], each=True)
    assert norm == 0 and each.tolist() == [0.0]


@pytest.mark.gpu
def test_norm_beyond_32_bits():
    x = torch.zeros((1 << 32) + 4099, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.tensor([3.0, 4.0, 12.0])
    x[0] = 84.0
    norm_check(g14.grad_norm([x]), 85.0 + 0.0)  # 84, and 13
    g14.clip_grad_norm([x], 42.5)
    assert x[0] == 42.0 and x[-3:].tolist() == [1.5, 2.0, 6.0] and x.count_nonzero() == 4


# ---- streams, captures

@pytest.mark.gpu
def test_on_another_stream_and_repeated():
    xs, _ = tensors_of([(300, 1001), (1001,), (70000,), (3,)], ["bf16", "f32"], 3)
    want = g14.grad_norm(xs, each=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [g14.grad_norm(xs, each=True, stream=side) for _ in range(6)]
    torch.cuda.synchronize()
    for norm, each in got:
        assert torch.equal(norm, want[0]) and torch.equal(each, want[1])


@pytest.mark.gpu
def test_captured_and_replayed():
    xs, _ = tensors_of([(200, 101), (101,), (50000,)] * 30, ["f16", "f32"], 3)
    outs = [torch.empty_like(x, dtype=torch.float32) for x in xs]
    grads, out_list = g14.GradList(xs), g14.GradList(outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        total, each = g14.grad_norm(grads, each=True)
        norm = g14.clip_grad_norm(grads, 1.0, scale=0.5, out=out_list)
        g14.clip_grad_norm(grads, 2.0)
    for seed in (5, 6):
        new, _ = tensors_of([(200, 101), (101,), (50000,)] * 30, ["f16", "f32"], seed)
        for x, y in zip(xs, new):
            x.copy_(y)
        true = math.sqrt(math.fsum(squares(x) for x in xs))
        graph.replay()
        torch.cuda.synchronize()
        norm_check(total, true)
        norm_check(norm, 0.5 * true)
        for y, x, z in zip(outs, new, xs):
            out_check(y, x, factor_of(0.5 * true, 1.0, 0.5))
            out_check(z, x, factor_of(true, 2.0, 1.0))


# ---- refusals (host only)

def args_of(*tensors):
    a = (g14.TensorArg * len(tensors))()
    for x, t in zip(a, tensors):
        x.data, x.rows, x.cols, x.ld, x.dtype = t
    return a


GOOD = (P, 4, 8, 8, 1)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n=(1 << 20) + 1), dict(grads=None), dict(norm=0), dict(norm=P + 2), dict(each=P + 1),
    dict(scale=math.inf), dict(scale=math.nan), dict(ws=P + 8),
    dict(grads=(P, 4, 8, 8, 3)), dict(grads=(P, 4, 8, 8, 9)), dict(grads=(P, -1, 8, 8, 1)),
    dict(grads=(P, 4, -8, 8, 1)), dict(grads=(P, 4, 8, 7, 1)), dict(grads=(0, 4, 8, 8, 1)),
    dict(grads=(P + 1, 4, 8, 8, 1)), dict(grads=(P + 2, 4, 8, 8, 0)), dict(grads=(P, 1 << 41, 8, 8, 1)),
    dict(grads=(P, 1 << 40, 1 << 40, 1 << 40, 1)), dict(grads=(P, 1, 1 << 41, 1, 1))])
def test_refusals(bad):
    a = dict(n=1, grads=GOOD, scale=1.0, norm=P, each=P, ws=P, bytes=1 << 30) | bad
    grads = args_of(a["grads"]) if a["grads"] else None
    bad_arg = g14.GEMM14_ERR_INVALID_ARG
    assert g14.grad_norm_raw(a["n"], grads, a["scale"], a["norm"], a["each"], a["ws"], a["bytes"],
                             check=False) == bad_arg
    assert g14.grad_clip_raw(a["n"], grads, None, a["scale"], 1.0, a["norm"], a["each"], a["ws"], a["bytes"],
                             check=False) == bad_arg


@pytest.mark.parametrize("limit", [-1.0, math.nan, -math.inf])
def test_limits_that_are_refused(limit):
    assert g14.grad_clip_raw(1, args_of(GOOD), None, 1.0, limit, P, None, P, 1 << 30,
                             check=False) == g14.GEMM14_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        g14.clip_grad_norm([], limit)


@pytest.mark.parametrize("out", [(P, 4, 7, 8, 1), (P, 3, 8, 8, 1), (P, 4, 8, 8, 2), (P, 4, 8, 7, 1), (0, 4, 8, 8, 1),
                                 (P + 0x1001, 4, 8, 8, 1), (P + 0x1002, 4, 8, 8, 0)])
def test_outputs_that_are_refused(out):
    assert g14.grad_clip_raw(1, args_of(GOOD), args_of(out), 1.0, 1.0, P, None, P, 1 << 30,
                             check=False) == g14.GEMM14_ERR_INVALID_ARG


Q = P + 0x10000


@pytest.mark.parametrize("grads,outs", [
    ([GOOD, GOOD], None),                                                # twice the same
    ([(P, 1, 100, 100, 1), (P + 198, 1, 4, 4, 1)], None),               # the last element
    ([(P, 10, 20, 64, 1), (P + 38, 10, 20, 64, 1)], None),              # columns of one matrix that cross
    ([(P, 10, 20, 64, 1), (P + 100, 10, 20, 64, 1)], None),             # ... over a row's end
    ([(P, 10, 20, 64, 1), (P + 40, 10, 20, 63, 1)], None),              # of other pitches
    ([GOOD, (Q, 4, 8, 8, 1)], [(Q, 4, 8, 8, 1), (P, 4, 8, 8, 1)]),       # each other's
    ([GOOD, (Q, 4, 8, 8, 1)], [(P + 0x1000, 4, 8, 8, 1)] * 2),           # one output for both
    ([GOOD], [(P, 4, 8, 8, 0)]),                                         # fp32 over its own 16 bits
    ([(P, 4, 8, 16, 1)], [(P, 4, 8, 24, 1)]),                            # another pitch over itself
    ([GOOD], [(P + 2, 4, 8, 8, 1)])])
def test_memory_that_is_shared_is_refused(grads, outs):
    st = g14.grad_clip_raw(len(grads), args_of(*grads), args_of(*outs) if outs else None, 1.0, 1.0, P + 0x100000, None,
                           P + 0x200000, 1 << 30, check=False)
    assert st == g14.GEMM14_ERR_INVALID_ARG and "share memory" in g14.last_error_string()


@pytest.mark.parametrize("grads,outs", [
    ([(P, 10, 20, 64, 1), (P + 40, 10, 20, 64, 1), (P + 80, 10, 24, 64, 1)], None),  # columns side by side
    ([GOOD], [GOOD]), ([GOOD, GOOD], [(Q, 4, 8, 8, 0), (Q + 128, 4, 8, 8, 1)]),      # read twice
    ([(P + 64, 4, 8, 8, 1), GOOD], None)])
def test_memory_that_is_not_shared_passes(grads, outs):
    """(Without a GPU the call then ends at the device.)"""
    st = g14.grad_clip_raw(len(grads), args_of(*grads), args_of(*outs) if outs else None, 1.0, 1.0, P + 0x100000, None,
                           None, 0, check=False)
    assert "share memory" not in g14.last_error_string() or st != g14.GEMM14_ERR_INVALID_ARG


@pytest.mark.parametrize("grads,outs,shared", [
    ([(P, 10, 20, 64, 1), (P + 40, 1, 44, 44, 1)], None, False),      # a row behind a row of columns, up to the next
    ([(P, 10, 20, 64, 1), (P + 40, 1, 44, 7, 1)], None, False),       # (one row has no pitch)
    ([(P, 10, 20, 64, 1), (P + 8 * 128 + 42, 1, 43, 43, 1)], None, False),  # behind the last row but one
    ([(P, 10, 20, 64, 1), (P + 9 * 128 + 40, 1, 500, 500, 1)], None, False),  # behind the last
    ([(P + 128, 10, 20, 64, 1), (P, 1, 64, 64, 1)], None, False),     # before the first
    ([(P, 10, 20, 64, 1), (P + 40, 1, 22, 22, 0)], None, False),      # of another type
    ([(P, 10, 20, 64, 1), (P + 38, 1, 4, 4, 1)], None, True),         # from a row's last element
    ([(P, 10, 20, 64, 1), (P + 40, 1, 45, 45, 1)], None, True),       # into the next row
    ([(P, 10, 20, 64, 1), (P + 40, 1, 1000, 1000, 1)], None, True),   # over several
    ([(P, 10, 20, 64, 1), (P + 9 * 128 + 38, 1, 4, 4, 1)], None, True),  # the last row's last element
    ([(P + 126, 10, 20, 64, 1), (P, 1, 64, 64, 1)], None, True),      # before the first, and its first
    ([(P, 1, 100, 100, 1), (P + 150, 3, 5, 64, 1)], None, True),      # rows that begin within a single one
    ([(P, 10, 20, 64, 1), (P + 40, 10, 20, 128, 1)], None, True),     # another pitch is refused
    ([(P, 10, 20, 64, 1)], [(Q, 10, 20, 64, 0)], False),
    ([(P, 10, 20, 64, 1), (P + 40, 1, 44, 44, 1)], [(Q, 10, 20, 64, 1), (P + 168, 1, 44, 44, 1)], False),
    ([(P, 10, 20, 64, 1), (P + 40, 1, 44, 44, 1)], [(Q, 10, 20, 64, 1), (P + 160, 1, 44, 44, 1)], True)])
def test_a_row_between_rows(grads, outs, shared):
    """(Without a GPU a call that passes ends at the device, with one at its workspace.)"""
    g14.grad_clip_raw(1, args_of(GOOD), args_of((P, 4, 7, 8, 1)), 1.0, 1.0, P, None, P, 0, check=False)
    assert "share memory" not in g14.last_error_string()
    st = g14.grad_clip_raw(len(grads), args_of(*grads), args_of(*outs) if outs else None, 1.0, 1.0, P + 0x100000, None,
                           None, 0, check=False)
    assert st != g14.GEMM14_OK and ("share memory" in g14.last_error_string()) == shared


@pytest.mark.gpu
def test_a_row_beside_columns_is_clipped():
    """A matrix's first columns and, in the same memory, a vector behind one of its rows."""
    for pick in (slice(0, 1), slice(4, 5), slice(39, 40)):
        x = torch.randn(40, 30, device="cuda")
        old, vector = x.clone(), torch.zeros(40, 30, dtype=torch.bool, device="cuda")
        vector[pick, 10:] = True
        vector[:, :10] = True
        true = math.sqrt(squares(old[vector]))
        norm_check(g14.clip_grad_norm([x[pick, 10:], x[:, :10]], 1.0), true)
        out_check(x[vector], old[vector], 1.0 / true)
        assert torch.equal(x[~vector], old[~vector])


def test_stores_of_32_bytes_stand_in_kernels():
    """What the kernels are built of is inlined, but for the function that stores single elements."""
    import os
    import re

    from dense_gemm_14_gb300 import build
    log = os.path.join(build.BUILD_DIR, "grad_norm.ptxas.log")
    if not os.path.exists(log):
        pytest.skip("the build has left no log")
    text = open(log).read()
    kernels = set(re.findall(r"Compiling entry function '(\w+)'", text))
    functions = set(re.findall(r"Function properties for (\w+)", text)) - kernels
    assert kernels and all("scale_small" in f for f in functions), functions


def test_workspace_sizes():
    need = g14.grad_workspace_bytes
    assert need(0, 152) == 0 and need(-1, 152) == 0 and need((1 << 20) + 1, 152) == 0
    assert 0 < need(1, 152) <= need(576, 152) < need(1 << 20, 152) < 1 << 20


@pytest.mark.gpu
def test_small_workspace_is_refused():
    x, norm = torch.randn(100, device="cuda"), torch.zeros((), device="cuda")
    grads = g14.GradList([x])
    need = g14.grad_workspace_bytes(1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for ptr, n in ((ws.data_ptr(), need - 1), (None, 0)):
        assert g14.grad_norm_raw(1, grads._args, 1.0, norm.data_ptr(), None, ptr, n,
                                 check=False) == g14.GEMM14_ERR_INVALID_ARG
        assert str(need) in g14.last_error_string()


def test_tensor_call_refusals():
    x = torch.randn(8)
    with pytest.raises(ValueError):
        g14.grad_norm([x])  # not on a GPU
    with pytest.raises(TypeError):
        g14.GradList([x.double()])


@pytest.mark.gpu
def test_tensor_call_refusals_on_the_gpu():
    x = torch.randn(40, 30, device="cuda")
    for bad in (x[:, ::7], x[0].expand(5, 30), x.unfold(1, 4, 2)):
        with pytest.raises(ValueError):
            g14.GradList([bad])
    with pytest.raises(ValueError):
        g14.clip_grad_norm([x, x], 1.0)
    with pytest.raises(ValueError):
        g14.clip_grad_norm([x, x[3]], 1.0)
    with pytest.raises(ValueError):
        g14.grad_norm([x], scale=math.inf)
    for out in ([], [x.bfloat16()], [torch.empty(30, 40, device="cuda")], [torch.empty(30, 40, device="cuda").t()], [x[:39]]):
        with pytest.raises(ValueError):
            g14.clip_grad_norm([x], 1.0, out=out)
    left, right = x[:, :10], x[:, 10:]
    old = x.clone()
    true = math.sqrt(squares(x))
    norm_check(g14.clip_grad_norm([left, right], 1.0), true)
    out_check(x, old, 1.0 / true)
