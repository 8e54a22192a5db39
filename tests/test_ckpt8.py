"""Activations kept in 8 bits (gemm14_ckpt8_save / _restore) and the weight
gradient formed from them (gemm14_ckpt8_wgrad). The format is exact: q and the
scale bytes are compared with the header's rule carried out in Python
rationals' arithmetic (64-bit floats, which hold every step exactly), and
restored values with q 2^(s - 133). The product is held to the library's fp32
bound |dW - alpha dY^T X - beta dW0| <= 1e-5 (|alpha| |dY|^T|X| + |beta dW0|)
against the restored values (fp32 accumulation; the restored values enter it
exactly)."""
import numpy as np
import pytest
import torch

import dense_gemm_14_gb300 as g14

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODE = {"f32": 0, "bf16": 1, "f16": 2}
P = 0x10000


def rule(x: torch.Tensor):
    """(q, s) of x by the header's rule."""
    x = x.cpu().double().numpy()
    rows, cols = x.shape
    blocks = -(-cols // 32)
    q = np.zeros((rows, cols), np.int8)
    s = np.zeros((rows, blocks), np.uint8)
    for b in range(blocks):
        part = x[:, 32 * b:32 * b + 32]
        top = np.abs(part).max(axis=1)
        bad = ~np.isfinite(part).all(axis=1)
        with np.errstate(all="ignore"):
            e = np.frexp(np.where(bad, 1.0, top))[1] + 126  # exponent field of an fp32
        e = np.where(top == 0, 7, np.clip(e, 7, 254))
        step = np.ldexp(1.0, 133 - e)[:, None]
        with np.errstate(all="ignore"):
            v = np.clip(np.rint(np.where(bad[:, None], 0.0, part) * step), -127, 127)
        q[:, 32 * b:32 * b + 32] = v
        s[:, b] = np.where(bad, 255, e)
    return q, s


def values(q, s):
    """What q and s stand for, in 64 bits."""
    rows, cols = q.shape
    step = np.where(s == 255, np.nan, np.ldexp(1.0, np.maximum(s.astype(np.int64), 7) - 133))
    return q.astype(np.float64) * np.repeat(step, 32, axis=1)[:, :cols]


def data(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x[torch.rand(rows, cols, generator=g) < 0.1] = 0.0
    return x.to(DT[dtype])


def view_of(x, pad, offset):
    rows, cols = x.shape
    buf = torch.zeros(offset + rows * (cols + pad) + 64, dtype=x.dtype, device="cuda")
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(x.cuda())
    return v


def check(x, c, dtype):
    q, s = rule(x)
    assert np.array_equal(c.scale.cpu().numpy(), s)
    assert np.array_equal(c.q.cpu().numpy(), q)
    want = torch.from_numpy(values(q, s))
    for out in (torch.float32, torch.bfloat16, DT[dtype]):
        got = g14.ckpt8_restore(c, out).cpu()
        assert torch.equal(torch.nan_to_num(got.double(), nan=7e300, posinf=None),
                           torch.nan_to_num(want, nan=7e300)), out
    assert torch.equal(torch.isnan(g14.ckpt8_restore(c, torch.float16)).cpu(), torch.isnan(want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (1, 32), (3, 33), (7, 64), (5, 100),
                                       (2, 4096), (129, 1001), (1000, 256), (3001, 96), (64, 1000)])
def test_save_and_restore_follow_the_format(rows, cols, dtype):
    x = data(rows, cols, dtype, rows + cols)
    check(x, g14.ckpt8_save(x.cuda()), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 5), (8, 8), (16, 0)])
def test_save_reads_any_pitch_and_offset(pad, offset, dtype):
    x = data(61, 224, dtype, pad + offset)
    check(x, g14.ckpt8_save(view_of(x, pad, offset)), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("ldq,q_off,lds,s_off", [(225, 0, 8, 0), (224, 1, 7, 0), (240, 16, 7, 3),
                                                 (232, 8, 9, 1), (228, 4, 16, 0)])
def test_any_pitch_of_the_kept_form(ldq, q_off, lds, s_off):
    x = data(61, 224, "bf16", 3).cuda()
    qbuf = torch.full((q_off + 61 * ldq,), 99, dtype=torch.int8, device="cuda")
    sbuf = torch.full((s_off + 61 * lds,), 99, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    g14.ckpt8_save_raw(1, 61, 224, x.data_ptr(), 224, qbuf.data_ptr() + q_off, ldq,
                       sbuf.data_ptr() + s_off, lds, stream)
    q = qbuf[q_off:].view(61, ldq)
    s = sbuf[s_off:].view(61, lds)
    check(x, g14.Ckpt8(q[:, :224], s[:, :7]), "bf16")
    # nothing beside the rows is written
    assert bool((q[:, 224:] == 99).all()) and bool((s[:, 7:] == 99).all())
    assert bool((qbuf[:q_off] == 99).all()) and bool((sbuf[:s_off] == 99).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_blocks_of_extreme_values(dtype):
    f = torch.finfo(DT[dtype])
    rows = []
    for top in (0.0, f.max, f.min, f.tiny, f.smallest_normal / 2 ** 3, 1.0, 2.0 ** -14, 1.9921875,
                0.99609375, float("inf"), -float("inf"), float("nan"), 2.0 ** 14):
        x = torch.linspace(-1, 1, 64).to(DT[dtype])
        x = x * min(abs(top), 1.0) if np.isfinite(top) else x
        x[40] = top
        rows.append(x.to(DT[dtype]))
    rows.append(torch.full((64,), -0.0, dtype=DT[dtype]))
    rows.append(torch.full((64,), f.max, dtype=DT[dtype]))
    x = torch.stack(rows)
    c = g14.ckpt8_save(x.cuda())
    q, s = rule(x)
    assert np.array_equal(c.scale.cpu().numpy(), s) and np.array_equal(c.q.cpu().numpy(), q)
    want = values(q, s)
    got = g14.ckpt8_restore(c, DT[dtype]).cpu().double().numpy()
    assert np.array_equal(got, want, equal_nan=True)
    # half a step of the block; one step where the largest is held at 127
    x = x.double().numpy()
    for b in range(2):
        part, back = x[:, 32 * b:32 * b + 32], want[:, 32 * b:32 * b + 32]
        fine = np.isfinite(part).all(axis=1)
        step = np.ldexp(1.0, s[fine, b].astype(int) - 133)[:, None]
        held = np.abs(q[fine, 32 * b:32 * b + 32].astype(int)) == 127
        assert (np.abs(part[fine] - back[fine]) <= np.where(held, 1.0, 0.5) * step).all()


def wgrad_check(dy, c, got, alpha=1.0, beta=0.0, dw0=None):
    x = torch.from_numpy(values(c.q.cpu().numpy(), c.scale.cpu().numpy()))
    d = dy.cpu().double()
    want, scale = alpha * (d.t() @ x), abs(alpha) * (d.abs().t() @ x.abs())
    if beta:
        want, scale = want + beta * dw0.double(), scale + (beta * dw0.double()).abs()
    diff = (got.cpu().double() - want).abs()
    assert bool((diff <= 1e-5 * scale + 1e-37).all()), float((diff / (scale + 1e-300)).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,mode", [("bf16", None), ("f16", None), ("f32", None),
                                        ("f32", "3xtf32")])
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 64, 96), (7, 65, 33), (16, 256, 256), (64, 130, 128),
                                   (65, 300, 1001), (100, 33, 2000), (515, 512, 264), (1000, 264, 520),
                                   (2048, 300, 320)])
def test_weight_gradient(T, N, K, dtype, mode):
    x, dy = data(T, K, dtype, T + K), data(T, N, dtype, T + N + 1)
    c = g14.ckpt8_save(x.cuda())
    got = g14.ckpt8_weight_grad(dy.cuda(), c, fp32_mode=mode)
    wgrad_check(dy, c, got)
    dw0 = torch.randn(N, K, generator=torch.Generator().manual_seed(1)) * 10
    out = dw0.cuda()
    g14.ckpt8_weight_grad(dy.cuda(), c, out=out, alpha=-0.5, beta=1.0, fp32_mode=mode)
    wgrad_check(dy, c, out, -0.5, 1.0, dw0)
    assert g14.check_device_error(torch.cuda.current_stream().cuda_stream) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dy_pad,dy_off,q_pad,out_pad", [(1, 0, 0, 0), (0, 1, 5, 0), (8, 8, 16, 4),
                                                         (3, 3, 1, 3)])
def test_weight_gradient_pitches(dy_pad, dy_off, q_pad, out_pad, dtype):
    T, N, K = 130, 200, 224
    x, dy = data(T, K, dtype, 5), data(T, N, dtype, 6)
    c = g14.ckpt8_save(x.cuda())
    c = g14.Ckpt8(view_of(c.q, q_pad, q_pad), view_of(c.scale, q_pad, q_pad))
    buf = torch.full((N, K + out_pad), float("nan"), device="cuda")
    g14.ckpt8_weight_grad(view_of(dy, dy_pad, dy_off), c, out=buf[:, :K])
    wgrad_check(dy, c, buf[:, :K])
    assert bool(torch.isnan(buf[:, K:]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,mode", [("bf16", None), ("f16", None), ("f32", None),
                                        ("f32", "3xtf32")])
@pytest.mark.parametrize("T", [1, 3, 4, 5, 8, 9, 15, 16, 17])
@pytest.mark.parametrize("N,K,pad", [(5, 31, 0), (700, 1500, 0), (257, 1027, 1), (3001, 96, 4)])
def test_weight_gradient_of_a_handful_of_rows(T, N, K, pad, dtype, mode):
    """Rows and columns over several blocks, rows of dW on 16 bytes and not, from an
    offset and with room beside them that stays as it is."""
    x, dy = data(T, K, dtype, T + K), data(T, N, dtype, T + N + 1)
    c = g14.ckpt8_save(x.cuda())
    dyv = view_of(dy, pad, pad)
    for off in (0, 1):
        buf = torch.full((N * (K + pad) + 8,), float("nan"), device="cuda")
        out = buf[off:off + N * (K + pad)].view(N, K + pad)
        g14.ckpt8_weight_grad(dyv, c, out=out[:, :K], fp32_mode=mode)  # NaN there is not read
        wgrad_check(dy, c, out[:, :K])
        before = out[:, :K].cpu()
        g14.ckpt8_weight_grad(dyv, c, out=out[:, :K], alpha=-0.5, beta=0.75, fp32_mode=mode)
        wgrad_check(dy, c, out[:, :K], -0.5, 0.75, before)
        assert bool(torch.isnan(out[:, K:]).all()) and bool(torch.isnan(buf[off + N * (K + pad):]).all())
        assert off == 0 or bool(torch.isnan(buf[:off]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [16, 40])
def test_f16_values_beyond_its_range_enter_as_infinities(T):
    x = torch.ones(T, 64)
    x[:, 32:] = 1e6  # kept from fp32; beyond fp16's range
    c = g14.ckpt8_save(x.cuda())
    got = g14.ckpt8_weight_grad(torch.ones(T, 8, dtype=torch.float16, device="cuda"), c).cpu()
    assert bool((got[:, :32] == float(T)).all()) and bool((got[:, 32:] == float("inf")).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_a_poisoned_block_in_a_handful_of_rows(dtype):
    x, dy = data(9, 96, dtype, 1), data(9, 70, dtype, 2)
    x[3, 35] = float("nan")
    c = g14.ckpt8_save(x.cuda())
    got = g14.ckpt8_weight_grad(dy.cuda(), c).cpu()
    assert bool(torch.isnan(got[:, 32:64]).all())
    assert not bool(torch.isnan(got[:, :32]).any()) and not bool(torch.isnan(got[:, 64:]).any())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_poisoned_block_reaches_its_columns_only(dtype):
    x, dy = data(40, 96, dtype, 1), data(40, 70, dtype, 2)
    x[3, 35] = float("inf")
    c = g14.ckpt8_save(x.cuda())
    got = g14.ckpt8_weight_grad(dy.cuda(), c).cpu()
    assert bool(torch.isnan(got[:, 32:64]).all())
    assert not bool(torch.isnan(got[:, :32]).any()) and not bool(torch.isnan(got[:, 64:]).any())


@pytest.mark.gpu
def test_f16_rounds_only_outside_its_range():
    """An fp16 activation kept and multiplied with an fp16 dY: the values enter exactly down to subnormals."""
    x = (data(64, 64, "f32", 1) * 1e-6).half()
    dy = torch.eye(64).half()
    c = g14.ckpt8_save(x.cuda())
    got = g14.ckpt8_weight_grad(dy.cuda(), c).cpu().double().numpy()
    assert np.array_equal(got, values(c.q.cpu().numpy(), c.scale.cpu().numpy()))


@pytest.mark.gpu
def test_degenerate_sizes():
    c = g14.ckpt8_save(torch.empty(0, 64, device="cuda", dtype=torch.bfloat16))
    assert g14.ckpt8_restore(c).shape == (0, 64)
    dy = torch.empty(0, 8, device="cuda", dtype=torch.bfloat16)
    assert not g14.ckpt8_weight_grad(dy, c).any()
    out = torch.full((8, 64), 2.0, device="cuda")
    g14.ckpt8_weight_grad(dy, c, out=out, beta=0.5)
    assert bool((out == 1.0).all())
    c = g14.ckpt8_save(torch.empty(5, 0, device="cuda"))
    assert g14.ckpt8_restore(c, torch.float32).shape == (5, 0)
    # alpha = 0: neither dY nor the checkpoint is read
    c = g14.ckpt8_save(torch.full((4, 64), float("nan"), device="cuda"))
    out.fill_(3.0)
    g14.ckpt8_weight_grad(torch.full((4, 8), float("nan"), device="cuda"), c, out=out, alpha=0.0, beta=2.0)
    assert bool((out == 6.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_weight_gradient_repeats_on_another_stream(dtype):
    x, dy = data(700, 520, dtype, 1).cuda(), data(700, 264, dtype, 2).cuda()
    want = g14.ckpt8_weight_grad(dy, g14.ckpt8_save(x))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = g14.ckpt8_weight_grad(dy, g14.ckpt8_save(x, stream=side), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(want, got)


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """A checkpoint of 2.2e9 values: its last rows are kept, restored and multiplied."""
    rows, cols = 70001, 32768
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = data(8, cols, "bf16", 3)
    x[-8:] = tail.cuda()
    c = g14.ckpt8_save(x)
    q, s = rule(tail)
    assert np.array_equal(c.q[-8:].cpu().numpy(), q) and np.array_equal(c.scale[-8:].cpu().numpy(), s)
    back = g14.ckpt8_restore(c)
    assert torch.equal(back[-8:].cpu().double(), torch.from_numpy(values(q, s)))
    assert not back[:-8].any()
    del back, x
    dy = data(rows, 3, "bf16", 4)
    got = g14.ckpt8_weight_grad(dy.cuda(), c)
    wgrad_check(dy[-8:], g14.Ckpt8(c.q[-8:], c.scale[-8:]), got)


# ---- refusals (host only)

@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=9), dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(ldx=63),
    dict(ldq=63), dict(lds=1), dict(X=0), dict(Q=0), dict(S=0), dict(X=P + 1)])
def test_save_and_restore_refusals(bad):
    a = dict(dtype=1, rows=4, cols=64, X=P, ldx=64, Q=P, ldq=64, S=P, lds=2) | bad
    assert g14.ckpt8_save_raw(a["dtype"], a["rows"], a["cols"], a["X"], a["ldx"], a["Q"], a["ldq"],
                              a["S"], a["lds"], check=False) == g14.GEMM14_ERR_INVALID_ARG
    assert g14.ckpt8_restore_raw(a["dtype"], a["rows"], a["cols"], a["Q"], a["ldq"], a["S"],
                                 a["lds"], a["X"], a["ldx"], check=False) == g14.GEMM14_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [
    dict(dtype=9), dict(T=-1), dict(N=-1), dict(K=1 << 31), dict(lddy=7), dict(ldq=63), dict(lds=1),
    dict(lddw=63), dict(dY=0), dict(Q=0), dict(S=0), dict(dW=0), dict(dY=P + 1), dict(dW=P + 2),
    dict(ws=P + 8)])
def test_weight_gradient_refusals(bad):
    a = dict(dtype=1, T=4, N=8, K=64, dY=P, lddy=8, Q=P, ldq=64, S=P, lds=2, dW=P, lddw=64, ws=P) | bad
    assert g14.ckpt8_wgrad(a["dtype"], a["T"], a["N"], a["K"], 1.0, a["dY"], a["lddy"], a["Q"],
                           a["ldq"], a["S"], a["lds"], 0.0, a["dW"], a["lddw"], a["ws"], 1 << 30,
                           check=False) == g14.GEMM14_ERR_INVALID_ARG


@pytest.mark.parametrize("size", ["T", "N", "K"])
def test_sizes_whose_tiles_pass_32_bits_are_refused(size):
    """Within 255 of 2^31 a count of whole tiles does not fit 32 bits."""
    for n in ((1 << 31) - 255, (1 << 31) - 1):
        a = dict(T=17, N=1, K=1) | {size: n}
        pitch = 1 << 31
        assert g14.ckpt8_wgrad(1, a["T"], a["N"], a["K"], 1.0, P, pitch, P, pitch, P, pitch, 0.0, P,
                               pitch, P, 1 << 30, check=False) == g14.GEMM14_ERR_INVALID_ARG
        assert g14.ckpt8_wgrad_workspace_bytes(1, a["T"], a["N"], a["K"], P, pitch, P, pitch,
                                               152) == 0
    a = dict(T=17, N=1, K=1) | {size: (1 << 31) - 256}
    assert g14.ckpt8_wgrad_workspace_bytes(1, a["T"], a["N"], a["K"], P, pitch, P, pitch, 152) > 0


@pytest.mark.gpu
def test_weight_gradient_small_workspace_is_refused():
    x, dy = data(64, 64, "bf16", 1).cuda(), data(64, 64, "bf16", 2).cuda()
    c = g14.ckpt8_save(x)
    dw = torch.zeros(64, 64, device="cuda")
    need = g14.ckpt8_wgrad_workspace_bytes(1, 64, 64, 64, dy.data_ptr(), 64, dw.data_ptr(), 64)
    if need == 0:
        pytest.skip("this product needs no workspace")
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for ptr, n in ((ws.data_ptr(), need - 1), (None, 0)):
        st = g14.ckpt8_wgrad(1, 64, 64, 64, 1.0, dy.data_ptr(), 64, c.q.data_ptr(), 64,
                             c.scale.data_ptr(), 16, 0.0, dw.data_ptr(), 64, ptr, n, check=False)
        assert st == g14.GEMM14_ERR_INVALID_ARG
        assert str(need) in g14.last_error_string()


def test_tensor_call_refusals():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        g14.ckpt8_save(x)  # not on a GPU
    with pytest.raises(TypeError):
        g14.ckpt8_save(x.double())
    with pytest.raises(TypeError):
        g14.ckpt8_restore(g14.Ckpt8(x.to(torch.int8), torch.zeros(4, 2, dtype=torch.uint8)), torch.int8)
