"""Failure detection of the training products, as for the products: a wait
that nothing completes ends the kernel with an error status, and the context
stays usable. Also their workspaces: shared with the other calls' and by
streams, and the bits they give with whatever was in them."""
import time

import pytest
import torch

import dense_gemm_14_gb300 as g14
from dense_gemm_14_gb300 import training


def ce_inputs(T, dtype, seed=1, V=3000, D=136):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, D, generator=g).to(dtype).cuda()
    w = (torch.randn(V, D, generator=g) / D ** 0.5).to(dtype).cuda()
    y = torch.randint(0, V, (T,), generator=g).cuda()
    return h, w, y, torch.full((T,), 1.0 / T, device="cuda")




def stream_status():
    return g14.check_device_error(torch.cuda.current_stream().cuda_stream)


@pytest.mark.gpu
@pytest.mark.parametrize("T,dtype,mode", [(12, torch.bfloat16, None), (300, torch.float16, None),
                                          (300, torch.float32, "3xtf32"),
                                          (2048, torch.float32, "fp32")])
@pytest.mark.parametrize("backward", [False, True])
def test_expired_wait_in_cross_entropy(T, dtype, mode, backward):
    h, w, y, up = ce_inputs(T, dtype)
    want = g14.linear_cross_entropy(h, w, y, fp32_mode=mode)

    def call():
        if not backward:
            return g14.linear_cross_entropy(h, w, y, fp32_mode=mode)
        return g14.linear_cross_entropy_backward(h, w, y, want[1], up, fp32_mode=mode)

    good = call()
    assert stream_status() == g14.GEMM14_OK
    assert g14.debug_inject(1, 20_000_000) == 0  # 20 ms per wait
    t0 = time.perf_counter()
    call()
    assert stream_status() == g14.GEMM14_ERR_TIMEOUT
    assert time.perf_counter() - t0 < 10.0
    # read and cleared; the request is spent and the next call is right
    again = call()
    assert stream_status() == g14.GEMM14_OK
    for a, b in zip(good, again):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_handful_of_rows_has_no_wait_to_expire():
    """Those calls (CUDA cores, block barriers alone) take the request and compute as usual."""
    h, w, y, up = ce_inputs(3, torch.float32)
    want = g14.linear_cross_entropy(h, w, y)
    assert g14.debug_inject(1, 20_000_000) == 0
    got = g14.linear_cross_entropy(h, w, y)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    g14.linear_cross_entropy(*ce_inputs(300, torch.bfloat16)[:3])
    assert stream_status() == g14.GEMM14_OK


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,mode", [(torch.bfloat16, None), (torch.float32, "3xtf32")])
@pytest.mark.parametrize("T", [40, 2000])
def test_expired_wait_in_weight_gradient(T, dtype, mode):
    g = torch.Generator().manual_seed(3)
    c = g14.ckpt8_save(torch.randn(T, 512, generator=g).to(dtype).cuda())
    dy = torch.randn(T, 264, generator=g).to(dtype).cuda()
    good = g14.ckpt8_weight_grad(dy, c, fp32_mode=mode)
    assert g14.debug_inject(1, 20_000_000) == 0
    g14.ckpt8_weight_grad(dy, c, fp32_mode=mode)
    assert stream_status() == g14.GEMM14_ERR_TIMEOUT
    assert torch.equal(good, g14.ckpt8_weight_grad(dy, c, fp32_mode=mode))
    assert stream_status() == g14.GEMM14_OK


@pytest.mark.gpu
def test_a_weight_gradient_of_a_handful_of_rows_has_no_wait_to_expire():
    g = torch.Generator().manual_seed(3)
    c = g14.ckpt8_save(torch.randn(16, 512, generator=g).half().cuda())
    dy = torch.randn(16, 264, generator=g).half().cuda()
    want = g14.ckpt8_weight_grad(dy, c)
    assert g14.debug_inject(1, 20_000_000) == 0
    assert torch.equal(want, g14.ckpt8_weight_grad(dy, c))
    g14.linear_cross_entropy(*ce_inputs(300, torch.bfloat16)[:3])  # the request is spent
    assert stream_status() == g14.GEMM14_OK


def test_a_refused_call_takes_the_request():
    g14.load()
    assert g14.debug_inject(1, 1000) == 0
    assert g14.linear_ce_forward(1, -1, 8, 8, 0, 8, 0, 8, 0, -100, 0, 0, None, 0, check=False) == 1
    assert g14.gemm_f32(0, 4, 4, 0, 4, 0, 4, 0, 4, None, check=False) == 0
    assert g14.debug_inject(1, 1000) == 0
    assert g14.ckpt8_wgrad(1, -1, 8, 8, 1.0, 0, 8, 0, 8, 0, 1, 0.0, 0, 8, None, 0, check=False) == 1
    assert g14.gemm_f32(0, 4, 4, 0, 4, 0, 4, 0, 4, None, check=False) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,dtype,mode", [(5, torch.bfloat16, None), (300, torch.bfloat16, None),
                                          (300, torch.float32, "3xtf32"), (300, torch.float32, None)])
def test_one_workspace_serves_products_and_training_calls_in_turn(T, dtype, mode):
    """A zeroed workspace is used by a split product, a training call and the
    product again; each gives what it gives with a workspace of its own."""
    h, w, y, up = ce_inputs(T, dtype)
    loss, lse = g14.linear_cross_entropy(h, w, y, fp32_mode=mode)
    dh, dw = g14.linear_cross_entropy_backward(h, w, y, lse, up, fp32_mode=mode)
    code = {torch.bfloat16: 1, torch.float32: 4 if mode else 0}[dtype]
    V, D = w.shape
    n = max(g14.linear_ce_workspace_bytes(code, 1, T, V, D, h.data_ptr(), D, w.data_ptr(), D),
            g14.linear_ce_workspace_bytes(code, 0, T, V, D, h.data_ptr(), D, w.data_ptr(), D))
    a = torch.randn(2304, 4096, device="cuda").bfloat16()
    b = torch.randn(4096, 2560, device="cuda").bfloat16()
    need = g14.workspace_bytes(1, 2304, 2560, 4096, 0)
    assert need > 0
    ws = torch.zeros(max(n, need), dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    want = torch.empty(2304, 2560, device="cuda")
    own = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def product(out, space):
        g14.gemm_bf16_f32acc_ws(2304, 2560, 4096, a.data_ptr(), 4096, b.data_ptr(), 2560,
                                out.data_ptr(), 2560, space.data_ptr(), space.numel(), s)

    product(want, own)
    got = torch.empty_like(want)
    dh2, dw2 = torch.empty_like(dh), torch.empty_like(dw)
    for _ in range(3):
        product(got.fill_(float("nan")), ws)
        assert torch.equal(got, want)
        g14.linear_ce_backward(code, T, V, D, h.data_ptr(), D, w.data_ptr(), D, y.data_ptr(), -100,
                               lse.data_ptr(), up.data_ptr(), dh2.data_ptr(), D, dw2.data_ptr(), D,
                               ws.data_ptr(), ws.numel(), s)
        assert torch.equal(dh, dh2) and torch.equal(dw, dw2)
    assert stream_status() == g14.GEMM14_OK


@pytest.mark.gpu
@pytest.mark.parametrize("T,dtype", [(5, torch.bfloat16), (300, torch.float16), (300, torch.float32)])
def test_what_the_workspace_held_does_not_matter(T, dtype):
    """All but the flag words of the workspace filled with NaN patterns before the call."""
    h, w, y, up = ce_inputs(T, dtype)
    y[::3] = -100
    mode = "3xtf32" if dtype == torch.float32 else None
    code = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 4}[dtype]
    loss, lse = g14.linear_cross_entropy(h, w, y, fp32_mode=mode)
    dh, dw = g14.linear_cross_entropy_backward(h, w, y, lse, up, fp32_mode=mode)
    V, D = w.shape
    n = g14.linear_ce_workspace_bytes(code, 1, T, V, D, h.data_ptr(), D, w.data_ptr(), D)
    ws = torch.full((n,), 0xff, dtype=torch.uint8, device="cuda")
    ws[:4096] = 0
    s = torch.cuda.current_stream().cuda_stream
    dh2, dw2 = torch.empty_like(dh), torch.empty_like(dw)
    g14.linear_ce_backward(code, T, V, D, h.data_ptr(), D, w.data_ptr(), D, y.data_ptr(), -100,
                           lse.data_ptr(), up.data_ptr(), dh2.data_ptr(), D, dw2.data_ptr(), D,
                           ws.data_ptr(), n, s)
    assert torch.equal(dh, dh2) and torch.equal(dw, dw2)
    ws.fill_(0xff)
    ws[:4096] = 0
    out = torch.empty(2, T, device="cuda")
    g14.linear_ce_forward(code, T, V, D, h.data_ptr(), D, w.data_ptr(), D, y.data_ptr(), -100,
                          out.data_ptr(), out.data_ptr() + 4 * T, ws.data_ptr(), n, s)
    assert torch.equal(out[0], loss) and torch.equal(out[1], lse)


@pytest.mark.gpu
def test_calls_on_two_streams_at_once():
    data = [ce_inputs(300, torch.bfloat16, seed=s) for s in (1, 2)]
    want = []
    for h, w, y, up in data:
        loss, lse = g14.linear_cross_entropy(h, w, y)
        want.append((loss, lse) + g14.linear_cross_entropy_backward(h, w, y, lse, up))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(5):
        for i, (h, w, y, up) in enumerate(data):
            loss, lse = g14.linear_cross_entropy(h, w, y, stream=streams[i])
            got[i] = (loss, lse) + g14.linear_cross_entropy_backward(h, w, y, lse, up,
                                                                     stream=streams[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, z in zip(a, b):
            assert torch.equal(x, z)


@pytest.mark.gpu
def test_the_example_learns():
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import train_head
    finally:
        sys.path.pop(0)
    losses = train_head.train(steps=20)
    assert all(x == x for x in losses)
    assert losses[-1] < 0.7 * losses[0], losses


@pytest.mark.parametrize("status", [g14.GEMM14_ERR_TIMEOUT, g14.GEMM14_ERR_CUDA])
def test_a_failed_call_is_reported_and_not_repeated(status, monkeypatch):
    """A call that failed after its launches may have added to its output: only
    one that was refused for its workspace is made again."""
    device, handle = torch.device("cuda", 0), 7
    monkeypatch.setitem(training._workspaces, (device.index, handle),
                        torch.empty(64, dtype=torch.uint8))
    calls = []

    def call(pointer, size):
        calls.append(size)
        return status

    with pytest.raises(g14.Gemm14Error):
        training._in_workspace(device, handle, call, lambda: 128, "a call")
    assert calls == [64]


def test_a_call_refused_for_its_workspace_is_made_again(monkeypatch):
    device, handle = torch.device("cuda", 0), 7
    monkeypatch.setitem(training._workspaces, (device.index, handle),
                        torch.empty(64, dtype=torch.uint8))
    monkeypatch.setattr(training, "_workspace",
                        lambda d, h, n: torch.empty(n, dtype=torch.uint8))
    calls = []

    def call(pointer, size):
        calls.append(size)
        return g14.GEMM14_OK if size >= 128 else g14.GEMM14_ERR_INVALID_ARG

    training._in_workspace(device, handle, call, lambda: 128, "a call")
    assert calls == [64, 128]
