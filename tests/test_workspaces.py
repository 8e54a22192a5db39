"""The workspaces that the tensor-level calls keep for each (device, stream):
host threads that call on one stream at once, the stream a workspace is made on, and graphs being captured."""
import contextlib
import threading
import time

import pytest
import torch

import dense_gemm_14_gb300 as g14
from dense_gemm_14_gb300 import api, training


def in_threads(*bodies):
    errors = []

    def run(body):
        try:
            body()
        except BaseException as e:  # noqa: BLE001 - reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(b,)) for b in bodies]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors, errors
    assert not any(t.is_alive() for t in threads)


def test_launches_of_two_threads_on_one_stream_do_not_interleave(monkeypatch):
    """A call's launches hand data on through the stream's workspace: none of another
    thread's call may come between them. Calls on two streams do not wait for each other."""
    device = torch.device("cuda", 0)
    monkeypatch.setattr(api, "_workspaces", {})
    monkeypatch.setattr(training, "_workspaces", api._workspaces)
    for handle in (7, 8):
        api._workspaces[(0, handle)] = torch.empty(64, dtype=torch.uint8)
    launches = []

    def call_of(name):
        def call(pointer, size):
            for _ in range(4):
                launches.append(name)
                time.sleep(0.005)
            return g14.GEMM14_OK
        return call

    def body(name, handle):
        return lambda: [training._in_workspace(device, handle, call_of(name), lambda: 64, name)
                        for _ in range(5)]

    in_threads(body("a", 7), body("b", 7))
    assert len(launches) == 40
    for i in range(0, 40, 4):
        assert len(set(launches[i:i + 4])) == 1, launches
    # two streams: each of the two calls waits for the other to have begun
    begun = {7: threading.Event(), 8: threading.Event()}

    def meet(handle, other):
        def call(pointer, size):
            begun[handle].set()
            return g14.GEMM14_OK if begun[other].wait(10) else g14.GEMM14_ERR_TIMEOUT
        return lambda: training._in_workspace(device, handle, call, lambda: 64, "meeting")

    in_threads(meet(7, 8), meet(8, 7))


@pytest.mark.parametrize("current", [0, 7])
def test_a_workspace_is_made_on_the_stream_that_uses_it(current, monkeypatch):
    """Its zero fill would else run on the current stream, after calls on the other had begun."""
    stack = [current]

    @contextlib.contextmanager
    def stream(handle):
        stack.append(handle)
        yield
        stack.pop()

    made = []

    def zeros(n, dtype=None, device=None):
        made.append((n, stack[-1]))
        return torch.empty(n, dtype=dtype)

    monkeypatch.setattr(api, "_workspaces", {})
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: stack[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch, "zeros", zeros)
    device = torch.device("cuda", 0)
    small = api._workspace(device, 7, 64)
    assert api._workspace(device, 7, 32) is small
    assert api._workspace(device, 7, 128).numel() == 128
    assert made == [(64, 7), (128, 7)]


@pytest.mark.gpu
def test_a_product_on_a_given_stream_waits_for_nothing_on_the_current_one():
    """gemm_into's first call on a stream of its own, with the current stream held up: the
    stream's workspace is zero before the product's split tiles use it."""
    a = torch.randn(2304, 4096, device="cuda").bfloat16()
    b = torch.randn(4096, 2560, device="cuda").bfloat16()
    want = g14.gemm(a, b)
    side = torch.cuda.Stream()
    got = torch.empty_like(want)
    dirt = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del dirt  # what the allocator hands out next holds no zeros
    torch.cuda._sleep(1_000_000_000)  # about half a second
    g14.gemm_into(a, b, got, stream=side)
    side.synchronize()
    busy = not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    assert g14.check_device_error(side.cuda_stream) == 0
    assert busy and torch.equal(got, want)


@pytest.mark.gpu
def test_threads_on_one_stream_give_what_each_gives_alone():
    def step(T, V, D, dtype, mode, seed):
        g = torch.Generator().manual_seed(seed)
        h = torch.randn(T, D, generator=g).to(dtype).cuda()
        w = (torch.randn(V, D, generator=g) / D ** 0.5).to(dtype).cuda()
        y = torch.randint(0, V, (T,), generator=g).cuda()
        up = torch.full((T,), 1.0 / T, device="cuda")

        def run():
            loss, lse = g14.linear_cross_entropy(h, w, y, fp32_mode=mode)
            return (loss, lse) + g14.linear_cross_entropy_backward(h, w, y, lse, up, fp32_mode=mode)
        return run

    def product():
        g = torch.Generator().manual_seed(9)
        a = torch.randn(515, 1001, generator=g).cuda()  # copied and split in the workspace
        b = torch.randn(1001, 333, generator=g).cuda()
        return lambda: (g14.gemm(a, b, fp32_mode="3xtf32"),)

    def gradient():
        g = torch.Generator().manual_seed(10)
        c = g14.ckpt8_save(torch.randn(700, 520, generator=g).bfloat16().cuda())
        dy = torch.randn(700, 264, generator=g).bfloat16().cuda()
        return lambda: (g14.ckpt8_weight_grad(dy, c),)

    work = [step(300, 3000, 136, torch.bfloat16, None, 1), step(700, 1031, 72, torch.float16, None, 2),
            step(60, 2000, 65, torch.float32, "3xtf32", 3), product(), gradient()]
    want = [run() for run in work]
    torch.cuda.synchronize()
    got = [[] for _ in work]
    in_threads(*[lambda i=i, run=run: got[i].extend(run() for _ in range(30))
                 for i, run in enumerate(work)])
    torch.cuda.synchronize()
    assert g14.check_device_error(torch.cuda.current_stream().cuda_stream) == 0
    for a, rounds in zip(want, got):
        assert len(rounds) == 30
        for b in rounds:
            for x, z in zip(a, b):
                assert torch.equal(x, z)


def test_a_captured_call_takes_no_kept_workspace_and_keeps_none(monkeypatch):
    """A graph holds its workspace's address: one kept for the stream may be replaced (and its
    memory given away) before a replay, or be used beside it; one made during the capture is
    zero-filled by the graph alone."""
    device = torch.device("cpu")
    kept = torch.full((256,), 0xff, dtype=torch.uint8)
    monkeypatch.setattr(api, "_workspaces", {(None, 7): kept})
    monkeypatch.setattr(training, "_workspaces", api._workspaces)
    monkeypatch.setattr(api, "_current", lambda d, h: contextlib.nullcontext(), raising=False)
    monkeypatch.setattr(api, "_graph_workspaces", {}, raising=False)
    captures = []
    monkeypatch.setattr(api._lib, "capture_id", lambda stream: captures[-1], raising=False)
    for module in (api, training):
        monkeypatch.setattr(module, "_capturing", lambda: True, raising=False)
    given = []

    def call(pointer, size):
        given.append((pointer, size))
        return g14.GEMM14_OK if size >= 128 else g14.GEMM14_ERR_INVALID_ARG

    for capture, n in ((1, 256), (1, 128), (1, 512), (2, 128), (2, 128)):
        captures.append(capture)
        training._in_workspace(device, 7, call, lambda: n, "a call")
    assert [size for _, size in given] == [256, 256, 512, 128, 128]  # one for a capture, while it is enough
    assert all(pointer != kept.data_ptr() for pointer, _ in given)
    assert api._workspaces == {(None, 7): kept}


@pytest.mark.gpu
@pytest.mark.parametrize("warm", [False, True])
def test_graphs_and_larger_calls_on_one_stream(warm):
    """Two graphs captured on one stream, larger calls on it afterwards, and what the allocator
    then makes of smaller workspaces' memory: replays of both graphs at once, on streams of
    their own, give what the calls gave, and nothing else is written."""
    def data(T, V, seed):
        g = torch.Generator().manual_seed(seed)
        return (torch.randn(T, 136, generator=g).bfloat16().cuda(),
                (torch.randn(V, 136, generator=g) / 12.0).bfloat16().cuda(),
                torch.randint(0, V, (T,), generator=g).cuda(), torch.full((T,), 1.0 / T, device="cuda"))

    a = torch.randn(2304, 4096, device="cuda").bfloat16()
    b = torch.randn(4096, 2560, device="cuda").bfloat16()

    def calls(h, w, y, up):
        loss, lse = g14.linear_cross_entropy(h, w, y)
        return (loss, lse) + g14.linear_cross_entropy_backward(h, w, y, lse, up) + (g14.gemm(a, b),)

    sets = [data(300, 3000, 1), data(500, 2500, 2)]
    want = [calls(*x) for x in sets]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if warm:
        with torch.cuda.stream(side):
            calls(*sets[1])
    torch.cuda.synchronize()
    graphs, got = [], []
    for x in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got.append(calls(*x))
        graphs.append(graph)
    with torch.cuda.stream(side):  # calls of the same stream, before any replay, and larger ones
        again = calls(*sets[0])
        large = calls(*data(2000, 30000, 3))
        other = [torch.full((1 << 20,), 0x5a, dtype=torch.uint8, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    for x, z in zip(want[0], again):
        assert torch.equal(x, z)
    assert all(bool(torch.isfinite(x).all()) for x in large)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                for x in got[i]:
                    x.fill_(float("nan"))
                graphs[i].replay()
        with torch.cuda.stream(side):
            again = calls(*sets[0])
        torch.cuda.synchronize()
        for w_, g_ in list(zip(want, got)) + [(want[0], again)]:
            for x, z in zip(w_, g_):
                assert torch.equal(x, z)
    assert all(bool((o == 0x5a).all()) for o in other)
    assert g14.check_device_error(side.cuda_stream) == 0
