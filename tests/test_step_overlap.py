"""The calls of a training step's ends at once and in turn: from several threads on
streams of their own, in graphs replayed between other calls, and what the scaling
stores where an output begins anywhere. Equality is exact: a call repeats bit for bit,
and half of a 16-bit value is a float32."""
import math
import threading

import pytest
import torch

import dense_gemm_14_gb300 as g14

# one launch, two, three for the clipping; and a list with more than one launch a pass
LISTS = [[(33,), (7, 9)], [(200, 101)] * 8, [(640, 1000)] * 5, [(640, 1000), (1001,)] * 60, [(65,)] * 600]


def tensors(shapes, seed, dtype=torch.bfloat16):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(s, generator=g, device="cuda").to(dtype) for s in shapes]


@pytest.mark.gpu
@pytest.mark.parametrize("shapes", LISTS, ids=range(len(LISTS)))
def test_graphs_and_eager_calls_in_turn(shapes):
    xs = [tensors(shapes, 1), tensors(shapes, 2, torch.float32)]
    outs = [[torch.empty_like(x, dtype=torch.float32) for x in part] for part in xs]
    graphs = []
    for part, out in zip(xs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm, each = g14.clip_grad_norm(part, 0.5, scale=0.25, out=out, each=True)
        graphs.append((graph, norm, each))
    for turn in range(3):
        wants = []
        for k, part in enumerate(xs):
            for x, y in zip(part, tensors(shapes, 10 * turn + k + 3, part[0].dtype)):
                x.copy_(y)
            clipped = [torch.empty_like(x, dtype=torch.float32) for x in part]
            wants.append((clipped, *g14.clip_grad_norm(part, 0.5, scale=0.25, out=clipped, each=True)))
        for graph, *_ in graphs:
            graph.replay()
        other = g14.grad_norm(xs[1])
        for (_, norm, each), out, (clipped, n, e) in zip(graphs, outs, wants):
            assert torch.equal(norm, n) and torch.equal(each, e)
            assert all(torch.equal(a, b) for a, b in zip(out, clipped))
        assert torch.equal(other * 0.25, wants[1][1])


@pytest.mark.gpu
def test_threads_on_streams_of_their_own():
    jobs = []
    for k, (T, V, D, shapes) in enumerate([(300, 90, 264, LISTS[0]), (3000, 4000, 520, LISTS[1]),
                                           (9000, 700, 136, LISTS[2]), (20000, 9000, 64, LISTS[3])]):
        g = torch.Generator("cuda").manual_seed(k)
        tokens = torch.randint(0, V, (T,), generator=g, device="cuda") // 2 * 2  # every other row stays empty
        jobs.append((torch.randn(T, D, generator=g, device="cuda").bfloat16(), tokens, V,
                     tensors(shapes, k), [torch.empty(s, device="cuda") for s in shapes]))

    def step(dy, tokens, V, xs, outs):
        dw = g14.embedding_backward(dy, tokens, rows=V, dtype=torch.float32)
        g14.embedding_backward(dy, tokens, out=dw, beta=1.0)
        norm, each = g14.clip_grad_norm(xs + [dw], 1.0, out=outs + [torch.empty_like(dw)], each=True)
        return [dw, norm, each, g14.embedding(dw, tokens), *(x.clone() for x in outs)]

    wants = [step(*job) for job in jobs]
    torch.cuda.synchronize()
    failed = []

    def run(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(8):
                    got = step(*jobs[k])
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, wants[k])):
                        failed.append(f"job {k}: another result")
        except Exception as e:  # noqa: BLE001 (told to the test's thread)
            failed.append(f"job {k}: {e!r}")

    threads = [threading.Thread(target=run, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 3])
def test_every_value_is_stored_wherever_an_output_begins(dtype, rows):
    lengths = [1, 7, 8, 9, 63, 100, 255, 2047, 2048, 2049, 4096, 4159, 6200]
    for offset in (0, 1, 2, 3, 5, 8, 31, 33, 63):
        xs, outs, whole = [], [], []
        for i, n in enumerate(lengths):
            x = torch.randn(rows * (n + 8) + 8, generator=torch.Generator().manual_seed(i)).to(dtype).cuda()
            y = torch.full((rows * (n + 8) + 128,), math.nan, device="cuda")
            xs.append(x[i % 8:i % 8 + rows * (n + 8)].view(rows, n + 8)[:, :n])
            whole.append(y)
            outs.append(y[offset:offset + rows * (n + 8)].view(rows, n + 8)[:, :n])
        for few in (slice(0, 4), slice(None)):
            for y in whole:
                y.fill_(math.nan)
            g14.clip_grad_norm(xs[few], math.inf, scale=0.5, out=outs[few])
            for x, y, w in zip(xs[few], outs[few], whole[few]):
                assert torch.equal(y, x.float() * 0.5), (offset, x.shape)
                y.fill_(math.nan)
                assert bool(torch.isnan(w).all()), "written beside the output"
