"""Lists of gradients whose tensors are given other memory after the list was made: a
storage that is resized frees the memory that it had, which the allocator gives to
others, so that a call on the old addresses would read and write what is theirs.
Without a GPU the tensors only say that they are on one, and no kernel is called."""
import math

import pytest
import torch

import dense_gemm_14_gb300 as g14
from dense_gemm_14_gb300 import training


class OnGpu(torch.Tensor):
    is_cuda = True


def on_gpu(*shape):
    return torch.randn(*shape).as_subclass(OnGpu)


def grown(x):
    x.resize_(100000)


def freed(x):
    x.untyped_storage().resize_(0)


def freed_and_smaller(x):
    """(An allocator may give the same address again.)"""
    x.untyped_storage().resize_(0)
    x.untyped_storage().resize_(64)


def shrunk(x):
    x.untyped_storage().resize_(200)


def other_data(x):
    x.data = torch.zeros_like(x)


def other_storage(x):
    x.set_(torch.zeros(50))


CHANGES = [grown, freed, freed_and_smaller, shrunk, other_data, other_storage]


@pytest.fixture
def calls(monkeypatch):
    made = []
    monkeypatch.setattr(training, "_grad_call", lambda grads, *a: made.append([x.data for x in grads._args]))
    return made


@pytest.mark.parametrize("change", CHANGES)
@pytest.mark.parametrize("which", [0, 1, 2])
def test_a_list_of_memory_that_is_gone_is_refused(change, which, calls):
    xs = [on_gpu(50), on_gpu(50), on_gpu(50)]
    grads, outs = g14.GradList(xs), g14.GradList([on_gpu(50) for _ in xs])
    g14.grad_norm(grads)
    g14.clip_grad_norm(grads, 1.0)
    g14.clip_grad_norm(outs, 1.0, out=grads)
    assert calls == [[x.data_ptr() for x in xs]] * 2 + [[x.data_ptr() for x in outs.tensors]]
    del calls[:]
    change(xs[which])
    for call in (lambda: g14.grad_norm(grads), lambda: g14.clip_grad_norm(grads, 1.0),
                 lambda: g14.clip_grad_norm(outs, 1.0, out=grads)):
        with pytest.raises(ValueError, match="new GradList"):
            call()
    assert not calls
    if change in (grown, other_data, other_storage):  # a list made anew serves
        again = [x.as_subclass(OnGpu) for x in xs]
        g14.grad_norm(g14.GradList(again))
        assert calls == [[x.data_ptr() for x in xs]]


def test_a_view_of_a_storage_that_is_resized(calls):
    buffer = on_gpu(100)
    grads = g14.GradList([buffer[:40], buffer[50:]])
    g14.grad_norm(grads)
    buffer.resize_(100000)
    with pytest.raises(ValueError, match="new GradList"):
        g14.grad_norm(grads)


def test_what_keeps_the_memory_is_accepted(calls):
    """Values that change, views that go, tensors without elements, a name for another tensor."""
    buffer = on_gpu(100)
    xs = [buffer[:60].view(6, 10), on_gpu(0), on_gpu(3, 0, 2), buffer[60:]]
    grads = g14.GradList(xs)
    want = [x.data_ptr() or None for x in xs]
    buffer.mul_(2.0)
    xs[0].zero_()
    xs[3] = on_gpu(7)
    del buffer, xs
    g14.grad_norm(grads)
    g14.grad_norm(g14.GradList([]))
    assert calls == [want, []]


@pytest.mark.gpu
def test_lists_on_the_gpu():
    xs = [torch.randn(300, 40, device="cuda"), torch.randn(1000, device="cuda"), torch.empty(0, device="cuda")]
    grads = g14.GradList(xs)
    true = math.sqrt(sum(float(x.double().square().sum()) for x in xs))
    assert abs(float(g14.grad_norm(grads)) - true) <= 10.1 * 2.0 ** -24 * true
    old, new = xs[0].clone(), torch.randn(300, 40, device="cuda")
    xs[0].data = new
    for call in (lambda: g14.grad_norm(grads), lambda: g14.clip_grad_norm(grads, 1e-3)):
        with pytest.raises(ValueError, match="tensor 0"):
            call()
    assert float(g14.grad_norm(g14.GradList(xs))) != float(g14.grad_norm([old, *xs[1:]]))
    grads = g14.GradList(xs)
    xs[1].resize_(1 << 22)
    with pytest.raises(ValueError, match="tensor 1"):
        g14.clip_grad_norm(grads, 1e-3)
    xs[2].resize_(5)
    xs[1].resize_(1000).fill_(1.0)
    xs[2].fill_(1.0)
    true = math.sqrt(float(new.double().square().sum()) + 1005)
    assert abs(float(g14.grad_norm(xs)) - true) <= 10.1 * 2.0 ** -24 * true
