"""g.rotary of a tensor that requires a gradient: the rotation is linear, and its gradient is the inverse rotation
of the incoming one, with the same rounding."""
import pytest
import torch

import gqa_decode_blackwell_gb300 as g
from gqa_decode_blackwell_gb300 import build as gbuild
from tests.test_paged import BF16, FP16, FP32, _check_turned, _ints, _randn, _turned

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gbuild.build()
    return torch.device("cuda:0")


def _inputs(dev, dtype, dim=48, T=5):
    x, w = _randn(dev, T, 2, 64, dtype=dtype, seed=2), _randn(dev, T, 2, 64, dtype=dtype, seed=3)
    return x.requires_grad_(), w, _ints(dev, [0, 1, 77, 1000, 123456][:T]), g.rotary_turns(dim, device=dev)


@gpu
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(dev, dtype, inverse, interleaved):
    x, w, positions, turns = _inputs(dev, dtype)
    kw = dict(interleaved=interleaved, inverse=inverse, magnitude=0.75)
    y = g.rotary(x, positions, turns, **kw)
    assert y.requires_grad
    y.backward(w)
    _check_turned(x.grad, _turned(w, positions, turns, interleaved, not inverse, 0.75))
    with torch.no_grad():
        assert torch.equal(y, g.rotary(x, positions, turns, **kw))
        assert torch.equal(x.grad, g.rotary(w, positions, turns, **{**kw, "inverse": not inverse}))
    assert not g.rotary(x.detach(), positions, turns, **kw).requires_grad


@gpu
def test_gradient_of_views_and_of_broadcast_ones(dev):
    """Heads out of one projection's output, and incoming gradients without strides of their own."""
    qkv = _randn(dev, 5, 6, 64, dtype=FP32, seed=4).requires_grad_()
    _, _, positions, turns = _inputs(dev, FP32)
    g.rotary(qkv[:, 2:4], positions, turns).sum().backward()           # an expanded gradient of ones
    want, tol = _turned(torch.ones(5, 2, 64, device=dev), positions, turns, inverse=True)
    _check_turned(qkv.grad[:, 2:4], (want, tol))
    assert (qkv.grad[:, :2] == 0).all() and (qkv.grad[:, 4:] == 0).all()
    qkv.grad = None
    g.rotary(qkv[:, 2:4], positions, turns).transpose(0, 1).contiguous().backward(torch.ones(2, 5, 64, device=dev))
    _check_turned(qkv.grad[:, 2:4], (want, tol))


@gpu
def test_gradient_of_the_gradient(dev):
    """d/dw of the sum of u grad is the rotation of u."""
    x, w, positions, turns = _inputs(dev, FP32)
    w.requires_grad_()
    (grad,) = torch.autograd.grad(g.rotary(x, positions, turns), x, w, create_graph=True)
    u = _randn(dev, *x.shape, dtype=FP32, seed=5)
    (again,) = torch.autograd.grad(grad, w, u)
    assert torch.equal(again, g.rotary(u, positions, turns))


@gpu
@pytest.mark.parametrize("raw", [False, True])
def test_gradient_on_another_stream(dev, raw):
    """The backward pass runs on the stream of the forward one, and the engine waits for both sides."""
    x, w, positions, turns = _inputs(dev, BF16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y = g.rotary(x, positions, turns, stream=s.cuda_stream if raw else s)
    torch.cuda.current_stream().wait_stream(s)
    y.backward(w)
    torch.cuda.synchronize()
    assert torch.equal(x.grad, g.rotary(w, positions, turns, inverse=True))


@gpu
def test_gradient_in_a_graph(dev):
    """Forward and backward captured together and replayed with other values, while an eager graph of other leaves lives."""
    x, w, positions, turns = _inputs(dev, BF16)
    other = g.rotary(_randn(dev, 5, 2, 64, seed=9).requires_grad_(), positions, turns)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                                      # warm-up, as captures of gradients need it
        torch.autograd.grad(g.rotary(x, positions, turns), x, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = g.rotary(x, positions, turns)
        (grad,) = torch.autograd.grad(y, x, w)
    with torch.no_grad():
        x.copy_(_randn(dev, 5, 2, 64, seed=6))
        w.copy_(_randn(dev, 5, 2, 64, seed=7))
        positions.copy_(_ints(dev, [5, 4, 3, 2, 1]))
    graph.replay()
    torch.cuda.synchronize()
    with torch.no_grad():
        assert torch.equal(y, g.rotary(x, positions, turns))
        assert torch.equal(grad, g.rotary(w, positions, turns, inverse=True))
    assert other.requires_grad


@gpu
def test_refusals_are_the_same_with_a_gradient(dev):
    x, _, positions, turns = _inputs(dev, BF16)
    for bad in (None, positions.long(), positions[:-1], positions.cpu(), "a tensor"):
        errors = []
        for t in (x, x.detach()):
            with pytest.raises((TypeError, ValueError)) as e:
                g.rotary(t, bad, turns)
            errors.append((type(e.value), str(e.value)))
        assert errors[0] == errors[1]
    with pytest.raises(g.GQAError):
        g.rotary(x, positions, turns, magnitude=-1.0)
