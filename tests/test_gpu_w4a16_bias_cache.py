"""AWQLinear's bf16 copy of its bias: a first call that is captured, a bias changed
under a captured call, and first calls on two streams at once."""

import pytest
import torch

from tests.test_gpu_w4a16_modules import linear
from w4a4_quantized_diffusion_amd import linear as L

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
N, K = 256, 128


def layer():
    """(a biased layer, its values on x, x); the library is loaded and warm."""
    mod = L.AWQLinear.from_linear(linear(K, N, 1))
    warm = L.AWQLinear.from_linear(linear(K, N, 1))
    x = torch.randn(4, K, device="cuda").to(BF)
    y = warm(x)
    torch.cuda.synchronize()
    return mod, y, x


def test_first_call_captured():
    """A layer whose first call is captured gives an eager call, before any replay,
    its own bias, and follows a bias changed between replays."""
    mod, y, x = layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mod(x)
    assert torch.equal(mod(x), y)
    for i in range(3):
        with torch.no_grad():
            mod.bias.mul_(0.5 if i else 1.0)
        eager = mod(x)
        fill = [torch.full((N,), 9.0, dtype=BF, device="cuda") for _ in range(16)]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i
        del fill


def test_a_captured_call_after_an_eager_one():
    """The same with an eager call in front, which has left a copy of the bias."""
    mod, y, x = layer()
    assert torch.equal(mod(x), y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mod(x)
    for i in range(3):
        with torch.no_grad():
            mod.bias.add_(1.0)
        eager = mod(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and not torch.equal(eager, y), i


def test_first_calls_on_two_streams():
    """The second stream does not read a copy that the first has yet to write."""
    mod, y, x = layer()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        torch.cuda._sleep(20_000_000)            # some ms in front of the first call
        ya = mod(x)
    with torch.cuda.stream(b):
        yb = mod(x)
    torch.cuda.synchronize()
    assert torch.equal(ya, y) and torch.equal(yb, y)
