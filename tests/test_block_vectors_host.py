"""Which rows of x a module takes a vector's row for: a gate, scale or shift [images, dim]
goes with the first dimension of x, or the first ones together, and one laid out otherwise (a
row per token of every image, as torch would broadcast it) is refused instead of being taken
for other rows.  Without a GPU: what is accepted gets as far
as the library's check for a device tensor."""

import pytest
import torch

from w4a4_quantized_diffusion_amd import linear as L

BF = torch.bfloat16
D = 64


def awq(n, k):
    return L.AWQLinear(dict(N=n, K=k, group=64, q=torch.zeros((k // 64, n, 32), dtype=torch.uint8),
                            scales=torch.zeros((k // 64, n), dtype=torch.int16),
                            zeros=torch.zeros((k // 64, n), dtype=torch.int16)))


def calls(shape, vector):
    """The module's calls on x of the leading `shape` with one vector of every kind."""
    norm, lin = L.BlockNorm(D), awq(D, 128)
    x, v = torch.zeros(*shape, D, dtype=BF), torch.zeros(*vector, D)
    wide = torch.zeros(*shape, 128, dtype=BF)
    return [lambda: norm(x, x, gate=v), lambda: norm(x, scale=v), lambda: norm(x, shift=v),
            lambda: lin(wide, gate=v)]


@pytest.mark.parametrize("shape,vector", [
    ((2, 8), (8,)), ((2, 8), (4,)), ((2, 8), (1, 8)), ((2, 8), (8, 1)), ((2, 8), (2, 4)),
    ((4, 2, 3), (2,)), ((4, 2, 3), (3,)), ((4, 2, 3), (6,)), ((4, 2, 3), (1, 2, 1)), ((4, 2, 3), (4, 1, 3)),
    ((4, 2, 3), (1, 1, 3)), ((4, 2, 3), (2, 4, 1)), ((2, 1, 8), (8,)), ((2, 1, 8), (1, 1, 8))])
def test_refused(shape, vector):
    for call in calls(shape, vector):
        with pytest.raises(ValueError, match="rows"):
            call()


@pytest.mark.parametrize("shape,vector", [
    ((2, 8), ()), ((2, 8), (1,)), ((2, 8), (1, 1)), ((2, 8), (2,)), ((2, 8), (2, 1)), ((2, 8), (2, 8)),
    ((2, 8), (16,)), ((4, 2, 3), (4,)), ((4, 2, 3), (8,)), ((4, 2, 3), (24,)), ((4, 2, 3), (4, 1, 1)),
    ((4, 2, 3), (4, 2)), ((4, 2, 3), (4, 2, 3)), ((2, 1, 8), (2, 1, 1)), ((2, 1, 8), (2, 1, 8)),
    # rows along one dimension: runs of them
    ((1, 6), (6,)), ((1, 6), (1, 6)), ((1, 6), (3,)), ((6, 1), (3,)), ((6,), (3,)), ((6,), (6,)), ((6,), (3, 1)),
    ((6,), (1,)), ((), (1,)), ((), ())])
def test_accepted(shape, vector):
    for call in calls(shape, vector):
        with pytest.raises(ValueError, match="device tensor"):
            call()
