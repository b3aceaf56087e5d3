"""svdq_block_norm and its backward pass on two streams at once."""

import pytest
import torch

from tests import test_gpu_block_norm as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [((700, 1032), (37, 4096)), ((64, 12288), (9, 16383)), ((1, 7), (600, 264))])
def test_two_streams(sizes):
    """Forward and backward calls on two streams at once."""
    ps = [B.problem(m, d, "layer", 1) for m, d in sizes]
    want = [B.call(p) + B.call_grad(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [None, None]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = B.call(ps[i]) + B.call_grad(ps[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
