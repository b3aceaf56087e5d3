"""awq_moe_w4a16 on layers wide enough that the down-projections need no slices (K from
8192 on: 32 columns a workgroup, Y written by it), with the bounds of
tests/test_gpu_moe.py; and calls of it on two streams at once."""

import pytest
import torch

from tests import test_gpu_moe as M

pytestmark = pytest.mark.gpu

BF = M.BF


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("t,e,top,k,n", [(1, 8, 2, 8192, 128), (1, 3, 3, 8256, 64), (5, 4, 2, 8256, 64),
                                          (64, 2, 2, 8192, 64), (64, 6, 1, 8192, 192), (33, 40, 6, 8192, 64),
                                          (2, 5, 5, 12288, 320)])
def test_sizes(t, e, top, k, n, act):
    M.check_all(M.problem(t, e, top, k, n), act, True)
    M.check_all(M.problem(t, e, top, k, n, BF, seed=7), act, False)


@pytest.mark.parametrize("k,n", [(8192, 64), (1024, 320)])
def test_rows_behind(k, n):
    """Y, ids and weights of a call on fewer tokens than their buffers hold."""
    p = M.problem(9, 8, 2, k, n)
    want = M.call(p)
    buf = torch.full((12, k), 7.0, dtype=BF, device="cuda")
    got = M.call(p, Y=buf[:9])
    assert torch.equal(got, want) and bool((buf[9:] == 7).all())


def test_two_streams():
    """One and many tokens, with and without slices, side by side."""
    ps = [M.problem(*s, seed=i) for i, s in enumerate([(1, 8, 2, 1024, 320), (61, 40, 6, 512, 192),
                                                       (64, 2, 2, 8192, 64), (17, 5, 2, 576, 192)])]
    want = [M.call(p, routing=True) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for a, b in ((0, 1), (1, 2), (2, 3), (3, 3)):
        got = {}
        for _ in range(10):
            for i, st in zip((a, b), streams):
                with torch.cuda.stream(st):
                    got[st] = (i, M.call(ps[i], routing=True))
        torch.cuda.synchronize()
        for i, out in got.values():
            for x, y in zip(out, want[i]):
                assert torch.equal(x, y)
