"""svdq_block_norm_grad with vectors of many images (modulation per token) beside shared
ones, whose gradients are sums over all images of products with each image's factors."""

import statistics

import pytest
import torch

from tests import test_gpu_block_norm as B

pytestmark = pytest.mark.gpu

F32 = B.F32


@pytest.mark.parametrize("images,rows", [(2, 4), (63, 1), (64, 1), (65, 1), (513, 3), (512, 9), (1500, 1),
                                          (1024, 2), (300, 4), (129, 40),
                                          (40, 60), (20, 60), (33, 31)])
@pytest.mark.parametrize("d", [1, 72, 1000])
def test_sums_over_images(images, rows, d):
    for kind, vt in (("layer", F32), ("rms", B.BF)):
        p = B.problem(images * rows, d, kind, images, xt=F32, ht=F32, yt=F32, vt=vt)
        B.check_grad(p)
        again = B.call_grad(p)
        for a, b in zip(B.call_grad(p), again):
            assert torch.equal(a, b)


@pytest.mark.parametrize("images,rows", [(1, 9), (3, 50), (70, 2), (300, 1)])
@pytest.mark.parametrize("d", [200, 4099])
def test_post_and_weight_of_every_image(images, rows, d):
    """Beside shared gates, scales and shifts, and with all of them per image."""
    g = torch.Generator(device="cuda").manual_seed(d + images)
    for shared in (("gate", "scale", "shift"), ("scale",), ()):
        p = B.problem(images * rows, d, "layer" if rows > 1 else "rms", images, xt=F32, ht=B.BF, yt=F32,
                      vt=F32, shared=shared)
        for f in ("post", "weight"):
            p[f] = B.draw(g, (images, 2 * d + 3), F32, 0.3, 1.0)[:, 3:3 + d]
        B.check_forward(p)
        B.check_grad(p)


def test_bad_factors_stay_in_their_columns():
    """An infinite scale in one image's column: that column's sums only."""
    p = B.problem(700, 264, "layer", 700, vectors=("weight", "scale", "gate", "post"), xt=F32)
    want = B.call_grad(p)[4]
    p["scale"] = p["scale"].clone()
    p["scale"][650, 100] = float("inf")
    got = B.call_grad(p)[4]
    # (row 650's own gradient is infinite; its sum dY n is not)
    assert not torch.isfinite(got[100])
    keep = torch.arange(264, device="cuda") != 100
    assert torch.equal(got[keep], want[keep])


def test_many_images_are_not_summed_one_after_the_other():
    """A vector for each of 4608 rows moves 2.4 times the bytes of one for all of them, and
    takes 8 times as long; image after image its sums took 57 times as long."""
    def time(images):
        p = B.problem(4608, 4096, "layer", images)
        took = []
        for _ in range(7):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(3):
                B.call_grad(p)
            b.record()
            b.synchronize()
            took.append(a.elapsed_time(b))
        return statistics.median(took)
    assert time(4608) < 20 * time(1)
