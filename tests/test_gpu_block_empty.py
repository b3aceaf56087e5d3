"""The backward passes of the operators around a block on no rows: the vectors' gradients
are zeros, whatever the vectors hold."""

import pytest
import torch

from w4a4_quantized_diffusion_amd import svdq

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 1.0])
@pytest.mark.parametrize("images", [1, 2, 3])
def test_norm_without_rows(bad, images):
    """Shared vectors beside vectors of every image, and the other way round."""
    d = 96
    x = torch.empty((0, d), dtype=BF, device="cuda")
    each, one = (torch.full(s, bad, device="cuda") for s in ((images, d), (d,)))
    for post, gate, weight, scale, shift in ((one, each, one, each, each), (each, one, each, one, one),
                                             (one, one, one, one, one)):
        got = svdq.svdq_block_norm_grad(x, x, x, x, "layer", 1e-6, post, gate, weight, scale, shift)
        assert got[0].shape == got[1].shape == (0, d)
        for v, dv in zip((post, gate, weight, scale, shift), got[2:]):
            assert dv.shape == v.shape and torch.equal(dv, torch.zeros_like(dv))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_product_without_rows(bad):
    k, n = 128, 64
    layer = dict(N=n, K=k, group=64, q=torch.zeros((k // 64, n, 32), dtype=torch.uint8, device="cuda"),
                 scales=torch.zeros((k // 64, n), dtype=torch.int16, device="cuda"),
                 zeros=torch.zeros((k // 64, n), dtype=torch.int16, device="cuda"))
    z = torch.empty((0, n), dtype=BF, device="cuda")
    for images in (1, 3):
        gate = torch.full((images, n), bad, device="cuda")
        dx, dz, dgate = svdq.awq_linear_w4a16_res_grad(z, z, layer, "gelu", gate)
        assert dx.shape == (0, k) and dz.shape == (0, n)
        assert torch.equal(dgate, torch.zeros_like(gate))
