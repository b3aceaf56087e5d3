"""The modules on rows that start between 16-byte addresses."""

import pytest
import torch

from tests.test_gpu_w4a16_modules import block, linear
from w4a4_quantized_diffusion_amd import linear as L

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_block_on_a_slice_of_a_flat_buffer():
    b = block(128, 192)
    x, dy = torch.randn(5, 128, device="cuda").to(BF), torch.randn(5, 128, device="cuda").to(BF)
    flat = torch.cat((torch.zeros(3, dtype=BF, device="cuda"), x.flatten())).requires_grad_()
    a = x.clone().requires_grad_()
    ya = b(a)
    ya.backward(dy)
    y = b(flat[3:].view_as(x))
    assert torch.equal(y, ya)
    # the gradient of the concatenation reaches the block at an odd address too
    one = torch.zeros(1, dtype=BF, device="cuda")
    torch.cat((one, y.flatten())).backward(torch.cat((one, dy.flatten())))
    assert torch.equal(flat.grad[3:].view_as(x), a.grad)


@pytest.mark.parametrize("rows", [3, 40])
def test_svdq_linear_on_a_slice(rows):
    m = L.SVDQLinear.from_linear(linear(128, 192, 5), rank=16, a16_rows=8)
    x = torch.randn(rows, 128, device="cuda").to(BF)
    flat = torch.zeros(1 + x.numel(), dtype=BF, device="cuda")
    flat[1:] = x.flatten()
    assert torch.equal(m(flat[1:].view_as(x)), m(x))
