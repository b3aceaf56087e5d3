"""The layer norm's mean: rows of equal values, and rows whose mean is large against
their deviation, in svdq_block_norm and its backward pass.

A row's sum is 64 bits wide: k v for up to 2^14 equal fp32 values is exact, and with it
the mean, so that every difference is zero.  Otherwise the mean is known to 2 u^2 of
itself (u = 2^-24: an fp32 value and the fp32 value of what it leaves out), and a
difference v - mean takes two roundings of about its own size: 2 u |v - mean| + 2 u^2
|mean|, where the bounds of tests/test_gpu_block_norm.py allow 40 u mean |v|.  The rest of
those bounds stands."""

import pytest
import torch

from tests import test_gpu_block_norm as B

pytestmark = pytest.mark.gpu

BF, F32, U = B.BF, B.F32, B.U


def norm64(v, e, kind, eps):
    """n, r and the error bound of n, from v with error e (B.norm64 with the mean's own
    error as above)."""
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    r = ((v - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    n = (v - mean) * r
    e = e + e.mean(-1, keepdim=True) if kind == "layer" else e
    a = r * (2 * U * (v - mean).abs() + 2 * U * U * mean.abs() + e)
    return n, r, a + n.abs() * (24 * U + (n.abs() * a).mean(-1, keepdim=True))


@pytest.fixture
def exact_mean(monkeypatch):
    monkeypatch.setattr(B, "norm64", norm64)


@pytest.mark.parametrize("d", [1, 7, 64, 768, 1000, 1024, 4099, 5455, 8192, 12288, 16383])
@pytest.mark.parametrize("xt", [F32, BF])
def test_equal_values(d, xt):
    """n is zero: y is the shift, x' with a post norm is x, and the gradients that are
    sums of products with n are zeros."""
    p = B.problem(6, d, "layer", xt=xt, ht=xt, yt=F32, vt=F32)
    values = torch.tensor([0.1, 3.0, 1000.0, -30000.0, 3e37, 1e-30], device="cuda")
    p["x"] = values.to(xt)[:, None].expand(6, d).contiguous()
    p["h"] = p["x"].flip(0).contiguous()
    xo, y = B.call(p)
    assert torch.equal(xo, p["x"]) and torch.equal(y, p["shift"].expand(6, d))
    dpost, dgate, dweight, dscale, dshift = B.call_grad(p)[2:]
    for v in (dpost, dgate, dweight, dscale):
        assert not v.any()
    # six fp32 terms in any order: five roundings of partial sums
    dy = p["dy"].double()
    B.check(dshift.flatten(), dy.sum(0), 5 * U * dy.abs().sum(0), "dshift")


@pytest.mark.parametrize("d", [7, 200, 1000, 4096, 4099, 5455, 12288])
@pytest.mark.parametrize("mean", [3e4, -1e6])
def test_large_mean(exact_mean, d, mean):
    g = torch.Generator(device="cuda").manual_seed(d)
    p = B.problem(5, d, "layer", xt=F32, yt=F32, vt=F32, h=False)
    p["x"] = B.draw(g, (5, d), F32, 1.0, mean)
    B.check_forward(p)
    B.check_grad(p)
    # in front of a post norm
    p = B.problem(5, d, "layer", xt=F32, ht=F32, yt=F32, vt=F32)
    p["h"] = B.draw(g, (5, d), F32, 1.0, mean)
    B.check_forward(p)
    B.check_grad(p)


@pytest.mark.parametrize("m,d", B.SHAPES)
def test_shapes(exact_mean, m, d):
    for xt, yt in ((BF, BF), (F32, F32)):
        p = B.problem(m, d, "layer", xt=xt, ht=xt, yt=yt, vt=xt)
        B.check_forward(p, 1e-5)
        B.check_grad(p, 1e-5)
