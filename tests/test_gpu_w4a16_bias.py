"""Biases at odd element offsets: the calls ask no more of them than the alignment
of their elements, in every form of the operators.  Tolerances as in
test_gpu_w4a16.py."""

import pytest
import torch

from tests.test_gpu_w4a16 import (BF, F32, a16_ref, awq_layer, bf, check, gated_ref, round_tol,
                                  svdq_layer)
from w4a4_quantized_diffusion_amd import svdq

pytestmark = pytest.mark.gpu


def odd(t):
    """The same values one element behind an aligned address."""
    v = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:]
    v.copy_(t)
    assert v.data_ptr() % (2 * t.element_size()) == t.element_size() and v.is_contiguous()
    return v


# one launch; slices of K (wide and narrow) with a second launch; the 128 x 128 tiles
# with and without slices; the 256 x 256 tiles; these with a rest of few rows
@pytest.mark.parametrize("m,k,n", [(3, 256, 80), (33, 8192, 272), (64, 4160, 1008), (130, 2048, 144),
                                   (300, 192, 8208), (2050, 320, 336), (4099, 2048, 4112)])
def test_gated(m, k, n):
    print(f"odd biases {m} {k} {n}", flush=True)
    gate, wg = awq_layer(n, k, 1)
    up, wu = awq_layer(n, k, 2)
    x, bg, bu = bf((m, k), 3), bf((n,), 4, 0.3), bf((n,), 5, 0.3)
    (g, tg), (u, tu), (h, th) = gated_ref(x, wg, wu, bg, bu, "silu")
    H, G, U = svdq.awq_gated_w4a16(x, gate, up, "silu", odd(bg), odd(bu), save=True)
    check(H, h, th + round_tol(h, BF) + 1e-30, "H")
    check(G, g, tg + round_tol(g, BF) + 1e-30, "G")
    check(U, u, tu + round_tol(u, BF) + 1e-30, "U")
    # aligned biases, and one of them alone, give the same bits
    assert torch.equal(H, svdq.awq_gated_w4a16(x, gate, up, "silu", bg, bu))
    for b in ((bg, None), (None, bu)):
        o = [None if t is None else odd(t) for t in b]
        assert torch.equal(svdq.awq_gated_w4a16(x, gate, up, "silu", *o, h_dtype=F32),
                           svdq.awq_gated_w4a16(x, gate, up, "silu", *b, h_dtype=F32))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a16(dtype):
    m, k, n = 5, 512, 272
    d, parts = svdq_layer(n, k, 16, "int4", 6)
    x, bias = bf((m, k), 7), bf((n,), 8).to(dtype)
    y, tol = a16_ref(x, parts, bias, 2.0 ** -24)
    Y = svdq.svdq_linear_w4a16(x, d, odd(bias))
    check(Y, y, tol + round_tol(y, F32) + 1e-30, "Y")
    assert torch.equal(Y, svdq.svdq_linear_w4a16(x, d, bias))
