"""awq_linear_w4a16_res_grad with a gate of its own for each of 2^20 rows, which is more
than one launch's threads."""

import pytest
import torch

from w4a4_quantized_diffusion_amd import svdq
from tests.test_gpu_moe import experts, weight

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -24


def test_gate_of_every_row():
    """The rows at the ends and around the launches' border (2^23 workgroups, 16 a row)
    as in a call of their own, to the bit; dX from the rounded dZ: N fp32 roundings of its
    sum and the rounding to bf16."""
    m, k, n = 1 << 20, 64, 8192
    torch.cuda.empty_cache()
    lay = experts(1, n, k, 3)
    layer = dict(N=n, K=k, group=64, **{f: lay[f][0] for f in ("q", "scales", "zeros")})
    dy, z, gate = (torch.empty((m, n), dtype=BF, device="cuda").normal_() for _ in range(3))
    dx, dz, dgate = svdq.awq_linear_w4a16_res_grad(dy, z, layer, "silu", gate)
    w = weight(lay, 0)
    half = (1 << 23) // 16
    for r in (slice(0, 3), slice(half - 3, half + 3), slice(m - 5, m)):
        _, dz0, dgate0 = svdq.awq_linear_w4a16_res_grad(dy[r], z[r], layer, "silu", gate[r])
        assert torch.equal(dz[r], dz0) and torch.equal(dgate[r], dgate0)
        d = dz[r].double()
        ref, size = d @ w, d.abs() @ w.abs()
        assert bool(((dx[r].double() - ref).abs() <= n * U * size + 2.0 ** -8 * ref.abs()).all())
