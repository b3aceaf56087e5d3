"""What the weight-only operators promise of their precision, pinned closely enough that
a lost term, a lost derivative or a missing half of the gated block fails.

bf16 has 8 significant bits: a rounding is off by at most 2^-8 of the value.
"""

import pytest
import torch

from tests.test_gpu_w4a16 import act64, awq_layer, bf, check
from w4a4_quantized_diffusion_amd import svdq

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- gated gradient

def wrong_gradients(x, wg, wu, dh, act):
    """dX with something missing, each of which the bound below has to notice."""
    g, u = x @ wg.t(), x @ wu.t()
    a, da = act64(g, act)
    s = a / torch.where(g == 0, torch.ones_like(g), g)             # the sigmoid alone
    return {"nothing": torch.zeros_like(x),
            "act' without x s'": (dh * u * s) @ wg + (dh * a) @ wu,
            "no up half": (dh * u * da) @ wg,
            "no gate half": (dh * a) @ wu,
            "act of the up half": (dh * u * da) @ wg + (dh * u * act64(u, act)[1]) @ wu}


@pytest.mark.parametrize("m,k,n", [(5, 128, 48), (40, 192, 80), (130, 128, 64), (1100, 64, 48)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradient_element_by_element(m, k, n, act):
    """Forward and backward pass together against the float64 block: dX of every
    element, whose formula is itself held against central differences.  First-order
    bound of the bf16 roundings on the way: G and U as stored, dG and dU before the
    products, dX (2^-8 each; |act'| <= 1.13, |act''| <= 0.8)."""
    print(f"gradient {m} {k} {n} {act}", flush=True)
    gate, wg = awq_layer(n, k, 41)
    up, wu = awq_layer(n, k, 42)
    xb, dhb = bf((m, k), 43), bf((m, n), 44)
    _, G, U = svdq.awq_gated_w4a16(xb, gate, up, act, save=True)
    dX, _, _ = svdq.awq_gated_w4a16_grad(dhb, G, U, gate, up, act)
    x, dh = xb.double(), dhb.double()
    g, u = x @ wg.t(), x @ wu.t()
    a, da = act64(g, act)
    dx = (dh * u * da) @ wg + (dh * a) @ wu

    def rows(x):
        return (act64(x @ wg.t(), act)[0] * (x @ wu.t()) * dh).sum(1)

    e = 1e-5
    for c in range(0, k, 7):
        d = torch.zeros(k, dtype=torch.float64, device="cuda")
        d[c] = e
        num = (rows(x + d) - rows(x - d)) / (2 * e)
        assert ((num - dx[:, c]).abs() <= 1e-6 * (1 + (dh * u).abs().sum(1) + dh.abs().sum(1))).all()

    r, h, G1, U1 = 2.0 ** -8, dh.abs(), g.abs(), u.abs()
    edg = h * U1 * da.abs() * 2 * r + h * U1 * 0.8 * G1 * r        # dG and U, then G through act'
    edu = h * a.abs() * r + h * 1.13 * G1 * r                      # dU, then G through act
    tol = (edg @ wg.abs() + edu @ wu.abs()) * (1 + 2.0 ** -6) + dx.abs() * r + 1e-30
    check(dX, dx, tol, "dX")
    for name, bad in wrong_gradients(x, wg, wu, dh, act).items():
        assert ((bad - dx).abs() > 2 * tol).float().mean() > 0.3, name

