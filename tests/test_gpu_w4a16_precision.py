"""What the weight-only operators promise of their precision, pinned closely enough that
a lost term, a lost derivative or a missing half of the gated block fails.

bf16 has 8 significant bits: a rounding is off by at most 2^-8 of the value.  Three
bf16 terms hold any fp32 number exactly away from underflow: the first leaves at most
2^-8 of a leading bit's 2^e, the second 2^-17, and what is left is a multiple of
2^(e-23), at most 6 bits, which the third holds.
"""

import numpy as np
import pytest
import torch

from oracle import svdq as O
from tests.gpu_helpers import gm_codes, gm_int4, t_u8
from tests.test_gpu_w4a16 import BF, F32, act64, awq_layer, bf, check, svdq_layer
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


# ------------------------------------------------- fp32 outputs of a16

def full_mantissas(m, k, seed):
    """fp32 numbers with their lowest bit set.  Two bf16 terms are not enough for them,
    but for the few whose first term leaves less than 2^(e-15), which the second
    holds whole (a share of about 2^-7)."""
    g = torch.Generator("cuda").manual_seed(seed)
    # bits 8 and 9 set too, so that the first term always leaves something
    mant = torch.randint(0, 1 << 23, (m, k), generator=g, device="cuda", dtype=torch.int32) | 0x301
    exp = torch.randint(117, 138, (m, k), generator=g, device="cuda", dtype=torch.int32)
    sign = torch.randint(0, 2, (m, k), generator=g, device="cuda", dtype=torch.int32)
    x = (mant | (exp << 23) | (sign << 31)).view(F32)
    t1 = x.to(BF).float()
    t2 = (x - t1).to(BF).float()
    t3 = (x - t1 - t2).to(BF).float()
    assert (t2 != 0).all() and (t3 != 0).float().mean() > 0.9
    assert torch.equal(t1.double() + t2.double() + t3.double(), x.double())
    return x


def one_weight_layer(n, k, prec, seed):
    """A layer of rank 0 with unit scales and smoothing and one weight 1, 2 or 4 or its
    negative per output: (layer, k of every output, the weights in float64)."""
    g = np.random.default_rng([seed, n, k])
    at, e, neg = g.integers(0, k, n), g.integers(0, 3, n), g.integers(0, 2, n)
    w = (1 << e) * (1 - 2 * neg)
    one = torch.ones(1, device="cuda")
    d = dict(rank=0, prec=0 if prec == "int4" else 1, N=n, K=k, smooth=torch.ones(k, device="cuda"),
             w_tensor_scale=one, x_tensor_scale=one.clone(),
             lora_down=torch.zeros(1, dtype=torch.int16, device="cuda"),
             lora_up=torch.zeros(1, dtype=torch.int16, device="cuda"))
    if prec == "int4":
        q = np.zeros((n, k), dtype=np.int64)
        q[np.arange(n), at] = w
        d["wcodes"] = t_u8(gm_int4(O.pack_int4(q)))
        d["wscales"] = torch.ones(k // 64, n, device="cuda")
    else:
        nib = np.zeros((n, k), dtype=np.uint8)                     # E2M1: 1, 2, 4 are 2, 4, 6
        nib[np.arange(n), at] = 2 * (e + 1) + 8 * neg
        d["wcodes"] = t_u8(gm_codes(nib[:, 0::2] | (nib[:, 1::2] << 4)))
        d["wscales"] = torch.full((k // 64, n, 4), 0x38, dtype=torch.uint8, device="cuda")     # E4M3 1
    return d, torch.from_numpy(at).cuda(), torch.from_numpy(w).double().cuda()


# 16 columns a wave and 32, one to four blocks of rows, one slice of K and many
SHAPES = [(1, 64, 16), (3, 512, 272), (17, 2048, 208), (40, 8256, 48), (64, 256, 144), (5, 192, 8208),
          (50, 128, 8208)]


@pytest.mark.parametrize("m,k,n", SHAPES)
@pytest.mark.parametrize("prec", ["int4", "nvfp4"])
def test_fp32_products_are_exact(m, k, n, prec):
    """One weight that is a power of two per output: x times it is an fp32 number, and
    so is every partial sum, so Y is exact; two terms of x would leave 2^-17 of it."""
    print(f"exact {m} {k} {n} {prec}", flush=True)
    d, at, w = one_weight_layer(n, k, prec, 51)
    x = full_mantissas(m, k, 52)
    Y = svdq.svdq_linear_w4a16(x, d)
    assert torch.equal(Y.double(), x[:, at].double() * w)
    # in bf16: the rounding, and two terms
    Y = svdq.svdq_linear_w4a16(x, d, y_dtype=BF)
    ref = x[:, at].double() * w
    check(Y, ref, ref.abs() * (2.0 ** -8 + 2.0 ** -17), "bf16")


@pytest.mark.parametrize("m,k,n,rank", [(1, 64, 16, 16), (3, 512, 272, 48), (17, 8256, 208, 64),
                                        (64, 1024, 144, 256), (50, 128, 8208, 80)])
@pytest.mark.parametrize("prec", ["int4", "nvfp4"])
def test_fp32_low_rank_branch_is_exact(m, k, n, rank, prec):
    """No residual weights, one 1 per row of lora_down and one power of two per row of
    lora_up: LR is a column of x, and Y a multiple of it, both exact in fp32."""
    print(f"exact low rank {m} {k} {n} {rank} {prec}", flush=True)
    d, _, _ = one_weight_layer(n, k, prec, 53)
    d["wcodes"] = torch.zeros_like(d["wcodes"])
    g = torch.Generator("cuda").manual_seed(54)
    at = torch.randint(0, k, (rank,), generator=g, device="cuda")
    to = torch.randint(0, rank, (n,), generator=g, device="cuda")
    w = 2.0 ** torch.randint(-2, 3, (n,), generator=g, device="cuda").float()
    down = torch.zeros(rank, k, device="cuda")
    down[torch.arange(rank), at] = 1
    up = torch.zeros(n, rank, device="cuda")
    up[torch.arange(n), to] = w
    d.update(rank=rank, lora_down=down.to(BF).view(torch.int16), lora_up=up.to(BF).view(torch.int16))
    # the residual branch reads X times its smoothing, the low-rank branch X itself
    d["smooth"] = torch.full_like(d["smooth"], 0.37)
    x = full_mantissas(m, k, 55)
    assert torch.equal(svdq.svdq_linear_w4a16(x, d).double(), x[:, at[to]].double() * w.double())


@pytest.mark.parametrize("m,k,n", [(1, 192, 48), (17, 1088, 8208), (64, 320, 272)])
@pytest.mark.parametrize("prec", ["int4", "nvfp4"])
def test_fp32_near_the_top_of_the_range(m, k, n, prec):
    """A value of 3e38 times weights of size one at most (before their scale): three
    products summed, the scale and the join with zeros, at most 8 roundings of 2^-24."""
    d, parts = svdq_layer(n, k, 0, prec, 99)
    d["smooth"] = torch.ones_like(d["smooth"])
    x = torch.zeros(m, k, device="cuda")
    x[m - 1, 1] = 3.0e38
    scale = d["wscales"][0].double() if prec == "int4" else d["w_tensor_scale"].double()
    w = parts[1][:, 1]
    fits = w.abs() / scale <= 1.001
    assert fits.any()
    ref = x[m - 1, 1].double() * w
    Y = svdq.svdq_linear_w4a16(x, d)
    check(Y[m - 1][fits], ref[fits], ref[fits].abs() * 2.0 ** -21, "large")
